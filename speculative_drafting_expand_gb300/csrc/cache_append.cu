// cache_append.cu -- new rows of q, k and v into a paged KV cache: rotate-half
// rotary embedding of q and k at the row's position, k and v stored in the
// position's page slot (include/peagle_cache.h).
#include <algorithm>

#include "cache_common.cuh"
#include "pe_kernels.h"

namespace pe {

struct AppendArgs {
  CachePool pool;
  int T, B, Hq, Hkv, bt_stride;
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride, qo_stride;
  const int32_t* pos;
  const int32_t* req;
  const int32_t* block_table;
  void* q_out;
  int* err;
  float k_scale, v_scale;
  RopeSteps rope;
};

// A chunk of activations into a pool, as the pool holds it.
template <typename S, int N>
__device__ __forceinline__ void store_kv(void* base, size_t at, const float (&x)[N], float scale) {
  if constexpr (sizeof(S) == 1) {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
             (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale),
                                                    __fdiv_rn(x[4 * i + 3], scale)))
              << 16);
    static_assert(N == 8, "bf16 activations beside e4m3 pools");
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + at) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<S*>(base) + at) = Chunk<S>::put(x);
  }
}

// A CTA a row.  A thread takes 16 bytes of a head's low half and the 16 of
// its high half that they pair with (q heads, then k heads); more threads
// copy v.  Bound by bytes for many rows and by latency for few: every load is
// on its way before the first use, and the row's sines and cosines (one pair
// a thread, shared by all heads) are worked out meanwhile.  With more rows
// than CTAs fit, a CTA takes every grid-th row and the next row's first loads,
// one item a thread, are under way while it finishes one.  Measured (GB300):
// one row of 64 + 8 heads of 64, 2.4 us, a launch's latency; 2048 rows of 32 +
// 4 heads of 128, 11 us, 3.8 TB/s: 912 CTAs of 192 threads take 2.2 rows each,
// and of a row's 320 items the 128 that no thread has loaded ahead wait for
// memory when they are used.
constexpr int kAppendMost = 384;
constexpr int kAppendCtas = 3;  // an SM

template <typename A, typename S, int DH>
__global__ void __launch_bounds__(kAppendMost, kAppendCtas) kv_append_kernel(
    const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using C = Chunk<A>;
  constexpr int N = C::N;        // elements of a chunk
  constexpr int HALF = DH / N / 2;  // threads of a head
  __shared__ __align__(16) float cs2[2][DH / 2], sn2[2][DH / 2];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int hq = a.q ? a.Hq : 0, heads = hq + a.Hkv;
  const int turned = heads * HALF, all = turned + a.Hkv * HALF;
  // this thread's chunks of item w: of a head that turns, or of one of v
  auto load = [&](int t, int w, uint4 (&x)[2]) {
    const int h = w / HALF, c = w % HALF;
    const A* src = w < hq * HALF ? static_cast<const A*>(a.q) + t * a.q_stride + h * DH
                   : w < turned
                       ? static_cast<const A*>(a.k) + t * a.k_stride + (h - hq) * DH
                       : static_cast<const A*>(a.v) + t * a.v_stride + (h - heads) * DH;
    if (w < all) {
      x[0] = *reinterpret_cast<const uint4*>(src + c * N);
      x[1] = *reinterpret_cast<const uint4*>(src + DH / 2 + c * N);
    }
  };
  uint4 next[2];
  load(blockIdx.x, tid, next);
  int p_next = a.pos[blockIdx.x], r_next = a.req ? a.req[blockIdx.x] : blockIdx.x;
  int odd = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    uint4 x[2] = {next[0], next[1]};
    const int p = p_next, r = r_next;
    if (const int u = t + gridDim.x; u < a.T) {
      load(u, tid, next);
      p_next = a.pos[u];
      r_next = a.req ? a.req[u] : u;
    }
    if (p < 0) continue;  // padding
    int blk = -1;
    if (r < 0 || r >= a.B) {
      if (tid == 0) record_error(a.err, PE_DEV_BAD_ROW);
    } else if (p >= static_cast<long long>(a.bt_stride) * kPage) {
      if (tid == 0) record_error(a.err, PE_DEV_BAD_POSITION);
    } else {
      blk = a.block_table[static_cast<size_t>(r) * a.bt_stride + p / kPage];
      if (blk < 0 || blk >= a.pool.num_blocks) {
        if (tid == 0) record_error(a.err, PE_DEV_BAD_BLOCK);
        blk = -1;
      }
    }
    float* cs = cs2[odd];  // the other pair may still be read for the row before
    float* sn = sn2[odd];
    odd ^= 1;
    if (a.rope.on) {
      for (int i = tid; i < DH / 2; i += threads) rope_cos_sin(a.rope.step[i], p, cs[i], sn[i]);
      __syncthreads();
    }
    const int off = p % kPage;
    // element (head, 0) of the row's slot
    auto slot = [&](int h) {
      return ((static_cast<size_t>(blk) * a.Hkv + h) * kPage + off) * DH;
    };
    for (int w = tid; w < all; w += threads) {
      if (w >= threads) load(t, w, x);
      const int h = w / HALF, c = w % HALF * N;
      float u[N], y[N];
      C::get(x[0], u);
      C::get(x[1], y);
      if (a.rope.on && w < turned) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float4 co = *reinterpret_cast<const float4*>(cs + c + e);
          const float4 si = *reinterpret_cast<const float4*>(sn + c + e);
          const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float z = u[e + i] * cc[i] - y[e + i] * ss[i];
            y[e + i] = y[e + i] * cc[i] + u[e + i] * ss[i];
            u[e + i] = z;
          }
        }
      }
      if (h < hq) {
        A* out = static_cast<A*>(a.q_out) + t * a.qo_stride + h * DH + c;
        *reinterpret_cast<uint4*>(out) = C::put(u);
        *reinterpret_cast<uint4*>(out + DH / 2) = C::put(y);
      } else if (blk >= 0) {
        const bool key = h < heads;
        void* pool = key ? a.pool.k : a.pool.v;
        const size_t at = slot(key ? h - hq : h - heads) + c;
        const float scale = key ? a.k_scale : a.v_scale;
        store_kv<S>(pool, at, u, scale);
        store_kv<S>(pool, at + DH / 2, y, scale);
      }
    }
    if (a.pool.scores && blk >= 0)
      for (int h = tid; h < a.Hkv; h += threads)
        a.pool.scores[(static_cast<size_t>(blk) * a.Hkv + h) * kPage + off] = 0.f;
  }
}

template <typename A, typename S, int DH>
static cudaError_t launch_append_dim(const AppendArgs& a, int sms, cudaStream_t s) {
  const long long items =
      (static_cast<long long>(a.q ? a.Hq : 0) + 2 * a.Hkv) * (DH / Chunk<A>::N / 2);
  // Few rows: a thread for everything a row has, for the shortest way through.
  // More rows than CTAs of that size: half the threads and twice the CTAs, so
  // that more rows are at different stages (2048 rows of 32 + 4 heads of 128:
  // 10.6 us against 12.2; one row: 2.9 against 2.5).
  const bool many = a.T > kAppendCtas * sms;
  const int most = many ? kAppendMost / 2 : kAppendMost;
  const int threads = static_cast<int>(std::min<long long>(most, (items + 31) / 32 * 32));
  const int ctas = (many ? 2 : 1) * kAppendCtas * sms;
  return launch_pdl(kv_append_kernel<A, S, DH>, dim3(std::min(a.T, ctas)), dim3(threads), 0, s, a);
}
template <typename A, typename S>
static cudaError_t launch_append(const AppendArgs& a, int dh, int sms, cudaStream_t s) {
  return dh == 64 ? launch_append_dim<A, S, 64>(a, sms, s) : launch_append_dim<A, S, 128>(a, sms, s);
}

}  // namespace pe

extern "C" pe_status pe_kv_append(const pe_kv_pool* pool, int32_t T, int32_t B, int32_t n_heads,
                                  float rope_theta, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, const int32_t* pos, const int32_t* req,
                                  const int32_t* block_table, int32_t bt_stride, void* q_out,
                                  int64_t q_out_stride, int32_t* err, void* stream) {
  using namespace pe;
  if (const pe_status st = check_pool(pool); st != PE_OK) return st;
  const int dh = pool->head_dim, eb = act_elem_bytes(pool->dtype);
  const int64_t kw = static_cast<int64_t>(pool->n_kv_heads) * dh;
  if (T < 1 || B < 1 || (!req && T != B) || !pos || !block_table || bt_stride < 1 ||
      !std::isfinite(rope_theta) || rope_theta < 0.f || (q == nullptr) != (q_out == nullptr))
    return PE_ERR_INVALID_ARGUMENT;
  if (!row_ok(k, k_stride, kw, eb) || !row_ok(v, v_stride, kw, eb)) return PE_ERR_INVALID_ARGUMENT;
  if (q) {
    const int64_t qw = static_cast<int64_t>(n_heads) * dh;
    if (n_heads < 1 || n_heads % pool->n_kv_heads || !row_ok(q, q_stride, qw, eb) ||
        !row_ok(q_out, q_out_stride, qw, eb))
      return PE_ERR_INVALID_ARGUMENT;
  }
  AppendArgs a = {};
  a.pool = CachePool{pool->k, pool->v, pool->scores, pool->num_blocks};
  a.T = T;
  a.B = B;
  a.Hq = n_heads;
  a.Hkv = pool->n_kv_heads;
  a.bt_stride = bt_stride;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qo_stride = q_out_stride;
  a.pos = pos;
  a.req = req;
  a.block_table = block_table;
  a.q_out = q_out;
  a.err = err;
  a.k_scale = pool->k_scale;
  a.v_scale = pool->v_scale;
  a.rope = rope_steps(rope_theta, dh);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return PE_ERR_CUDA;
  if (pool->dtype == PE_KV_F32) e = launch_append<float, float>(a, dh, sms, s);
  else if (pool->dtype == PE_KV_BF16) e = launch_append<bf16, bf16>(a, dh, sms, s);
  else e = launch_append<bf16, uint8_t>(a, dh, sms, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
