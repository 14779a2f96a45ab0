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

// A CTA a row.  The lanes of a group take 16 bytes each of two heads (q heads,
// then k heads); to turn a pair (i, i + DH / 2) a lane needs the chunk that
// its partner half a head further holds, so the low half of the lanes turns
// the first head and the other half the second, with one exchange before and
// one after.  More threads copy v.  Bound by bytes for many rows and by
// latency for few: every load is on its way before the first use, and the
// row's sines and cosines (one pair a thread, shared by all heads) are worked
// out meanwhile.
constexpr int kAppendMost = 512;

template <typename A, typename S, int DH>
__global__ void __launch_bounds__(kAppendMost) kv_append_kernel(
    const __grid_constant__ AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  using C = Chunk<A>;
  constexpr int N = C::N;         // elements of a chunk
  constexpr int LANES = DH / N;   // lanes of a head
  constexpr int HALF = LANES / 2;
  __shared__ float cs[DH / 2], sn[DH / 2];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int hq = a.q ? a.Hq : 0, heads = hq + a.Hkv;
  const int turned = (heads + 1) / 2 * LANES, all = turned + a.Hkv * LANES;
  const int threads = blockDim.x;
  const A* q = static_cast<const A*>(a.q) + static_cast<size_t>(t) * a.q_stride;
  const A* k = static_cast<const A*>(a.k) + static_cast<size_t>(t) * a.k_stride;
  const A* v = static_cast<const A*>(a.v) + static_cast<size_t>(t) * a.v_stride;
  const int c = tid % LANES;
  const bool high = c >= HALF;
  // this thread's chunks of item w: two heads', or one of v
  auto load = [&](int w, uint4 (&x)[2]) {
    x[0] = x[1] = make_uint4(0, 0, 0, 0);
    if (w < turned) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int h = w / LANES * 2 + y;
        if (h < heads)
          x[y] = *reinterpret_cast<const uint4*>((h < hq ? q + h * DH : k + (h - hq) * DH) + c * N);
      }
    } else if (w < all) {
      x[0] = *reinterpret_cast<const uint4*>(v + static_cast<size_t>(w - turned) * N);
    }
  };
  uint4 x[2];
  load(tid, x);
  const int p = a.pos[t];
  if (p < 0) return;  // padding
  const int r = a.req ? a.req[t] : t;
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
  for (int i = tid; a.rope.on && i < DH / 2; i += threads) {
    float cc, ss;
    rope_cos_sin(a.rope.step[i], p, cc, ss);
    cs[i] = cc;
    sn[i] = ss;
  }
  __syncthreads();
  const int off = p % kPage;
  // element (head, 0) of the row's slot
  auto slot = [&](int h) {
    return ((static_cast<size_t>(blk) * a.Hkv + h) * kPage + off) * DH;
  };
  for (int w0 = tid / 32 * 32; w0 < all; w0 += threads) {  // whole warps: they exchange
    const int w = w0 + tid % 32;
    if (w0 >= threads) load(w, x);
    if (a.rope.on && w0 < turned) {
      const uint4 got = shfl_xor16(high ? x[0] : x[1], HALF);
      uint4 lo = high ? got : x[0], hi = high ? x[1] : got;
      float u[N], y[N];
      C::get(lo, u);
      C::get(hi, y);
      if (w < turned) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int i = c % HALF * N + e;
          const float z = u[e] * cs[i] - y[e] * sn[i];
          y[e] = y[e] * cs[i] + u[e] * sn[i];
          u[e] = z;
        }
        // q leaves rounded to its type, k as it is rounded by its pool: the
        // exchange is done on what is stored
        const int h = w / LANES * 2 + (high ? 1 : 0);
        if (h >= hq && h < heads && blk >= 0) {
          store_kv<S>(a.pool.k, slot(h - hq) + c % HALF * N, u, a.k_scale);
          store_kv<S>(a.pool.k, slot(h - hq) + c % HALF * N + DH / 2, y, a.k_scale);
        }
      }
      lo = C::put(u);
      hi = C::put(y);
      const uint4 back = shfl_xor16(high ? lo : hi, HALF);
      if (w < turned) {
        x[0] = high ? back : lo;
        x[1] = high ? hi : back;
      }
    }
    if (w < turned) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int h = w / LANES * 2 + y;
        if (h < hq) {
          *reinterpret_cast<uint4*>(static_cast<A*>(a.q_out) +
                                    static_cast<size_t>(t) * a.qo_stride + h * DH + c * N) = x[y];
        } else if (h < heads && blk >= 0 && !a.rope.on) {
          float z[N];
          C::get(x[y], z);
          store_kv<S>(a.pool.k, slot(h - hq) + c * N, z, a.k_scale);
        }
      }
    } else if (w < all && blk >= 0) {
      float z[N];
      C::get(x[0], z);
      const int e = (w - turned) * N;
      store_kv<S>(a.pool.v, slot(e / DH) + e % DH, z, a.v_scale);
    }
  }
  if (a.pool.scores && blk >= 0)
    for (int h = tid; h < a.Hkv; h += threads)
      a.pool.scores[(static_cast<size_t>(blk) * a.Hkv + h) * kPage + off] = 0.f;
}

template <typename A, typename S, int DH>
static cudaError_t launch_append_dim(const AppendArgs& a, cudaStream_t s) {
  constexpr int LANES = DH / Chunk<A>::N;
  const long long items =
      ((static_cast<long long>(a.q ? a.Hq : 0) + a.Hkv + 1) / 2 + a.Hkv) * LANES;
  const int threads = static_cast<int>(std::min<long long>(kAppendMost, (items + 31) / 32 * 32));
  return launch_pdl(kv_append_kernel<A, S, DH>, dim3(a.T), dim3(threads), 0, s, a);
}
template <typename A, typename S>
static cudaError_t launch_append(const AppendArgs& a, int dh, cudaStream_t s) {
  return dh == 64 ? launch_append_dim<A, S, 64>(a, s) : launch_append_dim<A, S, 128>(a, s);
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
  cudaError_t e;
  if (pool->dtype == PE_KV_F32) e = launch_append<float, float>(a, dh, s);
  else if (pool->dtype == PE_KV_BF16) e = launch_append<bf16, bf16>(a, dh, s);
  else e = launch_append<bf16, uint8_t>(a, dh, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
