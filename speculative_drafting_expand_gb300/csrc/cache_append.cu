// cache_append.cu -- new rows of q, k and v into a paged KV cache: rotate-half
// rotary embedding of q and k at the row's position, k and v stored in the
// position's page slot (include/peagle_cache.h).
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

template <typename T>
__device__ __forceinline__ void store_kv(void* base, size_t at, float x, float scale);
template <>
__device__ __forceinline__ void store_kv<float>(void* base, size_t at, float x, float) {
  static_cast<float*>(base)[at] = x;
}
template <>
__device__ __forceinline__ void store_kv<bf16>(void* base, size_t at, float x, float) {
  static_cast<bf16*>(base)[at] = __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ void store_kv<uint8_t>(void* base, size_t at, float x, float scale) {
  const uint16_t c = f32x2_to_e4m3x2(__fdiv_rn(x, scale), 0.f);
  static_cast<uint8_t*>(base)[at] = static_cast<uint8_t>(c & 0xff);
}

// One CTA a row, a thread per (head, pair).
template <typename A, typename S, int DH>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int HALF = DH / 2;
  __shared__ float cs[HALF], sn[HALF];
  const int t = blockIdx.x;
  const int p = a.pos[t];
  if (p < 0) return;  // padding
  const int r = a.req ? a.req[t] : t;
  int blk = -1;
  if (r < 0 || r >= a.B) {
    if (threadIdx.x == 0) record_error(a.err, PE_DEV_BAD_ROW);
  } else if (p >= static_cast<long long>(a.bt_stride) * kPage) {
    if (threadIdx.x == 0) record_error(a.err, PE_DEV_BAD_POSITION);
  } else {
    blk = a.block_table[static_cast<size_t>(r) * a.bt_stride + p / kPage];
    if (blk < 0 || blk >= a.pool.num_blocks) {
      if (threadIdx.x == 0) record_error(a.err, PE_DEV_BAD_BLOCK);
      blk = -1;
    }
  }
  const int off = p % kPage;
  if (threadIdx.x < HALF) {
    float c = 1.f, s = 0.f;
    if (a.rope.on) rope_cos_sin(a.rope.step[threadIdx.x], p, c, s);
    cs[threadIdx.x] = c;
    sn[threadIdx.x] = s;
  }
  __syncthreads();
  const A* q = static_cast<const A*>(a.q) + static_cast<size_t>(t) * a.q_stride;
  const A* k = static_cast<const A*>(a.k) + static_cast<size_t>(t) * a.k_stride;
  const A* v = static_cast<const A*>(a.v) + static_cast<size_t>(t) * a.v_stride;
  A* qo = static_cast<A*>(a.q_out) + static_cast<size_t>(t) * a.qo_stride;
  const int hq = a.q ? a.Hq : 0;
  for (int w = threadIdx.x; w < (hq + a.Hkv) * HALF; w += blockDim.x) {
    const int h = w / HALF, i = w % HALF;
    const A* x = h < hq ? q + h * DH : k + (h - hq) * DH;
    const float x1 = to_f(x[i]), x2 = to_f(x[i + HALF]);
    const float y1 = x1 * cs[i] - x2 * sn[i];
    const float y2 = x2 * cs[i] + x1 * sn[i];
    if (h < hq) {
      qo[h * DH + i] = from_f<A>(y1);
      qo[h * DH + i + HALF] = from_f<A>(y2);
    } else if (blk >= 0) {
      const size_t at = ((static_cast<size_t>(blk) * a.Hkv + (h - hq)) * kPage + off) * DH;
      store_kv<S>(a.pool.k, at + i, y1, a.k_scale);
      store_kv<S>(a.pool.k, at + i + HALF, y2, a.k_scale);
    }
  }
  if (blk < 0) return;
  for (int w = threadIdx.x; w < a.Hkv * DH; w += blockDim.x) {
    const size_t at =
        ((static_cast<size_t>(blk) * a.Hkv + w / DH) * kPage + off) * DH + w % DH;
    store_kv<S>(a.pool.v, at, to_f(v[w]), a.v_scale);
  }
  if (a.pool.scores)
    for (int h = threadIdx.x; h < a.Hkv; h += blockDim.x)
      a.pool.scores[(static_cast<size_t>(blk) * a.Hkv + h) * kPage + off] = 0.f;
}

template <typename A, typename S>
static cudaError_t launch_append(const AppendArgs& a, int dh, cudaStream_t s) {
  if (dh == 64)
    return launch_pdl(kv_append_kernel<A, S, 64>, dim3(a.T), dim3(256), 0, s, a);
  return launch_pdl(kv_append_kernel<A, S, 128>, dim3(a.T), dim3(256), 0, s, a);
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
