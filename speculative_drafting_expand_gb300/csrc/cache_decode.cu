// cache_decode.cu -- attention of one new token per request over a paged KV
// cache (include/peagle_cache.h):
//   out = sum_j p_j v_j,  p_j = exp(z_j - lse),  z_j = scale q.k_j,
//   lse = ln sum_j exp(z_j),
// with one pass over K and V (running maximum m and sum l; a new maximum
// scales what was summed by exp(m_old - m_new)) and, where asked, each
// position's weight summed over the query heads of its kv head.
#include <algorithm>

#include "cache_common.cuh"
#include "pe_kernels.h"

namespace pe {

struct DecodeArgs {
  CachePool pool;
  int B, Hq, Hkv, bt_stride, window;
  float scale;
  const void* q;
  long long q_stride, out_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;    // caller's, or NULL
  float* lse_w;  // workspace [B, Hq]
  int* err;
  float k_scale, v_scale;
};

template <typename S>
__device__ __forceinline__ float load_kv(const void* base, size_t at);
template <>
__device__ __forceinline__ float load_kv<float>(const void* base, size_t at) {
  return static_cast<const float*>(base)[at];
}
template <>
__device__ __forceinline__ float load_kv<bf16>(const void* base, size_t at) {
  return __bfloat162float(static_cast<const bf16*>(base)[at]);
}
template <>
__device__ __forceinline__ float load_kv<uint8_t>(const void* base, size_t at) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[at]);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffff)));
}

__device__ __forceinline__ int request_len(const DecodeArgs& a, int b, bool record) {
  const long long cap = static_cast<long long>(a.bt_stride) * kPage;
  int n = a.seq_lens[b];
  if (n < 0 || n > cap) {
    if (record) record_error(a.err, PE_DEV_BAD_POSITION);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}

// A CTA per (request, query head): its warps take every fourth position, a
// warp's lanes the elements of a row; joined through shared memory.
template <typename A, typename S, int DH>
__global__ void __launch_bounds__(128) attn_decode_kernel(const DecodeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int E = DH / 32;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][DH];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int hk = h / (a.Hq / a.Hkv);
  const int n = request_len(a, b, threadIdx.x == 0);
  const int lo = a.window > 0 ? max(0, n - a.window) : 0;
  const A* q = static_cast<const A*>(a.q) + static_cast<size_t>(b) * a.q_stride + h * DH;
  float qv[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_f(q[lane + 32 * e]) * (a.scale * a.k_scale);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo + w; j < n; j += 4) {
    const int blk = a.block_table[static_cast<size_t>(b) * a.bt_stride + j / kPage];
    if (blk < 0 || blk >= a.pool.num_blocks) {
      if (lane == 0) record_error(a.err, PE_DEV_BAD_BLOCK);
      continue;
    }
    const size_t at = ((static_cast<size_t>(blk) * a.Hkv + hk) * kPage + j % kPage) * DH;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += qv[e] * load_kv<S>(a.pool.k, at + lane + 32 * e);
#pragma unroll
    for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float c = __expf(m - base), p = __expf(z - base);
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * c + p * load_kv<S>(a.pool.v, at + lane + 32 * e);
    m = mn;
  }
  if (lane == 0) {
    sm_m[w] = m;
    sm_l[w] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[w][lane + 32 * e] = o[e];
  __syncthreads();
  const float mt = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
  const float base = mt == -INFINITY ? 0.f : mt;
  float lt = 0.f, c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = __expf(sm_m[i] - base);
    lt += c[i] * sm_l[i];
  }
  const float inv = lt == 0.f ? 0.f : a.v_scale / lt;
  A* out = static_cast<A*>(a.out) + static_cast<size_t>(b) * a.out_stride + h * DH;
  for (int d = threadIdx.x; d < DH; d += 128) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) x += c[i] * sm_o[i][d];
    out[d] = from_f<A>(x * inv);
  }
  if (threadIdx.x == 0) {
    const float s = lt == 0.f ? -INFINITY : mt + logf(lt);
    a.lse_w[b * a.Hq + h] = s;
    if (a.lse) a.lse[b * a.Hq + h] = s;
  }
}

// Weights of a page's positions, a warp per (request, kv head, page slice).
template <typename A, typename S, int DH>
__global__ void __launch_bounds__(128) attn_scores_kernel(const DecodeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int E = DH / 32;
  const int b = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv, G = a.Hq / a.Hkv;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = request_len(a, b, false);
  const int lo = a.window > 0 ? max(0, n - a.window) : 0;
  for (int j = lo + w + 4 * blockIdx.y; j < n; j += 4 * gridDim.y) {
    const int blk = a.block_table[static_cast<size_t>(b) * a.bt_stride + j / kPage];
    if (blk < 0 || blk >= a.pool.num_blocks) continue;
    const size_t row = (static_cast<size_t>(blk) * a.Hkv + hk) * kPage + j % kPage;
    float kv[E], sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) kv[e] = load_kv<S>(a.pool.k, row * DH + lane + 32 * e);
    for (int g = 0; g < G; ++g) {
      const A* q = static_cast<const A*>(a.q) + static_cast<size_t>(b) * a.q_stride +
                   (hk * G + g) * DH;
      float z = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) z += to_f(q[lane + 32 * e]) * (a.scale * a.k_scale) * kv[e];
#pragma unroll
      for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      const float lse = a.lse_w[b * a.Hq + hk * G + g];
      if (lse != -INFINITY) sum += __expf(z - lse);
    }
    if (lane == 0) atomicAdd(a.pool.scores + row, sum);
  }
}

template <typename A, typename S, int DH>
static cudaError_t launch_decode(const DecodeArgs& a, bool accumulate, cudaStream_t s) {
  cudaError_t e = launch_pdl(attn_decode_kernel<A, S, DH>, dim3(a.B * a.Hq), dim3(128), 0, s, a);
  if (e == cudaSuccess && accumulate)
    e = launch_pdl(attn_scores_kernel<A, S, DH>, dim3(a.B * a.Hkv, 16), dim3(128), 0, s, a);
  return e;
}

}  // namespace pe

extern "C" {

int64_t pe_attn_decode_workspace(int32_t B, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim) {
  if (B < 1 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return (static_cast<int64_t>(B) * n_heads * 4 + 15) / 16 * 16;
}

pe_status pe_attn_decode(const pe_kv_pool* pool, int32_t B, int32_t n_heads, float scale,
                         const void* q, int64_t q_stride, const int32_t* block_table,
                         int32_t bt_stride, const int32_t* seq_lens, int32_t window, void* out,
                         int64_t out_stride, float* lse, int32_t accumulate, void* workspace,
                         int64_t workspace_bytes, int32_t* err, void* stream) {
  using namespace pe;
  if (const pe_status st = check_pool(pool); st != PE_OK) return st;
  const int dh = pool->head_dim, eb = act_elem_bytes(pool->dtype);
  const int64_t qw = static_cast<int64_t>(n_heads) * dh;
  if (B < 1 || n_heads < 1 || n_heads % pool->n_kv_heads || !std::isfinite(scale) ||
      !block_table || bt_stride < 1 || !seq_lens || window < 0 || !row_ok(q, q_stride, qw, eb) ||
      !row_ok(out, out_stride, qw, eb) || (accumulate && !pool->scores) || !workspace ||
      !is_aligned16(workspace) ||
      workspace_bytes < pe_attn_decode_workspace(B, n_heads, pool->n_kv_heads, dh))
    return PE_ERR_INVALID_ARGUMENT;
  DecodeArgs a = {};
  a.pool = CachePool{pool->k, pool->v, pool->scores, pool->num_blocks};
  a.B = B;
  a.Hq = n_heads;
  a.Hkv = pool->n_kv_heads;
  a.bt_stride = bt_stride;
  a.window = window;
  a.scale = scale;
  a.q = q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.lse_w = static_cast<float*>(workspace);
  a.err = err;
  const bool codes = pool->dtype == PE_KV_E4M3;
  a.k_scale = codes ? pool->k_scale : 1.f;
  a.v_scale = codes ? pool->v_scale : 1.f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool acc = accumulate != 0;
  cudaError_t e;
  if (pool->dtype == PE_KV_F32)
    e = dh == 64 ? launch_decode<float, float, 64>(a, acc, s)
                 : launch_decode<float, float, 128>(a, acc, s);
  else if (pool->dtype == PE_KV_BF16)
    e = dh == 64 ? launch_decode<bf16, bf16, 64>(a, acc, s)
                 : launch_decode<bf16, bf16, 128>(a, acc, s);
  else
    e = dh == 64 ? launch_decode<bf16, uint8_t, 64>(a, acc, s)
                 : launch_decode<bf16, uint8_t, 128>(a, acc, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

}  // extern "C"
