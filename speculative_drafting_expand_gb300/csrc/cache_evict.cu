// cache_evict.cu -- trimming a paged KV cache to a budget by accumulated
// attention weight (include/peagle_cache.h).
//
// Keys are cached rotated to their positions, R(p) k.  Rotations compose,
// R(j - p) R(p) = R(j), so a key that moves from p to j is turned by j - p
// and is then the key of position j: the kept positions form an ordinary
// cache of positions 0 .. budget - 1.
#include <algorithm>

#include "cache_common.cuh"
#include "pe_kernels.h"

namespace pe {

constexpr int kMaxLayers = 64;

struct EvictArgs {
  int B, Hkv, bt_stride, dst_stride, budget, sinks, recent;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* dst_table;  // NULL: in place
  int32_t* kept;
  int32_t* new_lens;
  int* err;
  RopeSteps rope;
  CachePool pool[kMaxLayers];
};

// The order in which scores are compared: larger float, larger key; -0 is
// +0 and a NaN is -inf.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  return float_order_key(x + 0.f);
}

__device__ __forceinline__ int evict_len(const EvictArgs& a, int b, bool record) {
  const long long cap = static_cast<long long>(a.bt_stride) * kPage;
  int n = a.seq_lens[b];
  if (n < 0 || n > cap) {
    if (record) record_error(a.err, PE_DEV_BAD_POSITION);
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}

// Page of position p in a table row, -1 (recorded) when it is no page.
__device__ __forceinline__ int page_of(const int32_t* table, int stride, int b, int p, int blocks,
                                       int* err) {
  if (p / kPage >= stride) {
    record_error(err, PE_DEV_BAD_POSITION);
    return -1;
  }
  const int blk = table[static_cast<size_t>(b) * stride + p / kPage];
  if (blk >= 0 && blk < blocks) return blk;
  record_error(err, PE_DEV_BAD_BLOCK);
  return -1;
}

__device__ __forceinline__ int block_count(bool x, int* red) {
  const int c = __popc(__ballot_sync(0xffffffffu, x));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = c;
  __syncthreads();
  int t = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) t += red[i];
  return t;
}

// A CTA per (layer, request, kv head): the threshold by bisection of the 32
// key bits, the list by counting, then the rows in order.
template <typename S, int DH>
__global__ void __launch_bounds__(256) kv_evict_kernel(const __grid_constant__ EvictArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int red[8], warp_base[8];
  const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv, layer = blockIdx.y;
  const CachePool pool = a.pool[layer];
  const int tid = threadIdx.x;
  const int n = evict_len(a, b, tid == 0);
  const int m = min(n, a.budget);
  int32_t* kept =
      a.kept + ((static_cast<size_t>(layer) * a.B + b) * a.Hkv + h) * static_cast<size_t>(a.budget);
  if (layer == 0 && h == 0 && tid == 0) a.new_lens[b] = m;
  const int lo = a.sinks, hi = n - a.recent, need = a.budget - a.sinks - a.recent;
  const bool all = n <= a.budget;
  auto key_of = [&](int p) -> uint32_t {
    const int blk = page_of(a.block_table, a.bt_stride, b, p, pool.num_blocks, a.err);
    if (blk < 0) return score_key(-INFINITY);
    return score_key(pool.scores[(static_cast<size_t>(blk) * a.Hkv + h) * kPage + p % kPage]);
  };
  // largest T with count(key >= T) >= need
  uint32_t T = 0;
  int above = 0;  // count(key > T)
  if (!all && need > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = T | (1u << bit);
      int c = 0;
      for (int p = lo + tid; p - tid < hi; p += 256) c += block_count(p < hi && key_of(p) >= t, red);
      if (c >= need) T = t;
    }
    for (int p = lo + tid; p - tid < hi; p += 256)
      above += block_count(p < hi && key_of(p) > T, red);
  }
  int ties = need - above;  // of the positions at T, the first so many
  int base = 0, seen = 0;
  for (int p0 = 0; p0 < n; p0 += 256) {
    const int p = p0 + tid;
    bool keep = p < n, tie = false;
    if (!all && p >= lo && p < hi) {
      const uint32_t key = need > 0 ? key_of(p) : 0u;
      tie = need > 0 && key == T;
      keep = need > 0 && key > T;
    }
    // ties before this position
    const uint32_t tb = __ballot_sync(0xffffffffu, tie);
    __syncthreads();
    if ((tid & 31) == 0) warp_base[tid >> 5] = __popc(tb);
    __syncthreads();
    int before = seen + __popc(tb & ((1u << (tid & 31)) - 1)), round = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < (tid >> 5)) before += warp_base[w];
      round += warp_base[w];
    }
    seen += round;
    if (tie && before < ties) keep = true;
    const uint32_t kb = __ballot_sync(0xffffffffu, keep);
    __syncthreads();
    if ((tid & 31) == 0) warp_base[tid >> 5] = __popc(kb);
    __syncthreads();
    int at = base + __popc(kb & ((1u << (tid & 31)) - 1));
    round = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < (tid >> 5)) at += warp_base[w];
      round += warp_base[w];
    }
    if (keep && at < m) kept[at] = p;
    base += round;
  }
  for (int j = m + tid; j < a.budget; j += 256) kept[j] = -1;
  __syncthreads();
  // the rows, a warp each, eight at a time: kept[j] >= j and the list
  // ascends, so in place a round's stores never touch a later round's rows
  const bool in_place = a.dst_table == nullptr;
  const int32_t* dtab = in_place ? a.block_table : a.dst_table;
  const int dstride = in_place ? a.bt_stride : a.dst_stride;
  constexpr int HALF = DH / 2, E = HALF / 32;
  const int lane = tid & 31, w = tid >> 5;
  for (int j0 = 0; j0 < m; j0 += 8) {
    const int j = j0 + w;
    S klo[E], khi[E], vlo[E], vhi[E];
    float sc = 0.f;
    int sb = -1, db = -1, p = 0;
    if (j < m) {
      p = __ldcg(kept + j);
      sb = page_of(a.block_table, a.bt_stride, b, p, pool.num_blocks, a.err);
      db = page_of(dtab, dstride, b, j, pool.num_blocks, a.err);
    }
    if (sb >= 0) {
      const size_t r = (static_cast<size_t>(sb) * a.Hkv + h) * kPage + p % kPage;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = lane + 32 * e;
        klo[e] = static_cast<const S*>(pool.k)[r * DH + i];
        khi[e] = static_cast<const S*>(pool.k)[r * DH + HALF + i];
        vlo[e] = static_cast<const S*>(pool.v)[r * DH + i];
        vhi[e] = static_cast<const S*>(pool.v)[r * DH + HALF + i];
      }
      sc = pool.scores[r];
    }
    __syncthreads();
    if (sb >= 0 && db >= 0) {
      const size_t r = (static_cast<size_t>(db) * a.Hkv + h) * kPage + j % kPage;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = lane + 32 * e;
        if (a.rope.on && p != j) {
          float c, s;
          rope_cos_sin(a.rope.step[i], static_cast<long long>(j) - p, c, s);
          float x1, x2;
          if constexpr (sizeof(S) == 1) {
            const uint32_t u = e4m3x2_to_f16x2(klo[e] | (static_cast<uint32_t>(khi[e]) << 8));
            x1 = __half2float(__ushort_as_half(static_cast<unsigned short>(u & 0xffff)));
            x2 = __half2float(__ushort_as_half(static_cast<unsigned short>(u >> 16)));
          } else {
            x1 = to_f(klo[e]);
            x2 = to_f(khi[e]);
          }
          const float y1 = x1 * c - x2 * s, y2 = x2 * c + x1 * s;
          if constexpr (sizeof(S) == 1) {
            const uint16_t y = f32x2_to_e4m3x2(y1, y2);
            klo[e] = static_cast<uint8_t>(y & 0xff);
            khi[e] = static_cast<uint8_t>(y >> 8);
          } else {
            klo[e] = from_f<S>(y1);
            khi[e] = from_f<S>(y2);
          }
        }
        static_cast<S*>(pool.k)[r * DH + i] = klo[e];
        static_cast<S*>(pool.k)[r * DH + HALF + i] = khi[e];
        static_cast<S*>(pool.v)[r * DH + i] = vlo[e];
        static_cast<S*>(pool.v)[r * DH + HALF + i] = vhi[e];
      }
      if (lane == 0) pool.scores[r] = sc;
    }
  }
  __syncthreads();
  const int page_end = (m + kPage - 1) / kPage * kPage;
  const int end = in_place ? max(n, page_end) : page_end;
  for (int j = m + tid; j < end; j += 256) {
    const int db = page_of(dtab, dstride, b, j, pool.num_blocks, a.err);
    if (db >= 0) pool.scores[(static_cast<size_t>(db) * a.Hkv + h) * kPage + j % kPage] = 0.f;
  }
}

template <typename S>
static cudaError_t launch_evict(const EvictArgs& a, int n_layers, int dh, cudaStream_t s) {
  const dim3 grid(a.B * a.Hkv, n_layers);
  if (dh == 64) return launch_pdl(kv_evict_kernel<S, 64>, grid, dim3(256), 0, s, a);
  return launch_pdl(kv_evict_kernel<S, 128>, grid, dim3(256), 0, s, a);
}

}  // namespace pe

extern "C" pe_status pe_kv_evict(int32_t n_layers, const pe_kv_pool* pools, int32_t B,
                                 const int32_t* block_table, int32_t bt_stride,
                                 const int32_t* seq_lens, int32_t budget, int32_t sinks,
                                 int32_t recent, float rope_theta, const int32_t* dst_table,
                                 int32_t dst_stride, int32_t* kept, int32_t* new_lens,
                                 int32_t* err, void* stream) {
  using namespace pe;
  if (n_layers < 1 || n_layers > kMaxLayers || !pools) return PE_ERR_INVALID_ARGUMENT;
  for (int l = 0; l < n_layers; ++l) {
    if (const pe_status st = check_pool(pools + l); st != PE_OK) return st;
    if (!pools[l].scores || pools[l].n_kv_heads != pools[0].n_kv_heads ||
        pools[l].head_dim != pools[0].head_dim || pools[l].dtype != pools[0].dtype)
      return PE_ERR_INVALID_ARGUMENT;
  }
  if (B < 1 || !block_table || bt_stride < 1 || !seq_lens || budget < 1 || sinks < 0 ||
      recent < 0 || static_cast<int64_t>(sinks) + recent > budget || !std::isfinite(rope_theta) ||
      rope_theta < 0.f || (dst_table && dst_stride < 1) || !kept || !new_lens ||
      new_lens == seq_lens)
    return PE_ERR_INVALID_ARGUMENT;
  const int64_t rows = static_cast<int64_t>(B) * pools[0].n_kv_heads;
  if (rows * n_layers > 2147483647LL / budget) return PE_ERR_UNSUPPORTED;
  EvictArgs a = {};
  a.B = B;
  a.Hkv = pools[0].n_kv_heads;
  a.bt_stride = bt_stride;
  a.dst_stride = dst_stride;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.dst_table = dst_table;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = err;
  a.rope = rope_steps(rope_theta, pools[0].head_dim);
  for (int l = 0; l < n_layers; ++l)
    a.pool[l] = CachePool{pools[l].k, pools[l].v, pools[l].scores, pools[l].num_blocks};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int dh = pools[0].head_dim;
  cudaError_t e;
  if (pools[0].dtype == PE_KV_F32) e = launch_evict<float>(a, n_layers, dh, s);
  else if (pools[0].dtype == PE_KV_BF16) e = launch_evict<bf16>(a, n_layers, dh, s);
  else e = launch_evict<uint8_t>(a, n_layers, dh, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
