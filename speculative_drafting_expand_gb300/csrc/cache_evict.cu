// cache_evict.cu -- trimming a paged KV cache to a budget by accumulated
// attention weight (include/peagle_cache.h).
//
// Keys are cached rotated to their positions, R(p) k.  Rotations compose,
// R(j - p) R(p) = R(j), so a key that moves from p to j is turned by j - p
// and is then the key of position j: the kept positions form an ordinary
// cache of positions 0 .. budget - 1.
//
// Bound by the bytes of the kept rows, read and written once; the scores are
// a few percent of them.  One launch: a cluster of CTAs for each (layer,
// request, kv head) finds the weight of the last position that stays, makes
// the ordered list, and moves the rows.  The choosing of one row's CTAs runs
// beside the moving of another's.
//
// The weight is found by bisection of its 32 bits, two bits a step: the
// scores lie in shared memory as integers of the same order, and each step
// counts those at or above three candidates.  Its time does not depend on the
// values (a histogram's does: equal scores, such as the zeros of positions
// that were never attended, meet in one counter), and it ends as soon as a
// count is right.  Every CTA of a cluster chooses for itself: the scores are
// read again from L2, and nothing is exchanged.
//
// In place, row j is written where an earlier-listed row may still lie, never
// a later one (kept[j] >= j, ascending): a round of rows is read by the whole
// cluster before the first of it is written.
#include <algorithm>
#include <atomic>

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


constexpr int kEvictThreads = 512;
constexpr int kMostKeys = 24576;  // scores that are held in shared memory

// A row on its way: where from (-1: nowhere) and to, by how much the key
// turns.
struct Move {
  long long src, dst;  // row numbers in the pool, -1: none
  int turn;            // old position - new position
};

template <typename S, int DH, bool IN_PLACE>
__global__ void __launch_bounds__(kEvictThreads, 2)
    kv_evict_kernel(const __grid_constant__ EvictArgs a, int cluster, int key_room) {
  constexpr int T = kEvictThreads, WARPS = T / 32;
  constexpr int ROWB = DH * static_cast<int>(sizeof(S));
  constexpr int LANES = ROWB / 16;       // lanes that hold a row, 16 bytes each
  constexpr int ROUND = 2 * T / LANES;   // rows a CTA moves at a time: two a group of lanes
  constexpr int HALF = LANES / 2;
  extern __shared__ uint32_t keys[];     // [key_room]
  __shared__ uint64_t step[DH / 2];
  __shared__ int count[3][4];            // three steps' counters
  __shared__ int scan[2][WARPS];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, row = blockIdx.x / cluster;
  const int h = row % a.Hkv, b = row / a.Hkv, layer = blockIdx.y;
  const CachePool pool = a.pool[layer];
  const int n = evict_len(a, b, tid == 0);
  const int m = min(n, a.budget);
  int32_t* kept =
      a.kept + ((static_cast<size_t>(layer) * a.B + b) * a.Hkv + h) * static_cast<size_t>(a.budget);
  if (layer == 0 && h == 0 && rank == 0 && tid == 0) a.new_lens[b] = m;
  if (tid < DH / 2) step[tid] = a.rope.step[tid];
  if (tid < 12) count[tid / 4][tid % 4] = 0;
  const int32_t* table = a.block_table + static_cast<size_t>(b) * a.bt_stride;
  auto owns = [&](int j) { return j / ROUND % cluster == rank; };
  int same = m;  // positions below stay where they are
  if (n <= a.budget) {
    for (int j = tid; j < a.budget; j += T)
      if (owns(j)) kept[j] = j < m ? j : -1;
  } else {
    // ---- the weight of the last position that stays
    const int lo = a.sinks, mid = n - a.recent - lo, need = a.budget - a.sinks - a.recent;
    auto load_key = [&](int i) -> uint32_t {
      const int p = lo + i;
      const int blk = table[p / kPage];
      if (blk < 0 || blk >= pool.num_blocks) {
        record_error(a.err, PE_DEV_BAD_BLOCK);
        return score_key(-INFINITY);
      }
      return score_key(pool.scores[(static_cast<size_t>(blk) * a.Hkv + h) * kPage + p % kPage]);
    };
    const int held = min(mid, key_room);
    if (need > 0)
#pragma unroll 4
      for (int i = tid; i < held; i += T) keys[i] = load_key(i);
    auto key = [&](int i) { return i < held ? keys[i] : load_key(i); };
    __syncthreads();
    uint32_t floor = 0;   // count(key >= floor) >= need
    bool exact = false;   // it is need
    if (need > 0) {
      for (int shift = 30, turn = 0; shift >= 0 && !exact; shift -= 2, turn = turn == 2 ? 0 : turn + 1) {
        const uint32_t t1 = floor + (1u << shift), t2 = floor + (2u << shift),
                       t3 = floor + (3u << shift);
        int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll 4
        for (int i = tid; i < held; i += T) {
          const uint32_t k = keys[i];
          c1 += k >= t1;
          c2 += k >= t2;
          c3 += k >= t3;
        }
        for (int i = held + tid; i < mid; i += T) {
          const uint32_t k = load_key(i);
          c1 += k >= t1;
          c2 += k >= t2;
          c3 += k >= t3;
        }
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        if (lane == 0) {
          atomicAdd(&count[turn][0], c1);
          atomicAdd(&count[turn][1], c2);
          atomicAdd(&count[turn][2], c3);
        }
        __syncthreads();
        c1 = count[turn][0];
        c2 = count[turn][1];
        c3 = count[turn][2];
        // the counters that the step after next adds to
        if (tid < 3) count[turn == 0 ? 2 : turn - 1][tid] = 0;
        const int c = c3 >= need ? c3 : c2 >= need ? c2 : c1 >= need ? c1 : -1;
        floor = c3 >= need ? t3 : c2 >= need ? t2 : c1 >= need ? t1 : floor;
        exact = c == need;
      }
    }
    // stay: key > T, and the first `ties` of key == T
    const uint32_t cut = exact ? floor - 1 : floor;
    // ---- the list, in order: each thread an odd number of positions in a row
    const int seg = ((mid + T - 1) / T) | 1;
    const int i0 = min(tid * seg, mid), i1 = min(i0 + seg, mid);
    int gt = 0, eq = 0;
    if (need > 0)
      for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        gt += k > cut;
        eq += k == cut;
      }
    int g = gt, q = eq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, g, o), y = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) {
        g += x;
        q += y;
      }
    }
    if (lane == 31) {
      scan[0][warp] = g;
      scan[1][warp] = q;
    }
    __syncthreads();
    int all_gt = 0;
    g -= gt;
    q -= eq;
    for (int w = 0; w < WARPS; ++w) {
      const int x = scan[0][w], y = scan[1][w];
      all_gt += x;
      g += w < warp ? x : 0;
      q += w < warp ? y : 0;
    }
    const int ties = need - all_gt;
    int at = lo + g + min(q, ties);
    if (need > 0)
      for (int i = i0; i < i1; ++i) {
        const uint32_t k = key(i);
        const bool tie = k == cut;
        if (k > cut || (tie && q < ties)) {
          if (owns(at)) kept[at] = lo + i;
          ++at;
        }
        q += tie;
      }
    for (int j = tid; j < lo; j += T)
      if (owns(j)) kept[j] = j;
    for (int j = m - a.recent + tid; j < m; j += T)
      if (owns(j)) kept[j] = n - m + j;
    if (IN_PLACE) same = lo;
  }
  // the list is this CTA's own for the rows that it moves
  __syncthreads();
  if (IN_PLACE) {
    // no CTA of the cluster reads scores to choose by any more
    if (cluster > 1) cluster_sync_all();
  }
  const int32_t* dtab =
      IN_PLACE ? table : a.dst_table + static_cast<size_t>(b) * a.dst_stride;
  const int dstride = IN_PLACE ? a.bt_stride : a.dst_stride;
  const int group = tid / LANES, c = tid % LANES;
  const bool high = c >= HALF;
  // rows round + 2 group and + 1; in place from the first that may move
  for (int round = (IN_PLACE ? same / ROUND / cluster * cluster + rank : rank) * ROUND;
       round - rank * ROUND < m; round += ROUND * cluster) {
    Move mv[2];
    uint4 kv[2], vv[2];
    float sc[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = round + 2 * group + x;
      mv[x].src = mv[x].dst = -1;
      mv[x].turn = 0;
      if (j < m) {
        const int p = __ldcg(kept + j);
        if (!(IN_PLACE && p == j)) {
          const int sb = table[p / kPage];
          const int db = j / kPage < dstride ? dtab[j / kPage] : -2;
          const bool s_ok = sb >= 0 && sb < pool.num_blocks, d_ok = db >= 0 && db < pool.num_blocks;
          if (c == 0 && !(s_ok && d_ok))
            record_error(a.err, db == -2 && j / kPage >= dstride ? PE_DEV_BAD_POSITION
                                                                 : PE_DEV_BAD_BLOCK);
          if (s_ok && d_ok) {
            mv[x].src = (static_cast<long long>(sb) * a.Hkv + h) * kPage + p % kPage;
            mv[x].dst = (static_cast<long long>(db) * a.Hkv + h) * kPage + j % kPage;
            mv[x].turn = p - j;
          }
        }
      }
      kv[x] = vv[x] = make_uint4(0, 0, 0, 0);
      sc[x] = 0.f;
      if (mv[x].src >= 0) {
        const size_t at = static_cast<size_t>(mv[x].src) * ROWB + c * 16;
        kv[x] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(pool.k) + at));
        vv[x] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const char*>(pool.v) + at));
        if (c == 0) sc[x] = pool.scores[mv[x].src];
      }
    }
    if (IN_PLACE) {
      if (cluster > 1) cluster_sync_all();
      else __syncthreads();
    }
    if (a.rope.on) {
      // lanes of the low half take the pairs of the first row, the others
      // the second's: a lane's other row's chunk is its partner's missing one
      const uint4 got = shfl_xor16(high ? kv[0] : kv[1], HALF);
      uint4 x1 = high ? got : kv[0], x2 = high ? kv[1] : got;
      const int turn = high ? mv[1].turn : mv[0].turn;
      if (turn != 0) {
        constexpr int N = Chunk<S>::N;
        float u[N], v[N];
        Chunk<S>::get(x1, u);
        Chunk<S>::get(x2, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float cs, sn;
          rope_turn<sizeof(S) != 4>(step[(c % HALF) * N + e], -static_cast<long long>(turn), cs, sn);
          const float y = u[e] * cs - v[e] * sn;
          v[e] = v[e] * cs + u[e] * sn;
          u[e] = y;
        }
        x1 = Chunk<S>::put(u);
        x2 = Chunk<S>::put(v);
      }
      const uint4 back = shfl_xor16(high ? x1 : x2, HALF);
      kv[0] = high ? back : x1;
      kv[1] = high ? x2 : back;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
      if (mv[x].dst >= 0) {
        const size_t at = static_cast<size_t>(mv[x].dst) * ROWB + c * 16;
        *reinterpret_cast<uint4*>(static_cast<char*>(pool.k) + at) = kv[x];
        *reinterpret_cast<uint4*>(static_cast<char*>(pool.v) + at) = vv[x];
        if (c == 0) pool.scores[mv[x].dst] = sc[x];
      }
  }
  // positions that hold nothing any more
  if (rank != 0) return;
  const int page_end = (m + kPage - 1) / kPage * kPage;
  const int end = IN_PLACE ? max(n, page_end) : page_end;
  for (int j = m + tid; j < end; j += T) {
    const int db = page_of(dtab - static_cast<size_t>(b) * dstride, dstride, b, j, pool.num_blocks,
                           a.err);
    if (db >= 0) pool.scores[(static_cast<size_t>(db) * a.Hkv + h) * kPage + j % kPage] = 0.f;
  }
}

template <typename S, int DH, bool IN_PLACE>
static cudaError_t launch_evict_one(const EvictArgs& a, int n_layers, int dev, int sms,
                                    cudaStream_t s) {
  // Clusters while the rows alone leave SMs idle (two CTAs an SM).
  const long long rows = static_cast<long long>(a.B) * a.Hkv * n_layers;
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= 2LL * sms) cluster *= 2;
  const long long room = std::min<long long>(static_cast<long long>(a.bt_stride) * kPage, kMostKeys);
  static std::atomic<uint64_t> done{0};
  if (dev >= 64 || !((done.load(std::memory_order_relaxed) >> dev) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel<S, DH, IN_PLACE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMostKeys * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev);
  }
  return launch_pdl_cluster(kv_evict_kernel<S, DH, IN_PLACE>,
                            dim3(static_cast<unsigned>(a.B) * a.Hkv * cluster, n_layers),
                            dim3(kEvictThreads), static_cast<size_t>(room) * 4, s, cluster, a,
                            cluster, static_cast<int>(room));
}

template <typename S>
static cudaError_t launch_evict(const EvictArgs& a, int n_layers, int dh, int dev, int sms,
                                cudaStream_t s) {
  if (dh == 64)
    return a.dst_table ? launch_evict_one<S, 64, false>(a, n_layers, dev, sms, s)
                       : launch_evict_one<S, 64, true>(a, n_layers, dev, sms, s);
  return a.dst_table ? launch_evict_one<S, 128, false>(a, n_layers, dev, sms, s)
                     : launch_evict_one<S, 128, true>(a, n_layers, dev, sms, s);
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
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return PE_ERR_CUDA;
  if (pools[0].dtype == PE_KV_F32) e = launch_evict<float>(a, n_layers, dh, dev, sms, s);
  else if (pools[0].dtype == PE_KV_BF16) e = launch_evict<bf16>(a, n_layers, dh, dev, sms, s);
  else e = launch_evict<uint8_t>(a, n_layers, dh, dev, sms, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
