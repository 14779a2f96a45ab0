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
// counts those at or above three candidates.  No step's time depends on the
// values (a histogram's does: equal scores, such as the zeros of positions
// that were never attended, meet in one counter).  It ends as soon as a count
// is right, or when so few scores are left between two candidates that each
// of them can be ranked among the others.  Every CTA of a cluster chooses for itself: the scores are
// read again from L2, and nothing is exchanged.
//
// Measured (GB300, four layers): 64 requests of 295104 positions in all to 2048
// each, 8 kv heads of 64, bf16: 398 us, 5.2 TB/s of rows of 128 bytes from
// scattered places; 16 requests to 1501, 4 heads of 128, e4m3: 77 us, of which
// the choosing, at the same time in all CTAs, takes about 20; one request 4096
// to 1024: 14 us.
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


// Two CTAs of 512 threads an SM (batch 64, before the rows ran ahead: 476 us;
// four of 256: 526, one of 512: 688, one of 1024: 524).
constexpr int kEvictThreads = 512;
// Scores that are held in shared memory, with two CTAs an SM and with one
// (few rows); the rest of a longer row is read again from L2 at every step.
constexpr int kMostKeys = 24576;
constexpr int kMostKeysAlone = 49152;
constexpr int kRanked = 128;  // keys that are ranked at once (0: 15.9 us, 64 and 128: 14.3,
                              // 256: 16.4 for one request)

// A row on its way: its number in the pool where it goes (-1: nowhere) and by
// how much its key turns.
struct Move {
  long long dst;
  int turn;  // old position - new position
  int pad;
};

template <typename S, int DH>
struct EvictShape {
  static constexpr int T = kEvictThreads;
  static constexpr int ROWB = DH * static_cast<int>(sizeof(S));
  static constexpr int LANES = ROWB / 16;      // lanes that hold a row, 16 bytes each
  static constexpr int ROUND = 2 * T / LANES;  // rows a CTA moves at a time: two a group of lanes
  static constexpr int AHEAD = 3;              // rounds on their way
  // a thread's chunks of a round: K and V of two rows
  static constexpr int RING = AHEAD * 4 * T * 16;
  static constexpr int SMEM = RING + AHEAD * ROUND * static_cast<int>(sizeof(Move) + 4);
  static_assert(RING == kMostKeys * 4, "the scores and the rows share the space");
};

__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <typename S, int DH, bool IN_PLACE>
__global__ void __launch_bounds__(kEvictThreads, 2)
    kv_evict_kernel(const __grid_constant__ EvictArgs a, int cluster, int key_room) {
  using SH = EvictShape<S, DH>;
  constexpr int T = SH::T, WARPS = T / 32, LANES = SH::LANES, ROUND = SH::ROUND;
  constexpr int HALF = LANES / 2, AHEAD = SH::AHEAD;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t step[DH / 2];
  __shared__ int4 found[2][WARPS];  // counts of a bisection step, by warp
  __shared__ int scan[2][WARPS];
  __shared__ uint32_t ranked[kRanked], cut_key;
  __shared__ int n_ranked, cut_ties;
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x & (cluster - 1), row = blockIdx.x / cluster;
  const int h = row % a.Hkv, b = row / a.Hkv, layer = blockIdx.y;
  const CachePool pool = a.pool[layer];
  const int n = evict_len(a, b, tid == 0);
  const int m = min(n, a.budget);
  int32_t* kept =
      a.kept + ((static_cast<size_t>(layer) * a.B + b) * a.Hkv + h) * static_cast<size_t>(a.budget);
  if (layer == 0 && h == 0 && rank == 0 && tid == 0) a.new_lens[b] = m;
  if (tid < DH / 2) step[tid] = a.rope.step[tid];
  if (tid == 0) n_ranked = 0;
  const int32_t* table = a.block_table + static_cast<size_t>(b) * a.bt_stride;
  auto owns = [&](int j) { return (j / ROUND & (cluster - 1)) == rank; };
  int same = m;  // positions below stay where they are
  if (n <= a.budget) {
    for (int j = tid; j < a.budget; j += T)
      if (owns(j)) kept[j] = j < m ? j : -1;
  } else {
    // ---- the weight of the last position that stays.  Positions lo .. hi - 1
    // compete; the others' key is 0, which no score has.
    const int lo = a.sinks, hi = n - a.recent, need = a.budget - a.sinks - a.recent;
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    // four positions of a page
    auto load_keys = [&](int p) -> uint4 {
      const int blk = table[p / kPage];
      const bool ok = blk >= 0 && blk < pool.num_blocks;
      // read in any case, so that several reads can be under way
      float4 x = *reinterpret_cast<const float4*>(
          pool.scores + (static_cast<size_t>(ok ? blk : 0) * a.Hkv + h) * kPage + p % kPage);
      if (!ok) {
        record_error(a.err, PE_DEV_BAD_BLOCK);
        x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      }
      auto in = [&](int i) { return p + i >= lo && p + i < hi; };
      return make_uint4(in(0) ? score_key(x.x) : 0u, in(1) ? score_key(x.y) : 0u,
                        in(2) ? score_key(x.z) : 0u, in(3) ? score_key(x.w) : 0u);
    };
    const int held = min((hi + 3) / 4 * 4, key_room);  // positions whose keys are held
    if (need > 0)
#pragma unroll 2
      for (int p = tid * 4; p < held; p += T * 4)
        *reinterpret_cast<uint4*>(keys + p) = load_keys(p);
    __syncthreads();
    // Bisection: count(key >= floor) = at_floor >= need > above = count(key
    // >= floor + 2^shift).  Once few keys lie between, they are ranked.
    uint32_t floor = 0;
    int at_floor = hi - lo, above = 0, shift = 32;
    if (need > 0) {
      for (int odd = 0; shift > 0 && at_floor != need && at_floor - above > kRanked; odd ^= 1) {
        shift -= 2;
        const uint32_t t1 = floor + (1u << shift), t2 = floor + (2u << shift),
                       t3 = floor + (3u << shift);
        int c1 = 0, c2 = 0, c3 = 0;
        auto add = [&](const uint4& k) {
          c1 += (k.x >= t1) + (k.y >= t1) + (k.z >= t1) + (k.w >= t1);
          c2 += (k.x >= t2) + (k.y >= t2) + (k.z >= t2) + (k.w >= t2);
          c3 += (k.x >= t3) + (k.y >= t3) + (k.z >= t3) + (k.w >= t3);
        };
#pragma unroll 2
        for (int p = tid * 4; p < held; p += T * 4) add(*reinterpret_cast<const uint4*>(keys + p));
#pragma unroll 4
        for (int p = held + tid * 4; p < hi; p += T * 4) add(load_keys(p));
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        if (lane == 0) found[odd][warp] = make_int4(c1, c2, c3, 0);
        __syncthreads();  // the other slots were last read before this
        const int4 f = lane < WARPS ? found[odd][lane] : make_int4(0, 0, 0, 0);
        c1 = __reduce_add_sync(0xffffffffu, f.x);
        c2 = __reduce_add_sync(0xffffffffu, f.y);
        c3 = __reduce_add_sync(0xffffffffu, f.z);
        if (c3 >= need) {
          floor = t3;
          at_floor = c3;
        } else if (c2 >= need) {
          floor = t2;
          at_floor = c2;
          above = c3;
        } else if (c1 >= need) {
          floor = t1;
          at_floor = c1;
          above = c2;
        } else {
          above = c1;
        }
      }
    }
    // stay: key > cut, and the first `ties` of key == cut
    uint32_t cut = at_floor == need ? floor - 1 : floor;
    int ties = at_floor == need ? 0 : need - above;
    if (need > 0 && at_floor != need && shift > 0) {
      auto add = [&](uint32_t k) {
        if (k != 0 && (shift == 32 || k - floor < 1u << shift)) {
          const int i = atomicAdd(&n_ranked, 1);
          if (i < kRanked) ranked[i] = k;
        }
      };
      auto add4 = [&](const uint4& k) {
        add(k.x);
        add(k.y);
        add(k.z);
        add(k.w);
      };
      for (int p = tid * 4; p < held; p += T * 4) add4(*reinterpret_cast<const uint4*>(keys + p));
#pragma unroll 4
      for (int p = held + tid * 4; p < hi; p += T * 4) add4(load_keys(p));
      __syncthreads();
      const int count = at_floor - above;
      if (tid < count) {
        const uint32_t k = ranked[tid];
        int more = 0, same_key = 0;
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
          more += ranked[i] > k;
          same_key += ranked[i] == k;
        }
        if (above + more < need && need <= above + more + same_key) {
          cut_key = k;
          cut_ties = need - above - more;
        }
      }
      __syncthreads();
      cut = cut_key;
      ties = cut_ties;
    }
    // ---- the list, in order: each thread an odd number of positions in a row,
    // of as many as the shared memory holds at a time
    int kept_before = lo, eq_before = 0;
    for (int w0 = 0; need > 0 && w0 < hi; w0 += key_room) {
      const int w1 = min(w0 + key_room, hi);
      if (w0 > 0) {
        __syncthreads();
#pragma unroll 4
        for (int p = w0 + tid * 4; p < w1; p += T * 4)
          *reinterpret_cast<uint4*>(keys + p - w0) = load_keys(p);
        __syncthreads();
      }
      const int from = max(lo, w0), count = max(w1 - from, 0), seg = ((count + T - 1) / T) | 1;
      const int p0 = from + min(tid * seg, count), p1 = min(p0 + seg, from + count);
      int gt = 0, eq = 0;
#pragma unroll 4
      for (int p = p0; p < p1; ++p) {
        const uint32_t k = keys[p - w0];
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
      int all_gt = 0, all_eq = 0;
      g -= gt;
      q -= eq;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const int x = scan[0][w], y = scan[1][w];
        all_gt += x;
        all_eq += y;
        g += w < warp ? x : 0;
        q += w < warp ? y : 0;
      }
      const int t = max(ties - eq_before, 0);  // that stay of this window's
      int at = kept_before + g + min(q, t);
      if (gt + eq > 0)
#pragma unroll 4
        for (int p = p0; p < p1; ++p) {
          const uint32_t k = keys[p - w0];
          const bool tie = k == cut;
          if (k > cut || (tie && q < t)) {
            if (owns(at)) kept[at] = p;
            ++at;
          }
          q += tie;
        }
      kept_before += all_gt + min(all_eq, t);
      eq_before += all_eq;
    }
    for (int j = tid; j < lo; j += T)
      if (owns(j)) kept[j] = j;
    for (int j = m - a.recent + tid; j < m; j += T)
      if (owns(j)) kept[j] = n - m + j;
    if (IN_PLACE) same = lo;
  }
  // the list is this CTA's own for the rows that it moves, and the keys' space
  // is free
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
  const uint32_t ring = smem_u32(smem) + tid * 16;
  Move* moves = reinterpret_cast<Move*>(smem + SH::RING);                     // [AHEAD][ROUND]
  float* weights = reinterpret_cast<float*>(moves + AHEAD * ROUND);           // [AHEAD][ROUND]
  // the list's entry of this thread's row x of a round
  auto entry = [&](int round, int x) {
    const int j = round + 2 * group + x;
    return j < m ? __ldcg(kept + j) : -1;
  };
  // rows round + 2 group and + 1 on their way to the ring's place `slot`
  auto issue = [&](int round, const int (&from)[2], int slot) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = round + 2 * group + x, p = from[x];
      Move mv = {-1, 0, 0};
      if (p >= 0 && !(IN_PLACE && p == j)) {
        const int sb = table[p / kPage];
        const bool fits = j / kPage < dstride;
        const int db = fits ? dtab[j / kPage] : -1;
        if (sb >= 0 && sb < pool.num_blocks && db >= 0 && db < pool.num_blocks) {
          const long long src = (static_cast<long long>(sb) * a.Hkv + h) * kPage + p % kPage;
          mv.dst = (static_cast<long long>(db) * a.Hkv + h) * kPage + j % kPage;
          mv.turn = p - j;
          const size_t at = static_cast<size_t>(src) * SH::ROWB + c * 16;
          cp_async(ring + (slot * 4 + x) * T * 16, static_cast<const char*>(pool.k) + at);
          cp_async(ring + (slot * 4 + 2 + x) * T * 16, static_cast<const char*>(pool.v) + at);
          if (c == 0) cp_async4(smem_u32(weights + slot * ROUND + 2 * group + x), pool.scores + src);
        } else if (c == 0) {
          record_error(a.err, fits ? PE_DEV_BAD_BLOCK : PE_DEV_BAD_POSITION);
        }
      }
      if (c == 0) moves[slot * ROUND + 2 * group + x] = mv;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // in place from the first round that may move anything
  const int stride = ROUND * cluster;
  const int first = (IN_PLACE ? same / stride * stride : 0) + rank * ROUND;
  int from[AHEAD + 1][2];
#pragma unroll
  for (int i = 0; i <= AHEAD; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) from[i][x] = entry(first + i * stride, x);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) issue(first + i * stride, from[i], i);
  int slot = 0;
  for (int round = first; round - rank * ROUND < m; round += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    __syncwarp();  // the moves, which another lane of the group wrote
    if (IN_PLACE) {
      // the whole round is read before the first of it is written; later
      // rounds lie behind it
      if (cluster > 1) cluster_sync_all();
      else __syncthreads();
    }
    Move mv[2];
    uint4 kv[2], vv[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mv[x] = moves[slot * ROUND + 2 * group + x];
      kv[x] = *reinterpret_cast<const uint4*>(smem + ((slot * 4 + x) * T + tid) * 16);
      vv[x] = *reinterpret_cast<const uint4*>(smem + ((slot * 4 + 2 + x) * T + tid) * 16);
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
        const size_t at = static_cast<size_t>(mv[x].dst) * SH::ROWB + c * 16;
        *reinterpret_cast<uint4*>(static_cast<char*>(pool.k) + at) = kv[x];
        *reinterpret_cast<uint4*>(static_cast<char*>(pool.v) + at) = vv[x];
        if (c == 0) pool.scores[mv[x].dst] = weights[slot * ROUND + 2 * group + x];
      }
    __syncwarp();  // the slot is free
    issue(round + AHEAD * stride, from[AHEAD], slot);
#pragma unroll
    for (int x = 0; x < 2; ++x) from[AHEAD][x] = entry(round + (AHEAD + 1) * stride, x);
    if (++slot == AHEAD) slot = 0;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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
  // Clusters while there is an SM for every CTA: each of them repeats the
  // choosing, so more do not pay (32 rows of 4096 positions on 152 SMs: 15.7
  // us with 4 CTAs a row, 19.5 with 8).
  const long long rows = static_cast<long long>(a.B) * a.Hkv * n_layers;
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= sms) cluster *= 2;
  const bool alone = rows * cluster <= sms &&
                     static_cast<long long>(a.bt_stride) * kPage > kMostKeys;
  const int room = alone ? kMostKeysAlone : kMostKeys;
  const size_t smem = std::max(EvictShape<S, DH>::SMEM, room * 4);
  static std::atomic<uint64_t> done{0};
  if (dev >= 64 || !((done.load(std::memory_order_relaxed) >> dev) & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_evict_kernel<S, DH, IN_PLACE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               std::max(EvictShape<S, DH>::SMEM,
                                                        kMostKeysAlone * 4));
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev);
  }
  return launch_pdl_cluster(kv_evict_kernel<S, DH, IN_PLACE>,
                            dim3(static_cast<unsigned>(a.B) * a.Hkv * cluster, n_layers),
                            dim3(kEvictThreads), smem, s, cluster, a, cluster, room);
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
    // layers run at the same time
    for (int o = 0; o < l; ++o)
      if (pools[l].k == pools[o].k || pools[l].v == pools[o].v ||
          pools[l].scores == pools[o].scores)
        return PE_ERR_INVALID_ARGUMENT;
  }
  if (B < 1 || !block_table || bt_stride < 1 || !seq_lens || budget < 1 || sinks < 0 ||
      recent < 0 || static_cast<int64_t>(sinks) + recent > budget || !std::isfinite(rope_theta) ||
      rope_theta < 0.f || (dst_table && dst_stride < 1) || !kept || !new_lens ||
      new_lens == seq_lens)
    return PE_ERR_INVALID_ARGUMENT;
  const int64_t rows = static_cast<int64_t>(B) * pools[0].n_kv_heads;
  // the same pages as before: in place
  if (dst_table == block_table) {
    if (dst_stride != bt_stride) return PE_ERR_INVALID_ARGUMENT;
    dst_table = nullptr;
  }
  // positions and list entries are counted in 32 bits
  if (budget > (1 << 30) || bt_stride > (1 << 26) || rows * n_layers > 2147483647LL / budget)
    return PE_ERR_UNSUPPORTED;
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
