// sample.cu -- a token for each row of logits, and the verification of drafts
// by rejection sampling (include/peagle_sample.h has the definitions).
//
// A cluster of CTAs takes a row and holds it in shared memory, so that logits
// cross HBM once.  Weights are whole numbers of 2^-31 of the row's largest:
// counts and sums of them are exact in 64 bits, whatever order the threads,
// warps and CTAs add them in.
#include <algorithm>
#include <cmath>

#include "../../include/peagle_sample.h"
#include "pe_common.cuh"
#include "pe_kernels.h"

namespace pe {

constexpr int kSampleThreads = 384;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kMostCluster = 8;
constexpr int kMostVocab = 393216;  // fp32: 192 KB of each of eight CTAs' shared memory

struct SampleArgs {
  int rows, V, cluster;
  const void* logits;
  long long stride;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tokens;
  float* logprobs;
  pe_dist* dist;
  // verification: windows, drafts (NULL: sampling)
  int B;
  const int32_t* cu_in;
  const int32_t* ids;
  int greedy_drafts;
};

struct VerifyArgs {
  int B, T, V, cluster;
  const void* logits;
  long long stride;
  const int32_t* ids;
  const int32_t* cu_in;
  const float* accept_u;
  const float* u;
  const void* draft_logits;
  long long draft_stride;
  const pe_dist* draft_dist;
  int32_t* num_accepted;
  int32_t* sampled_ids;
  float* logprobs;
  const pe_dist* dist;
  int* err;
};

// ------------------------------------------------------------------ numbers
constexpr float kLargest = 3.402823466e38f;
// NaN counts as -inf, +inf as the largest finite number, -0 as 0 (which gives
// equal logits one sort key).
__device__ __forceinline__ float clean_logit(float x) {
  return fminf(fmaxf(x, -INFINITY), kLargest) + 0.f;
}
// min(x, most); NaN stays NaN.
__device__ __forceinline__ float at_most(float x, float most) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(most));
  return r;
}
// Tokens in their order are falling keys.
__device__ __forceinline__ unsigned long long token_key(float x, int id) {
  return argmax_key(x + 0.f, id);
}
template <typename T>
__device__ __forceinline__ float raw_logit(const T* p) {
  return clean_logit(to_f<T>(*p));
}

struct RowScale {
  float max, inv;
};
// e^((x - max) / T): 0 or NaN for x = -inf.  No contraction: the plain
// operations of the definition.
__device__ __forceinline__ float exp_of(float x, RowScale s) {
  return expf(__fmul_rn(__fsub_rn(x, s.max), s.inv));
}
// Whole numbers of 2^-31 (a NaN converts to 0).
__device__ __forceinline__ uint32_t weight_of(float e) {
  return __float2uint_rn(__fmul_rn(e, 2147483648.f));
}
__device__ __forceinline__ bool is_kept(float x, int id, float cut, int cut_token) {
  return x > cut || (x == cut && id <= cut_token);
}
__device__ __forceinline__ float key_float(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}
// The place that u has in a total.
__device__ __forceinline__ long long place_of(float u, long long total) {
  const long long at = static_cast<long long>(static_cast<double>(u) * static_cast<double>(total));
  return at < 0 ? 0 : at >= total ? total - 1 : at;
}
__device__ __forceinline__ float logprob_of(float x, RowScale s, long long total) {
  const float z = __fmul_rn(__fsub_rn(x, s.max), s.inv);
  return static_cast<float>(static_cast<double>(z) -
                            log(static_cast<double>(total) * 4.656612873077392578125e-10));
}

// ------------------------------------------------------- sums over a cluster
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, m);
    v = o > v ? o : v;
  }
  return v;
}

// No CTA's shared memory is written to by a peer before it has started: there
// is nothing to publish yet.
__device__ __forceinline__ void start_barrier() {
  cluster_arrive_relaxed();
  cluster_wait_acquire();
}

struct Exchange {
  unsigned long long warp[2][kSampleWarps];
  unsigned long long slot[2][2][kMostCluster];  // [parity][value][CTA]
};

// Two 64-bit sums (or a maximum and a sum) over the cluster; every thread gets
// them.  The CTAs' own values stay in ex.slot[parity].  One barrier: the slots
// of the round before the last are free, because whoever has passed the last
// barrier has read them.
template <bool MAX>
__device__ __forceinline__ void cluster_reduce(Exchange& ex, int& parity, int cluster, int rank,
                                               unsigned long long& a, unsigned long long& b) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  a = MAX ? warp_max_u64(a) : warp_sum_u64(a);
  b = warp_sum_u64(b);
  if (lane == 0) {
    ex.warp[0][warp] = a;
    ex.warp[1][warp] = b;
  }
  __syncthreads();
  if (warp < 2) {  // a warp a value
    unsigned long long x = lane < kSampleWarps ? ex.warp[warp][lane] : 0;
    x = MAX && warp == 0 ? warp_max_u64(x) : warp_sum_u64(x);
    if (lane < cluster)
      st_cluster_u64(cluster_map_shared(smem_u32(&ex.slot[parity][warp][rank]), lane), x);
  }
  // the two warps publish what they wrote, and with it what the CTA's other
  // warps wrote before they met above (with a release by every warp 448 rows by
  // temperature take 178 us for 174)
  if (warp < 2) cluster_arrive_release();
  else cluster_arrive_relaxed();
  cluster_wait_acquire();
  a = b = 0;
#pragma unroll
  for (int r = 0; r < kMostCluster; ++r) {
    if (r >= cluster) break;
    const unsigned long long x = ex.slot[parity][0][r];
    a = MAX ? (x > a ? x : a) : a + x;
    b += ex.slot[parity][1][r];
  }
  parity ^= 1;
}

// A CTA's part of a row: 16-byte chunks of the memory that the row lies in;
// elements of a chunk that are not the row's own count as -inf.
template <typename T>
struct Part {
  static constexpr int E = 16 / static_cast<int>(sizeof(T));
  int mis;     // elements of the first chunk of all that lie before the row
  int per;     // chunks of a CTA (the last ones may have fewer)
  int first;   // id of this CTA's first element (may be negative)
  int chunks;  // of this CTA
  __device__ __forceinline__ int owner(int id) const { return (id + mis) / E / per; }
};
template <typename T>
__device__ __forceinline__ Part<T> part_of(const T* row, int V, int cluster, int rank) {
  constexpr int E = Part<T>::E;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % E);
  const int all = (mis + V + E - 1) / E, per = (all + cluster - 1) / cluster;
  const int lo = min(rank * per, all);
  return Part<T>{mis, per, lo * E - mis, min(lo + per, all) - lo};
}
template <typename T>
__device__ __forceinline__ uint4 load_chunk(const T* row, int V, int id) {
  constexpr int E = Part<T>::E;
  if (id >= 0 && id + E <= V) return __ldcs(reinterpret_cast<const uint4*>(row + id));
  uint32_t w[4];
  auto bits = [&](int e) -> uint32_t {
    const bool in = id + e >= 0 && id + e < V;
    if constexpr (sizeof(T) == 4) return in ? __float_as_uint(row[id + e]) : 0xff800000u;
    else return in ? __bfloat16_as_ushort(row[id + e]) : 0xff80u;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = sizeof(T) == 4 ? bits(i) : bits(2 * i) | bits(2 * i + 1) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The logits of a chunk in shared memory, as they came: NaN has weight 0, is
// above and equal to nothing, and falls into the last bin without being asked
// for; a row with +inf is cleaned in place (16-bit logits have no room for the
// largest fp32 number: `most` is that, or +inf where the row has none).
template <typename T>
__device__ __forceinline__ void chunk_logits(const uint4* p, float most, float (&x)[Part<T>::E]) {
  const uint4 v = *p;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = at_most(__uint_as_float(w[i] << 16), most);
      x[2 * i + 1] = at_most(__uint_as_float(w[i] & 0xffff0000u), most);
    }
  }
}

// One of them (read as the words they were written as).
template <typename T>
__device__ __forceinline__ float held_logit(const unsigned char* held, int i, float most) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(held);
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
  else return at_most(__uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16), most);
}

// The largest logit of a chunk, whatever NaN there are (a chunk of NaN: NaN).
template <typename T>
__device__ __forceinline__ float largest_of(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmax3(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z)),
                 __uint_as_float(v.w));
  } else {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
}

// Contiguous chunks of a warp, and of a lane within them, so that sums over
// warps and lanes are in the order of the ids.
struct Segment {
  int lo, hi;
};
__device__ __forceinline__ int warp_segment_size(int chunks) {
  return (chunks + kSampleWarps - 1) / kSampleWarps;
}
__device__ __forceinline__ Segment warp_segment(int chunks) {
  const int per = warp_segment_size(chunks);
  const int lo = min(static_cast<int>(threadIdx.x) / 32 * per, chunks);
  return Segment{lo, min(lo + per, chunks)};
}
__device__ __forceinline__ unsigned long long warp_scan_u64(unsigned long long v) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}
// The element of a warp's segment at which the weights, in order, first
// exceed `at`: the lane's part that holds it, then the element.  Returns chunk
// * E + element on one lane, -1 on the others.
template <int E, typename W>
__device__ __forceinline__ int find_in_segment(Segment seg, long long at, W&& weight) {
  const int lane = threadIdx.x % 32;
  const int per = (seg.hi - seg.lo + 31) / 32;
  const int lo = min(seg.lo + lane * per, seg.hi), hi = min(lo + per, seg.hi);
  unsigned long long own = 0;
  for (int c = lo; c < hi; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) own += weight(c, e);
  const unsigned long long run = warp_scan_u64(own);
  const unsigned hit = __ballot_sync(0xffffffffu, static_cast<long long>(run) > at);
  if (hit == 0) return -1;  // not reached: the sums agree
  const int who = __ffs(hit) - 1;
  at -= static_cast<long long>(__shfl_sync(0xffffffffu, run - own, who));
  const int from = __shfl_sync(0xffffffffu, lo, who) * E, to = __shfl_sync(0xffffffffu, hi, who) * E;
  for (int i0 = from; i0 < to; i0 += 32) {
    const int i = i0 + lane;
    const unsigned long long w = i < to ? weight(i / E, i % E) : 0u;
    const unsigned long long sum = warp_scan_u64(w);
    const long long all = static_cast<long long>(__shfl_sync(0xffffffffu, sum, 31));
    if (at >= all) {
      at -= all;
      continue;
    }
    const unsigned h = __ballot_sync(0xffffffffu, static_cast<long long>(sum) > at);
    return lane == __ffs(h) - 1 ? i : -1;
  }
  return -1;
}

// ------------------------------------------------------------- sampling rows
// Bins of falling logits, 40 an octave of e = 2^(-bin / 40): rounding is
// monotonic, so a larger logit never has a larger bin.  Bins below kSure hold
// W > 0 alone, bins from kBins on (and NaN, which -inf gives) W = 0 alone.
// (64 requests of sampled drafts with mixed filters: 448 us with 48 an octave,
// 441 with 40, 444 with 32: fewer bins to clear and to add up, longer lists.)
constexpr int kPerOctave = 40;
constexpr int kSure = 32 * kPerOctave - 1;
constexpr int kBins = 32 * kPerOctave + 4;
static_assert(kBins >= 1024, "a further level cuts 2^64 keys into at most 2^10");
__device__ __forceinline__ int bin_of(float z) {
  // 8388608 + n has the bits 0x4B000000 + n, a larger or no number larger ones
  const float f = fmaf(z, -57.70780164f, 8388608.f);  // 40 / ln 2
  return static_cast<int>(min(__float_as_uint(f) - 0x4B000000u, static_cast<uint32_t>(kBins)));
}

// Tokens that are ranked one by one, from all CTAs of the cluster.
constexpr int kListed = 640;
struct Listed {
  unsigned long long key[kListed];
  uint32_t w[kListed];
  uint16_t own[kListed];  // this CTA's: element of its part
  uint32_t digits[3][256];
};
union Scratch {
  uint32_t bins[2][kBins];  // counts, or sums of the weights' low and high halves
  Listed list;
};
struct Found {
  unsigned long long before, inside, all;
  int bin;
};
struct SampleShared {
  Exchange ex;
  Found found;
  unsigned long long warp_mass[kSampleWarps];
  unsigned long long scan[kSampleWarps];
  unsigned long long digit_before, digit_inside;
  int digit, listed;
  uint32_t differ[2];
};

// Request r's window [w0, w1) is judged where it has rows of [0, T) and a row of
// the drafter's for each sampled draft, and where nothing in cu_in contradicts it:
// the entries before it lie at or before its start, those after it at or behind
// its end.  Then a bisection finds the window for each of its rows, and no other
// such window has any of them.
__device__ __forceinline__ bool window_fits(int B, int T, int r, int w0, int w1, bool sampled) {
  return w0 >= 0 && w1 > w0 && w1 <= T &&
         !(sampled && w1 - w0 > 1 && (w0 < r || w1 - 2 - r >= T - B));
}
// Whether a thread's share of cu_in contradicts it.
__device__ __forceinline__ bool window_contradicted(const int32_t* cu_in, int B, int r, int w0,
                                                    int w1) {
  bool bad = false;
  for (int i = threadIdx.x; i <= B; i += kSampleThreads) {
    const int at = cu_in[i];
    bad = bad || (i < r && at > w0) || (i > r && at < w1);
  }
  return bad;
}

// The largest k for which the threads' largest logits are asked: past it the
// threads of a row are too few for the k-th of theirs to be near the row's k-th.
// (33 rows of 50,257 bf16 logits with mixed filters: 30 us, and 37 with 64 as
// the limit.)
constexpr int kMostGuess = 256;

// A row's result.
__device__ __forceinline__ void store_row(const SampleArgs& a, bool verify, int r, RowScale sc,
                                          unsigned long long border, long long all, int token,
                                          float logprob) {
  if (!verify) {
    a.tokens[r] = token;
    if (a.logprobs) a.logprobs[r] = logprob;
  }
  if (a.dist) {
    const float cut = border ? key_float(static_cast<uint32_t>(border >> 32)) : -INFINITY;
    const int cut_token = border ? argmax_key_index(border) : a.V - 1;
    uint4* d = reinterpret_cast<uint4*>(a.dist + r);
    d[0] = make_uint4(__float_as_uint(sc.max), __float_as_uint(sc.inv), __float_as_uint(cut),
                      static_cast<uint32_t>(cut_token));
    d[1] = make_uint4(static_cast<uint32_t>(all), static_cast<uint32_t>(all >> 32),
                      static_cast<uint32_t>(token), 0u);
  }
}

// A row whose tokens that pass top-k and min-p are the `first` first of the n
// listed ones; of their weight top-p takes p.  By one CTA: every token's place
// and the weight before it from a comparison with every other, several threads
// a token where there are few.
struct ListRow {
  int n, first;
  bool by_mass, rest;  // rest: tokens of W > 0 are not listed
  double p;
};
template <typename T, bool VERIFY>
__device__ __noinline__ void draw_from_list(const SampleArgs& a, SampleShared& sh, Listed& list,
                                            const ListRow& lr, RowScale sc, int r, int q,
                                            const T* row, int left_out, bool no_draw) {
  constexpr int kEach = (kListed + kSampleThreads - 1) / kSampleThreads;
  const int tid = threadIdx.x, n = lr.n;
  __syncwarp();
  const int per = n <= kSampleThreads / 8   ? 8
                  : n <= kSampleThreads / 4 ? 4
                  : n <= kSampleThreads / 2 ? 2
                                            : 1;  // threads a token
  const int mine = tid / per, part = tid % per;
  unsigned long long key[kEach], before[kEach];
  uint32_t w[kEach], place[kEach];
#pragma unroll
  for (int s = 0; s < kEach; ++s) {
    const int i = mine + s * kSampleThreads;
    key[s] = i < n ? list.key[i] : 0;
    w[s] = i < n ? list.w[i] : 0;
    before[s] = place[s] = 0;
    if (i < n)
      for (int j = part; j < n; j += per)
        if (list.key[j] > key[s]) {
          ++place[s];
          before[s] += list.w[j];
        }
    for (int m = 1; m < per; m <<= 1) {
      place[s] += __shfl_xor_sync(0xffffffffu, place[s], m);
      before[s] += __shfl_xor_sync(0xffffffffu, before[s], m);
    }
  }
  double stop = 0.0;
  if (lr.by_mass) {
#pragma unroll
    for (int s = 0; s < kEach; ++s)
      if (w[s] && place[s] + 1 == lr.first) sh.scan[0] = before[s] + w[s];
    __syncthreads();
    stop = __dmul_rn(lr.p, static_cast<double>(sh.scan[0]));
  }
  int kept = 0;
#pragma unroll
  for (int s = 0; s < kEach; ++s)
    kept += __syncthreads_count(
        w[s] && part == 0 && place[s] < lr.first &&
        (!lr.by_mass || place[s] == 0 || static_cast<double>(before[s]) < stop));
#pragma unroll
  for (int s = 0; s < kEach; ++s)
    if (w[s] && part == 0 && place[s] + 1 == kept) {
      sh.found.before = key[s];
      sh.found.inside = before[s] + w[s];
    }
  __syncthreads();
  const unsigned long long last = sh.found.before, border = kept < n || lr.rest ? last : 0;
  const long long all = static_cast<long long>(sh.found.inside);
  long long share = all;
  if (left_out >= 0) {
    const float x = raw_logit(row + left_out);
    if (token_key(x, left_out) >= last) share -= weight_of(exp_of(x, sc));
  }
  if (share <= 0 || no_draw) {
    if (tid == 0) store_row(a, VERIFY, r, sc, border, all, -1, -INFINITY);
    return;
  }
  // the kept weight of lower ids (a key's low half falls as the id grows)
  const unsigned long long at = static_cast<unsigned long long>(place_of(a.u[q], share));
#pragma unroll
  for (int s = 0; s < kEach; ++s) {
    const bool in = w[s] && key[s] >= last && argmax_key_index(key[s]) != left_out;
    unsigned long long lower = 0;
    if (in)
      for (int j = part; j < n; j += per) {
        const unsigned long long other = list.key[j];
        if (other >= last && static_cast<uint32_t>(other) > static_cast<uint32_t>(key[s]) &&
            argmax_key_index(other) != left_out)
          lower += list.w[j];
      }
    for (int m = 1; m < per; m <<= 1) lower += __shfl_xor_sync(0xffffffffu, lower, m);
    if (in && part == 0 && at >= lower && at - lower < w[s]) {
      const int token = argmax_key_index(key[s]);
      store_row(a, VERIFY, r, sc, border, all, token,
                VERIFY ? 0.f : logprob_of(raw_logit(row + token), sc, all));
    }
  }
}

// A cluster a row.  W needs the row's largest logit before the first sum, and
// each filter a look at every token more, so the row is read from HBM once and
// stays in the cluster's shared memory: reading it again from L2 instead, in
// smaller CTAs or through rings of asynchronous copies, took 192 us where this
// takes 174 (448 rows of 201,088 fp32 logits by temperature, 2.1 TB/s).  What
// bounds a row is the way through its steps, which wait on each other: the
// copy, the largest, the sum, the draw, each behind a meeting of the cluster
// (about 1.5 us), against which two CTAs of different rows share an SM.
//
// Filters look for the last kept token.  Weights and logits fall together, so
// a histogram over falling logits has the sums "of the tokens before" at its
// bins' borders; the limit's own bin (a 40th of a factor of two, a few tokens
// of a usual row) is listed, and the limit found in it by the digits of the
// keys; a bin with more than a list takes is cut by a further histogram of its
// keys.  Additions to bins in shared memory bound that (15 cycles a warp's 32
// where they are spread, two of them a token for sums of weights): 128 rows of
// 151,936 fp32 logits with mixed filters take 101 to 105 us.  For top-k to kMostGuess
// the histogram is of one logit a thread, and one CTA ranks what it lists: one
// row 36 -> 21 us, the 128 mixed ones 131 -> 106 us.
template <typename T, bool VERIFY, bool FILTERS>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_rows_kernel(
    const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) unsigned char held[];
  __shared__ SampleShared sh;
  constexpr int E = Part<T>::E;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cluster = a.cluster, rank = cluster_ctarank();
  int parity = 0;
  start_barrier();
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x / cluster;
  // the row's request, its filters, and the draft that it judges
  int q = r, draft = -1;
  bool judges = false, contradicted = false;
  if (VERIFY) {
    int lo = 0, hi = a.B;  // the last request whose window starts at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu_in[mid] <= r) lo = mid;
      else hi = mid;
    }
    q = lo;
    const int w0 = a.cu_in[q], w1 = a.cu_in[q + 1];
    if (w0 > r || w1 <= r || !window_fits(a.B, a.rows, q, w0, w1, !a.greedy_drafts))
      return;  // the whole cluster
    contradicted = window_contradicted(a.cu_in, a.B, q, w0, w1);
    judges = r + 1 < w1;
    draft = judges ? a.ids[r + 1] : -1;
  }
  const float temp = a.temperature ? a.temperature[q] : 1.f;
  float inv = __fdiv_rn(1.f, temp);
  const bool greedy = !(temp > 0.f) || isinf(inv);
  if (greedy) inv = 0.f;
  const float p = a.top_p ? a.top_p[q] : 1.f;
  int k = a.top_k ? a.top_k[q] : 0;
  if (p <= 0.f) k = 1;  // top-p of nothing: the first token alone
  const bool by_count = k > 0 && k < a.V;
  const bool by_mass = p < 1.f && p > 0.f;
  float min_p = a.min_p ? a.min_p[q] : 0.f;
  min_p = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;  // NaN: 0
  const bool by_share = min_p > 2.328306436538696e-10f;  // 2^-32: W > 0 implies e >= 2^-32

  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  const Part<T> part = part_of(row, a.V, cluster, rank);
  uint4* mine = reinterpret_cast<uint4*>(held);
  Scratch& scr = *reinterpret_cast<Scratch*>(held + static_cast<size_t>(part.per) * 16);
  float top = -INFINITY;
  constexpr int kFly = 6;  // chunks of a thread on their way
  for (int c0 = tid; c0 < part.chunks; c0 += kFly * kSampleThreads) {
    uint4 v[kFly];
#pragma unroll
    for (int i = 0; i < kFly; ++i)
      if (c0 + i * kSampleThreads < part.chunks)
        v[i] = load_chunk(row, a.V, part.first + (c0 + i * kSampleThreads) * E);
#pragma unroll
    for (int i = 0; i < kFly; ++i) {
      const int c = c0 + i * kSampleThreads;
      if (c >= part.chunks) break;
      mine[c] = v[i];
      top = fmaxf(top, largest_of<T>(v[i]));
    }
  }
  unsigned long long x = float_order_key(top + 0.f), y = contradicted;
  cluster_reduce<true>(sh.ex, parity, cluster, rank, x, y);
  if (VERIFY && y) return;  // the whole cluster
  RowScale sc = {key_float(static_cast<uint32_t>(x)), inv};
  float most = INFINITY;
  if (sc.max == INFINITY) {
    sc.max = most = kLargest;
    if constexpr (sizeof(T) == 4) {
      for (int c = tid; c < part.chunks; c += kSampleThreads) {
        const uint4 v = mine[c];
        mine[c] = make_uint4(__float_as_uint(at_most(__uint_as_float(v.x), most)),
                             __float_as_uint(at_most(__uint_as_float(v.y), most)),
                             __float_as_uint(at_most(__uint_as_float(v.z), most)),
                             __float_as_uint(at_most(__uint_as_float(v.w), most)));
      }
      __syncthreads();
    }
  }

  // Every element of this CTA, in no order: test(logit, id).
  auto each = [&](auto&& test) {
#pragma unroll 2
    for (int c = tid; c < part.chunks; c += kSampleThreads) {
      float v[E];
      chunk_logits<T>(mine + c, most, v);
#pragma unroll
      for (int e = 0; e < E; ++e) test(v[e], c * E + e);
    }
  };

  // The last kept token's key; 0: every token of W > 0 is kept.
  unsigned long long border = 0;
  const Segment seg = warp_segment(part.chunks);
  unsigned long long own = 0;      // kept weight of this warp's segment
  bool summed = false;             // ... and is it there yet
  unsigned long long best = 0;     // a greedy row's token
  if (sc.max > -INFINITY && greedy) {
    // the lowest id of the largest logit, and whether any other logit is finite
    unsigned long long others = 0;
    each([&](float v, int i) {
      if (v == sc.max) {
        const unsigned long long key = token_key(v, part.first + i);
        best = key > best ? key : best;
      }
      others += __fsub_rn(v, sc.max) > -INFINITY;
    });
    cluster_reduce<true>(sh.ex, parity, cluster, rank, best, others);
    border = others > 1 ? best : 0;
  } else if (FILTERS && sc.max > -INFINITY && (by_count || by_mass || by_share)) {
    // Which tokens pass the filters other than the one that is being applied:
    // bins below `sure` do, bins above `last` do not, the rest are looked at.
    int sure = kSure, last = kBins - 1;
    if (by_share) {
      const int at = bin_of(logf(min_p));
      sure = min(sure, at - 2);
      last = min(last, at + 2);
    }
    unsigned long long floor_key = 0;
    bool short_of = false;  // some token of W > 0 is kept by no stage so far
    auto able = [&](float v, float z, int bin, int i) {
      if (bin < sure) return true;
      if (bin > last) return false;
      const float e = expf(z);
      return weight_of(e) > 0 && e >= min_p && token_key(v, part.first + i) >= floor_key;
    };
    auto clear_bins = [&]() {
      for (int i = tid; i < kBins; i += kSampleThreads) scr.bins[0][i] = scr.bins[1][i] = 0;
      __syncthreads();
    };
    // The bin, and within it the range of keys, that a limit falls into, and
    // the measure of what comes before.
    auto histogram = [&](bool count, auto&& place) {
      clear_bins();
      each([&](float v, int i) {
        const float z = __fmul_rn(__fsub_rn(v, sc.max), sc.inv);
        const int bin = bin_of(z);
        const int at = place(v, bin, i);
        if (at < 0) return;
        if (!able(v, z, bin, i)) {
          short_of = short_of || bin < kSure || weight_of(expf(z)) > 0;
          return;
        }
        if (count) {
          atomicAdd(&scr.bins[0][at], 1u);
        } else {
          const uint32_t w = weight_of(expf(z));
          atomicAdd(&scr.bins[0][at], w & 0xffffu);  // at most 2^16 elements a CTA
          atomicAdd(&scr.bins[1][at], w >> 16);
        }
      });
      cluster_barrier();
    };
    // Every CTA adds up its share of the bins over the cluster; whoever finds
    // the limit tells the others.  `limit` gets the measure of all bins.
    auto search = [&](bool count, unsigned long long base, auto&& limit) {
      constexpr int kMost = (kBins + kSampleThreads - 1) / kSampleThreads;
      const int share = (kBins + cluster - 1) / cluster, lo = rank * share;
      const int each_bins = (share + kSampleThreads - 1) / kSampleThreads;
      unsigned long long v[kMost], sum = 0;
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        v[j] = 0;
        const int at = tid * each_bins + j;
        if (j < each_bins && at < share && lo + at < kBins) {
          uint32_t l[kMostCluster] = {}, h[kMostCluster] = {};
#pragma unroll
          for (int c = 0; c < kMostCluster; ++c)
            if (c < cluster) {
              const uint32_t* from = cluster_pointer(&scr.bins[0][lo + at], c);
              l[c] = from[0];
              if (!count) h[c] = from[kBins];
            }
#pragma unroll
          for (int c = 0; c < kMostCluster; ++c)
            v[j] += l[c] + (static_cast<unsigned long long>(h[c]) << 16);
        }
        sum += v[j];
      }
      const unsigned long long run = warp_scan_u64(sum);
      if (lane == 31) sh.scan[warp] = run;
      unsigned long long all = sum, none = 0;
      const int par = parity;
      cluster_reduce<false>(sh.ex, parity, cluster, rank, all, none);
      unsigned long long before = base + run - sum;
      for (int i = 0; i < rank; ++i) before += sh.ex.slot[par][0][i];
      for (int i = 0; i < warp; ++i) before += sh.scan[i];
      const double stop = limit(all);
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        if (v[j] && static_cast<double>(before) < stop &&
            !(static_cast<double>(before + v[j]) < stop))
          for (int c = 0; c < cluster; ++c) {
            const uint32_t to = cluster_map_shared(smem_u32(&sh.found), c);
            st_cluster_u64(to, before);
            st_cluster_u64(to + 8, v[j]);
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 24),
                         "r"(lo + tid * each_bins + j)
                         : "memory");
          }
        before += v[j];
      }
      cluster_barrier();
      Found f = sh.found;
      f.all = all;
      return f;
    };
    // The last token of `listed` ones before which the measure is below the
    // limit: eight bits of the keys at a time.  Every CTA has the whole list.
    auto select = [&](int listed, bool count, unsigned long long base, double stop,
                      unsigned long long floor) {
      constexpr int kEach = (kListed + kSampleThreads - 1) / kSampleThreads;
      unsigned long long key[kEach];
      uint32_t w[kEach];
      bool on[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = tid + j * kSampleThreads;
        on[j] = i < listed;
        key[j] = on[j] ? scr.list.key[i] : 0;
        w[j] = on[j] ? scr.list.w[i] : 0;
        on[j] = on[j] && key[j] >= floor;
      }
      // what all keys have in common is skipped
      uint32_t hi_differ = 0, lo_differ = 0;
      const unsigned long long some = scr.list.key[0];
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (on[j]) {
          hi_differ |= static_cast<uint32_t>((key[j] ^ some) >> 32);
          lo_differ |= static_cast<uint32_t>(key[j] ^ some);
        }
      if (tid == 0) sh.differ[0] = sh.differ[1] = 0;
      __syncthreads();
      hi_differ = __reduce_or_sync(0xffffffffu, hi_differ);
      lo_differ = __reduce_or_sync(0xffffffffu, lo_differ);
      if (lane == 0 && hi_differ) atomicOr(&sh.differ[0], hi_differ);
      if (lane == 0 && lo_differ) atomicOr(&sh.differ[1], lo_differ);
      __syncthreads();
      const int bits = sh.differ[0] ? 64 - __clz(sh.differ[0]) : 32 - __clz(sh.differ[1]);
      const int first_shift = bits <= 8 ? 0 : (bits + 7) / 8 * 8 - 8;
      unsigned long long result =
          first_shift >= 56 ? 0 : some >> (first_shift + 8) << (first_shift + 8);
      for (int shift = first_shift; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSampleThreads)
          scr.list.digits[0][i] = scr.list.digits[1][i] = scr.list.digits[2][i] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (on[j]) {
            const int d = static_cast<int>(key[j] >> shift) & 255;
            atomicAdd(&scr.list.digits[0][d], 1u);
            atomicAdd(&scr.list.digits[1][d], w[j] & 0xffffu);
            atomicAdd(&scr.list.digits[2][d], w[j] >> 16);
          }
        __syncthreads();
        if (warp == 0) {
          // lane 0 has the largest digits
          unsigned long long v[8], sum = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = 255 - lane * 8 - i;
            v[i] = count ? scr.list.digits[0][d]
                         : scr.list.digits[1][d] + (static_cast<unsigned long long>(scr.list.digits[2][d]) << 16);
            sum += v[i];
          }
          unsigned long long before = base + warp_scan_u64(sum) - sum;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (v[i] && static_cast<double>(before) < stop &&
                !(static_cast<double>(before + v[i]) < stop)) {
              sh.digit = 255 - lane * 8 - i;
              sh.digit_before = before;
              sh.digit_inside = scr.list.digits[0][255 - lane * 8 - i];
            }
            before += v[i];
          }
        }
        __syncthreads();
        const unsigned long long d = static_cast<unsigned long long>(sh.digit);
        base = sh.digit_before;
        result |= d << shift;
#pragma unroll
        for (int j = 0; j < kEach; ++j) on[j] = on[j] && ((key[j] >> shift) & 255) == d;
        if (sh.digit_inside == 1) {
#pragma unroll
          for (int j = 0; j < kEach; ++j)
            if (on[j]) sh.found.before = key[j];
          __syncthreads();
          result = sh.found.before;
          break;
        }
        __syncthreads();
      }
      return result;
    };

    bool done = false;
    if (!by_count && !by_mass) {
      // min-p alone: a look at each token is enough
      own = 0;
      unsigned long long last_key = ~0ull, short_n = 0;
      for (int c = seg.lo + lane; c < seg.hi; c += 32) {
        float v[E];
        chunk_logits<T>(mine + c, most, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float z = __fmul_rn(__fsub_rn(v[e], sc.max), sc.inv);
          const int bin = bin_of(z);
          if (bin >= kBins) continue;
          if (able(v[e], z, bin, c * E + e)) {
            own += weight_of(expf(z));
            const unsigned long long key = token_key(v[e], part.first + c * E + e);
            last_key = key < last_key ? key : last_key;
          } else {
            short_n |= bin < kSure || weight_of(expf(z)) > 0;
          }
        }
      }
      own = warp_sum_u64(own);
      if (lane == 0) sh.warp_mass[warp] = own;
      unsigned long long inverse = ~last_key;
      cluster_reduce<true>(sh.ex, parity, cluster, rank, inverse, short_n);
      border = short_n ? ~inverse : 0;
      done = summed = true;
    } else if (by_count && k <= kMostGuess) {
      // Few tokens are kept, and they are among a few: of at least k threads the
      // largest logit is in the bin that is found, or before it, so at least k
      // tokens are.
      clear_bins();
      if (tid == 0) sh.listed = 0;
      const float tv = at_most(top, most), tz = __fmul_rn(__fsub_rn(tv, sc.max), sc.inv);
      const int tb = bin_of(tz);
      if (tb < kBins && able(tv, tz, tb, 0)) atomicAdd(&scr.bins[0][tb], 1u);
      cluster_barrier();
      const Found f = search(true, 0, [&](unsigned long long all) {
        return fmin(static_cast<double>(k), static_cast<double>(all));
      });
      const int hi_bin = f.all < k ? kBins - 1 : f.bin;
      bool rest = false;
      each([&](float v, int i) {
        const float z = __fmul_rn(__fsub_rn(v, sc.max), sc.inv);
        const int bin = bin_of(z);
        if (bin > hi_bin || !able(v, z, bin, i)) {
          rest = rest || bin < kSure || (bin < kBins && weight_of(expf(z)) > 0);
          return;
        }
        const int at = atomicAdd(&sh.listed, 1);
        if (at < kListed) scr.list.own[at] = static_cast<uint16_t>(i);
      });
      __syncthreads();
      unsigned long long n = tid == 0 ? static_cast<unsigned>(sh.listed) : 0u, others = rest;
      const int par = parity;
      cluster_reduce<false>(sh.ex, parity, cluster, rank, n, others);
      const int listed = static_cast<int>(n);
      if (listed <= kListed) {
        // the first CTA does the rest, and the others leave
        int at = 0;
        for (int i = 0; i < rank; ++i) at += static_cast<int>(sh.ex.slot[par][0][i]);
        const int here = static_cast<int>(sh.ex.slot[par][0][rank]);
        for (int j = tid; j < here; j += kSampleThreads) {
          const int el = scr.list.own[j];
          const float xv = held_logit<T>(held, el, most);
          st_cluster_u64(cluster_map_shared(smem_u32(&scr.list.key[at + j]), 0),
                         token_key(xv, part.first + el));
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                           cluster_map_shared(smem_u32(&scr.list.w[at + j]), 0)),
                       "r"(weight_of(exp_of(xv, sc)))
                       : "memory");
        }
        cluster_barrier();
        if (rank == 0) {
          const ListRow lr = {listed, min(k, listed), by_mass, others > 0, static_cast<double>(p)};
          const int left_out = VERIFY && a.greedy_drafts && draft >= 0 && draft < a.V ? draft : -1;
          draw_from_list<T, VERIFY>(a, sh, scr.list, lr, sc, r, q, row, left_out,
                                    VERIFY && judges && !a.greedy_drafts);
        }
        return;
      }
    }

    // by number (top-k), by weight (top-p), or one after the other
    for (int stage = by_count ? 0 : 1; stage < (by_mass ? 2 : 1) && !done; ++stage) {
      const bool count = stage == 0;
      double stop = 0.0;
      auto limit = [&](unsigned long long all) {
        const double n = static_cast<double>(all);
        return stop = count ? fmin(static_cast<double>(k), n) : __dmul_rn(static_cast<double>(p), n);
      };
      histogram(count, [&](float, int bin, int) { return bin < kBins ? bin : -1; });
      Found f = search(count, 0, limit);
      // (weights of what passes sum to more than 0 each, so both measures tell)
      short_of = short_of || f.before + f.inside < f.all;
      unsigned long long low = 0, high = ~0ull;  // keys within the bin
      int lo_bin = f.bin;
      if (count && f.before + f.inside <= kListed) {
        lo_bin = 0;  // few tokens in all: rank every one
        f.before = 0;
      }
      const int hi_bin = f.bin;
      int listed;
      unsigned long long dropped;  // somewhere in the range's bin, or short_of
      // (each further level has 2^-10 of the keys of the one before, of 2^64)
      for (int level = 0; level < 8; ++level) {
        // weights before the range, by segments; the range's own tokens
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        own = 0;
        bool drop = short_of;
        unsigned long long first_key = 0, last_key = ~0ull;
        for (int c = seg.lo + lane; c < seg.hi; c += 32) {
          float v[E];
          chunk_logits<T>(mine + c, most, v);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float z = __fmul_rn(__fsub_rn(v[e], sc.max), sc.inv);
            const int bin = bin_of(z);
            if (bin > hi_bin || !able(v[e], z, bin, c * E + e)) continue;
            if (bin < lo_bin) {
              own += weight_of(expf(z));
              continue;
            }
            const unsigned long long key = token_key(v[e], part.first + c * E + e);
            if (key > high) {
              own += weight_of(expf(z));
            } else if (key < low) {
              drop = true;
            } else {
              last_key = key < last_key ? key : last_key;
              first_key = key > first_key ? key : first_key;
              const int at = atomicAdd(&sh.listed, 1);
              if (at < kListed) scr.list.own[at] = static_cast<uint16_t>(c * E + e);
            }
          }
        }
        __syncthreads();
        unsigned long long n = static_cast<unsigned long long>(tid == 0 ? sh.listed : 0);
        dropped = drop;
        const int par = parity;
        cluster_reduce<false>(sh.ex, parity, cluster, rank, n, dropped);
        listed = static_cast<int>(n);
        if (listed <= kListed) {
          int at = 0;
          for (int i = 0; i < rank; ++i) at += static_cast<int>(sh.ex.slot[par][0][i]);
          const int here = static_cast<int>(sh.ex.slot[par][0][rank]);
          for (int i = tid; i < here * cluster; i += kSampleThreads) {
            const int to = i / here, j = i % here, el = scr.list.own[j];
            const float xv = held_logit<T>(held, el, most);
            st_cluster_u64(cluster_map_shared(smem_u32(&scr.list.key[at + j]), to),
                           token_key(xv, part.first + el));
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                             cluster_map_shared(smem_u32(&scr.list.w[at + j]), to)),
                         "r"(weight_of(exp_of(xv, sc)))
                         : "memory");
          }
          cluster_barrier();
          break;
        }
        // too many to rank: bins of the range's keys (ties go by their ids)
        unsigned long long inverse = ~last_key;
        cluster_reduce<true>(sh.ex, parity, cluster, rank, inverse, dropped);
        low = ~inverse;
        unsigned long long none = 0;
        cluster_reduce<true>(sh.ex, parity, cluster, rank, first_key, none);
        high = first_key;
        int shift = 0;
        while (shift < 54 && ((high - low) >> shift) >= kBins) ++shift;
        lo_bin = hi_bin;  // (the range is that bin's: lists of all bins are short)
        const unsigned long long lowest = low, highest = high;
        histogram(count, [&](float v, int bin, int i) {
          if (bin != hi_bin) return -1;
          const unsigned long long key = token_key(v, part.first + i);
          return key < lowest || key > highest ? -1 : static_cast<int>((highest - key) >> shift);
        });
        f = search(count, f.before, [&](unsigned long long) { return stop; });
        high = highest - (static_cast<unsigned long long>(f.bin) << shift);
        const unsigned long long end = high - ((1ull << shift) - 1);
        low = end > lowest && end <= high ? end : lowest;
      }
      listed = min(listed, kListed);
      border = select(listed, count, f.before, stop, 0);
      if (count && by_mass && lo_bin == 0 && listed <= kListed && hi_bin == f.bin && high == ~0ull) {
        // all that is left is in the list: the weights' limit in it
        unsigned long long mass = 0, none = 0;
        for (int i = tid; i < listed; i += kSampleThreads)
          if (scr.list.key[i] >= border) mass += scr.list.w[i];
        mass = warp_sum_u64(mass);
        if (lane == 0) sh.scan[warp] = mass;
        __syncthreads();
        for (int i = 0; i < kSampleWarps; ++i) none += sh.scan[i];
        __syncthreads();
        border = select(listed, false, 0, __dmul_rn(static_cast<double>(p), static_cast<double>(none)),
                        border);
        stage = 2;
      } else if (count && by_mass) {
        // the second stage's tokens: at or above this border
        floor_key = border;
        const float v = key_float(static_cast<uint32_t>(border >> 32));
        const int at = bin_of(__fmul_rn(__fsub_rn(v, sc.max), sc.inv));
        sure = min(sure, at);
        last = min(last, at);
        cluster_barrier();  // the list is read: its memory may be bins again
        continue;
      }
      // the list's kept tokens join their segments
      __syncthreads();
      own = warp_sum_u64(own);
      if (lane == 0) sh.warp_mass[warp] = own;
      __syncthreads();
      const int per = warp_segment_size(part.chunks);
      bool left = false;
      for (int i = tid; i < listed; i += kSampleThreads) {
        const unsigned long long key = scr.list.key[i], w = scr.list.w[i];
        if (key < border) {
          left = true;
          continue;
        }
        const int id = argmax_key_index(key);
        if (part.owner(id) == rank) atomicAdd(&sh.warp_mass[(id - part.first) / E / per], w);
      }
      if (!__syncthreads_or(left) && !dropped) border = 0;
      own = sh.warp_mass[warp];
      summed = true;
    }
  }
  const float cut = border ? key_float(static_cast<uint32_t>(border >> 32)) : -INFINITY;
  const int cut_token = border ? argmax_key_index(border) : a.V - 1;

  // Draw.  A greedy draft that this row may reject has no share.
  const int left_out = VERIFY && a.greedy_drafts && draft >= 0 && draft < a.V ? draft : -1;
  auto weight = [&](int c, int e) -> uint32_t {
    const float v = held_logit<T>(held, c * E + e, most);
    const int id = part.first + c * E + e;
    if (!is_kept(v, id, cut, cut_token) || id == left_out) return 0;
    return weight_of(exp_of(v, sc));
  };
  if (!summed) {
    // every token, or a greedy row's one
    own = 0;
    if (!greedy) {
#pragma unroll 2
      for (int c = seg.lo + lane; c < seg.hi; c += 32) {
        float v[E];
        chunk_logits<T>(mine + c, most, v);
#pragma unroll
        for (int e = 0; e < E; ++e) own += weight_of(exp_of(v[e], sc));
      }
    } else if (sc.max > -INFINITY && part.owner(argmax_key_index(best)) == rank) {
      const int at = (argmax_key_index(best) - part.first) / E;
      if (at / warp_segment_size(part.chunks) == warp && lane == 0) own = weight_of(1.f);
    }
    own = warp_sum_u64(own);
    if (lane == 0) sh.warp_mass[warp] = own;
  }
  unsigned long long total = lane == 0 ? own : 0, none = 0;
  const int par = parity;
  cluster_reduce<false>(sh.ex, parity, cluster, rank, total, none);
  const long long all = static_cast<long long>(total);
  long long share = all, out = 0;  // what is drawn from, and what is left out of it
  if (left_out >= 0) {
    const float v = raw_logit(row + left_out);
    if (is_kept(v, left_out, cut, cut_token)) out = weight_of(exp_of(v, sc));
    share -= out;
  }
  const bool draws = share > 0 && !(VERIFY && judges && !a.greedy_drafts);
  int token = -1;
  if (draws) {
    long long at = place_of(a.u[q], share);
    const int of = out ? part.owner(left_out) : -1;
    for (int i = 0; i < rank; ++i)
      at -= static_cast<long long>(sh.ex.slot[par][0][i]) - (i == of ? out : 0);
    const int in = of == rank ? (left_out - part.first) / E / warp_segment_size(part.chunks) : -1;
    for (int i = 0; i < warp; ++i)
      at -= static_cast<long long>(sh.warp_mass[i]) - (i == in ? out : 0);
    if (at >= 0 && at < static_cast<long long>(own) - (warp == in ? out : 0)) {
      const int i = find_in_segment<E>(seg, at, weight);
      if (i >= 0) token = part.first + i;
    }
  }
  if (token >= 0 || (!draws && rank == 0 && tid == 0))
    store_row(a, VERIFY, r, sc, border, all, token,
              token >= 0 && !VERIFY ? logprob_of(raw_logit(row + token), sc, all) : -INFINITY);
}

// -------------------------------------------------------------- verification
// The weight of a token in a row that a record describes.
template <typename T>
__device__ __forceinline__ uint32_t dist_weight(float x, int id, const pe_dist& d) {
  if (!is_kept(x, id, d.cut, d.cut_token)) return 0;
  return weight_of(exp_of(x, RowScale{d.max, d.inv}));
}

// A cluster a request: its first rejected draft, and the token drawn there.
// A request's window takes a few reads; with sampled drafts the two rows of the
// first rejected one are read once, 16 bytes at a time, and the weights of what
// the target has more of are held in shared memory for the draw, which goes by
// the order of ids.  Two exponentials a token and the wait for the rows bound
// that: 64 requests, 201,088 fp32 logits, take 72 us here (1.4 TB/s) after 394
// in the kernel above, which has their 512 rows.
template <typename T>
__global__ void __launch_bounds__(kSampleThreads) verify_kernel(
    const __grid_constant__ VerifyArgs a) {
  extern __shared__ __align__(16) unsigned char held_weights[];
  __shared__ Exchange ex;
  __shared__ unsigned long long warp_mass[2][kSampleWarps];
  constexpr int E = Part<T>::E;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cluster = a.cluster, rank = cluster_ctarank(), r = blockIdx.x / cluster;
  int parity = 0;
  start_barrier();
  grid_dep_wait();
  grid_dep_launch();
  const int w0 = a.cu_in[r], w1 = a.cu_in[r + 1];
  if (!window_fits(a.B, a.T, r, w0, w1, a.draft_logits != nullptr) ||
      __syncthreads_or(window_contradicted(a.cu_in, a.B, r, w0, w1))) {
    if (rank == 0 && tid == 0) {
      record_error(a.err, PE_DEV_BAD_ROW);
      a.num_accepted[r] = 0;
      a.sampled_ids[r] = -1;
    }
    return;  // the whole cluster
  }
  const T* logits = static_cast<const T*>(a.logits);
  const T* draft_logits = static_cast<const T*>(a.draft_logits);
  // drafts of no token are recorded wherever they are, judged or not
  if (rank == 0 && warp == kSampleWarps - 1)
    for (int t = w0 + lane; t < w1 - 1; t += 32)
      if (a.ids[t + 1] < 0 || a.ids[t + 1] >= a.V) record_error(a.err, PE_DEV_BAD_TOKEN);
  // every warp finds the first rejection for itself, 32 drafts at a time
  int stop = w1 - 1;
  for (int t0 = w0; t0 < w1 - 1; t0 += 32) {
    const int t = t0 + lane;
    bool ok = true;
    if (t < w1 - 1) {
      const int d = a.ids[t + 1], from = t - r;
      const pe_dist P = a.dist[t];
      uint32_t w = 0, wq = 0;
      long long totalq = 0;
      if (d >= 0 && d < a.V) {
        w = dist_weight<T>(raw_logit(logits + t * a.stride + d), d, P);
        if (draft_logits) {
          const pe_dist Q = a.draft_dist[from];
          wq = dist_weight<T>(raw_logit(draft_logits + from * a.draft_stride + d), d, Q);
          totalq = Q.total;
        }
      }
      const double u = a.accept_u[t];
      if (draft_logits)
        ok = w > 0 && u * static_cast<double>(wq) * static_cast<double>(P.total) <
                          static_cast<double>(w) * static_cast<double>(totalq);
      else
        ok = w > 0 && (w == P.total || u * static_cast<double>(P.total) < static_cast<double>(w));
    }
    const unsigned bad = __ballot_sync(0xffffffffu, !ok);
    if (bad) {
      stop = t0 + __ffs(bad) - 1;
      break;
    }
  }
  const pe_dist P = a.dist[stop];
  const T* row = logits + stop * a.stride;
  int token = P.token;
  bool writes = rank == 0 && tid == 0;
  const int from = stop - r;
  if (draft_logits && stop < w1 - 1 && P.total > 0) {
    // rejected: from what the target has more of than the drafter
    const pe_dist Q = a.draft_dist[from];
    const T* qrow = draft_logits + from * a.draft_stride;
    const float ap = static_cast<float>(2147483648.0 / static_cast<double>(P.total));
    const float aq =
        Q.total > 0 ? static_cast<float>(2147483648.0 / static_cast<double>(Q.total)) : 0.f;
    const Part<T> part = part_of(row, a.V, cluster, rank);
    // the drafter's row beside it: 16 bytes at a time where they lie alike
    const bool alike = (reinterpret_cast<uintptr_t>(row) - reinterpret_cast<uintptr_t>(qrow)) % 16 == 0;
    uint32_t* held = reinterpret_cast<uint32_t*>(held_weights);
    const RowScale ps = {P.max, P.inv}, qs = {Q.max, Q.inv};
    auto weights_of = [&](float x, float y, int id, uint32_t& m, uint32_t& n) {
      const uint32_t wp = is_kept(x, id, P.cut, P.cut_token) ? weight_of(exp_of(x, ps)) : 0u;
      const uint32_t wq = is_kept(y, id, Q.cut, Q.cut_token) ? weight_of(exp_of(y, qs)) : 0u;
      const float pw = __fmul_rn(static_cast<float>(wp), ap);
      n = __float2uint_rn(pw);
      m = __float2uint_rn(fmaxf(__fsub_rn(pw, __fmul_rn(static_cast<float>(wq), aq)), 0.f));
    };
    const Segment seg = warp_segment(part.chunks);
    unsigned long long more = 0, plain = 0;
#pragma unroll 2
    for (int c = seg.lo + lane; c < seg.hi; c += 32) {
      const int first = part.first + c * E;
      const uint4 pv = load_chunk(row, a.V, first);
      uint4 qv;
      if (alike) {
        qv = load_chunk(qrow, a.V, first);
      } else {
        uint32_t w[4];
        auto bits = [&](int e) -> uint32_t {
          const bool in = first + e >= 0 && first + e < a.V;
          if constexpr (sizeof(T) == 4) return in ? __float_as_uint(qrow[first + e]) : 0xff800000u;
          else return in ? __bfloat16_as_ushort(qrow[first + e]) : 0xff80u;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = sizeof(T) == 4 ? bits(i) : bits(2 * i) | bits(2 * i + 1) << 16;
        qv = make_uint4(w[0], w[1], w[2], w[3]);
      }
      float px[E], qx[E];
      chunk_logits<T>(&pv, INFINITY, px);
      chunk_logits<T>(&qv, INFINITY, qx);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t m, n;
        weights_of(clean_logit(px[e]), clean_logit(qx[e]), first + e, m, n);
        held[c * E + e] = m;
        more += m;
        plain += n;
      }
    }
    unsigned long long total_more = more, total_plain = plain;
    more = warp_sum_u64(more);
    plain = warp_sum_u64(plain);
    if (lane == 0) {
      warp_mass[0][warp] = more;
      warp_mass[1][warp] = plain;
    }
    cluster_reduce<false>(ex, parity, cluster, rank, total_more, total_plain);
    const int use = total_more ? 0 : 1;
    const long long total = static_cast<long long>(use ? total_plain : total_more);
    const long long own = static_cast<long long>(use ? plain : more);
    token = -1;
    writes = false;
    long long at = place_of(a.u[r], total);
    for (int i = 0; i < rank; ++i) at -= static_cast<long long>(ex.slot[0][use][i]);
    for (int i = 0; i < warp; ++i) at -= static_cast<long long>(warp_mass[use][i]);
    if (at >= 0 && at < own) {
      const int i = find_in_segment<E>(seg, at, [&](int c, int e) {
        if (!use) return held[c * E + e];
        const int id = part.first + c * E + e;
        uint32_t m = 0, n = 0;
        if (id >= 0 && id < a.V) weights_of(raw_logit(row + id), raw_logit(qrow + id), id, m, n);
        return n;
      });
      if (i >= 0) token = part.first + i;
      writes = token >= 0;
    }
  }
  if (writes) {
    a.num_accepted[r] = stop - w0;
    a.sampled_ids[r] = token;
  }
  if (a.logprobs) {
    if (writes) {
      float lp = -INFINITY;
      if (token >= 0 && token < a.V && P.total > 0) {
        const float x = raw_logit(row + token);
        if (dist_weight<T>(x, token, P)) lp = logprob_of(x, RowScale{P.max, P.inv}, P.total);
      }
      a.logprobs[stop] = lp;
    }
    if (rank == 0)
      for (int t = w0 + tid; t < w1; t += kSampleThreads) {
        if (t < stop) {  // accepted, so a token of the vocabulary that is kept
          const int d = a.ids[t + 1];
          const pe_dist D = a.dist[t];
          a.logprobs[t] =
              logprob_of(raw_logit(logits + t * a.stride + d), RowScale{D.max, D.inv}, D.total);
        } else if (t > stop) {
          a.logprobs[t] = 0.f;
        }
      }
  }
}

// -------------------------------------------------------------------- launch
// Shared memory of one of two CTAs on an SM.
constexpr size_t kHalfShared = 112 * 1024 - sizeof(SampleShared);
// The most that a CTA takes, of rows or of weights.  (A kernel's limit is always
// set to the same, never to what one call needs: another thread's call may lie
// between setting and launching.)
constexpr size_t kMostShared = static_cast<size_t>(kMostVocab / kMostCluster) * 4 + 64 + sizeof(Scratch);
struct SampleShape {
  int cluster;
  size_t smem;
};
// Few rows: as many CTAs a row as a cluster has, for the shortest way (33 rows
// of 50,257 bf16 logits: 30 us by eight CTAs each, 59 by one); more rows than
// that fills: as few as hold the row, two to an SM.
static SampleShape sample_shape(int rows, int V, int elem, int sms) {
  auto bytes = [&](int c) {
    const int e = 16 / elem, all = (V + 2 * (e - 1)) / e;
    return static_cast<size_t>((all + c - 1) / c) * 16 + sizeof(Scratch);
  };
  int c = 1;
  while (c < kMostCluster && bytes(c) > kHalfShared) c *= 2;
  while (c < kMostCluster && static_cast<long long>(rows) * c * 2 <= 2 * sms &&
         bytes(c) > sizeof(Scratch) + 4096)
    c *= 2;
  return SampleShape{c, bytes(c)};
}

template <typename T, bool VERIFY, bool FILTERS>
static cudaError_t launch_rows(SampleArgs a, int sms, cudaStream_t s) {
  const SampleShape sh = sample_shape(a.rows, a.V, sizeof(T), sms);
  a.cluster = sh.cluster;
  auto kernel = sample_rows_kernel<T, VERIFY, FILTERS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMostShared));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(a.rows) * sh.cluster),
                            dim3(kSampleThreads), sh.smem, s, sh.cluster, a);
}
// A call without top-k, top-p and min-p has a kernel without them: what they
// need of registers costs every row, whether it has filters or not.
template <typename T, bool VERIFY>
static cudaError_t launch_rows(const SampleArgs& a, int sms, cudaStream_t s) {
  return a.top_k || a.top_p || a.min_p ? launch_rows<T, VERIFY, true>(a, sms, s)
                                       : launch_rows<T, VERIFY, false>(a, sms, s);
}

template <typename T>
static cudaError_t launch_verify(VerifyArgs v, cudaStream_t s) {
  // greedy drafts: nothing is left to add up
  v.cluster = v.draft_logits ? kMostCluster : 1;
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const size_t smem =
      v.draft_logits ? static_cast<size_t>((v.V + 2 * (E - 1)) / E + v.cluster - 1) / v.cluster * E * 4 : 0;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        verify_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostShared));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl_cluster(verify_kernel<T>, dim3(static_cast<unsigned>(v.B) * v.cluster),
                            dim3(kSampleThreads), smem, s, v.cluster, v);
}

static cudaError_t sm_count(int& sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}

static bool logits_ok(const void* p, int64_t stride, int32_t vocab, int32_t dtype) {
  if (dtype != PE_DTYPE_BF16 && dtype != PE_DTYPE_F32) return false;
  const int elem = dtype == PE_DTYPE_F32 ? 4 : 2;
  return p && reinterpret_cast<uintptr_t>(p) % elem == 0 && stride >= vocab;
}
static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// Vectors of 32-bit numbers, those that are not given (NULL) among them.
template <typename... P>
static bool aligned4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) % 4 == 0) && ...);
}

}  // namespace pe

extern "C" pe_status pe_sample(int32_t rows, int32_t vocab, int32_t dtype, const void* logits,
                               int64_t stride, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, const float* u,
                               int32_t* tokens, float* logprobs, pe_dist* dist, void* stream) {
  using namespace pe;
  if (rows < 1 || vocab < 1 || !logits_ok(logits, stride, vocab, dtype) || !u || !tokens ||
      !aligned4(temperature, top_k, top_p, min_p, u, tokens, logprobs) || !aligned16(dist))
    return PE_ERR_INVALID_ARGUMENT;
  if (vocab > kMostVocab || rows > (1 << 27)) return PE_ERR_UNSUPPORTED;
  SampleArgs a = {};
  a.rows = rows;
  a.V = vocab;
  a.logits = logits;
  a.stride = stride;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.dist = dist;
  int sms = 0;
  cudaError_t e = sm_count(sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = dtype == PE_DTYPE_F32 ? launch_rows<float, false>(a, sms, s)
                              : launch_rows<bf16, false>(a, sms, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

extern "C" pe_status pe_verify(int32_t B, int32_t T, int32_t vocab, int32_t dtype,
                               const void* logits, int64_t stride, const int32_t* ids,
                               const int32_t* cu_in, const float* temperature,
                               const int32_t* top_k, const float* top_p, const float* min_p,
                               const float* accept_u, const float* u, const void* draft_logits,
                               int64_t draft_stride, const pe_dist* draft_dist,
                               int32_t* num_accepted, int32_t* sampled_ids, float* logprobs,
                               pe_dist* dist, int32_t* err, void* stream) {
  using namespace pe;
  if (B < 1 || T < B || vocab < 1 || !logits_ok(logits, stride, vocab, dtype) || !ids || !cu_in ||
      !accept_u || !u || !num_accepted || !sampled_ids || !dist || !aligned16(dist) ||
      !aligned4(ids, cu_in, temperature, top_k, top_p, min_p, accept_u, u, num_accepted,
                sampled_ids, logprobs, err))
    return PE_ERR_INVALID_ARGUMENT;
  if (draft_logits && T > B &&
      (!logits_ok(draft_logits, draft_stride, vocab, dtype) || !draft_dist ||
       !aligned16(draft_dist)))
    return PE_ERR_INVALID_ARGUMENT;
  if (vocab > kMostVocab || T > (1 << 27)) return PE_ERR_UNSUPPORTED;
  SampleArgs a = {};
  a.rows = T;
  a.V = vocab;
  a.logits = logits;
  a.stride = stride;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.dist = dist;
  a.B = B;
  a.cu_in = cu_in;
  a.ids = ids;
  a.greedy_drafts = draft_logits == nullptr;
  VerifyArgs v = {};
  v.B = B;
  v.T = T;
  v.V = vocab;
  v.logits = logits;
  v.stride = stride;
  v.ids = ids;
  v.cu_in = cu_in;
  v.accept_u = accept_u;
  v.u = u;
  v.draft_logits = draft_logits;
  v.draft_stride = draft_stride;
  v.draft_dist = draft_dist;
  v.num_accepted = num_accepted;
  v.sampled_ids = sampled_ids;
  v.logprobs = logprobs;
  v.dist = dist;
  v.err = err;
  int sms = 0;
  cudaError_t e = sm_count(sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = dtype == PE_DTYPE_F32;
  if (e == cudaSuccess)
    e = f32 ? launch_rows<float, true>(a, sms, s) : launch_rows<bf16, true>(a, sms, s);
  if (e == cudaSuccess) {
    e = f32 ? launch_verify<float>(v, s) : launch_verify<bf16>(v, s);
  }
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
