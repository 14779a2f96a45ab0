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

constexpr int kSampleThreads = 512;
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
// NaN counts as -inf, +inf as the largest finite number, -0 as 0 (which gives
// equal logits one sort key).
__device__ __forceinline__ float clean_logit(float x) {
  return fminf(fmaxf(x, -INFINITY), 3.402823466e38f) + 0.f;
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

struct Exchange {
  unsigned long long warp[2][kSampleWarps];
  unsigned long long slot[2][2][kMostCluster];  // [parity][value][CTA]
};

// Two 64-bit sums (or a maximum and a sum) over the cluster; every thread gets
// them.  The CTAs' own first sums stay in ex.slot[parity][0].  One barrier:
// the slots of the round before the last are free, because whoever has passed
// the last barrier has read them.
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
  if (warp == 0) {
    unsigned long long x = lane < kSampleWarps ? ex.warp[0][lane] : 0;
    unsigned long long y = lane < kSampleWarps ? ex.warp[1][lane] : 0;
    x = MAX ? warp_max_u64(x) : warp_sum_u64(x);
    y = warp_sum_u64(y);
    if (lane < cluster) {
      st_cluster_u64(cluster_map_shared(smem_u32(&ex.slot[parity][0][rank]), lane), x);
      st_cluster_u64(cluster_map_shared(smem_u32(&ex.slot[parity][1][rank]), lane), y);
    }
  }
  cluster_sync_all();
  a = b = 0;
  for (int r = 0; r < cluster; ++r) {
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
  int first;   // id of the first chunk's first element (may be negative)
  int chunks;  // of this CTA
};
template <typename T>
__device__ __forceinline__ Part<T> part_of(const T* row, int V, int cluster, int rank) {
  constexpr int E = Part<T>::E;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) % E);
  const int all = (mis + V + E - 1) / E, per = (all + cluster - 1) / cluster;
  const int lo = min(rank * per, all);
  return Part<T>{lo * E - mis, min(lo + per, all) - lo};
}
template <typename T>
__device__ __forceinline__ uint4 load_chunk(const T* row, int V, int id) {
  constexpr int E = Part<T>::E;
  if (id >= 0 && id + E <= V) return __ldg(reinterpret_cast<const uint4*>(row + id));
  uint4 v;
  T* t = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = id + e >= 0 && id + e < V ? row[id + e] : from_f<T>(-INFINITY);
  return v;
}

// The token at which the kept weights, in the order of the ids, first exceed
// `at`; weight(chunk, e) of this CTA's elements.  Every warp has a contiguous
// segment of chunks.  Returns the id on one thread of the cluster, -1 on all
// others.
struct Segment {
  int lo, hi;
};
__device__ __forceinline__ Segment warp_segment(int chunks) {
  const int per = ((chunks + 31) / 32 + kSampleWarps - 1) / kSampleWarps * 32;
  const int lo = min(static_cast<int>(threadIdx.x) / 32 * per, chunks);
  return Segment{lo, min(lo + per, chunks)};
}
template <int E, typename W>
__device__ __forceinline__ int find_in_segment(Segment seg, long long at, int first, W&& weight) {
  const int lane = threadIdx.x % 32;
  for (int c0 = seg.lo; c0 < seg.hi; c0 += 32) {
    const int c = c0 + lane;
    unsigned long long own = 0;
    if (c < seg.hi)
#pragma unroll
      for (int e = 0; e < E; ++e) own += weight(c, e);
    unsigned long long run = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, run, d);
      if (lane >= d) run += o;
    }
    const long long all = static_cast<long long>(__shfl_sync(0xffffffffu, run, 31));
    if (at >= all) {
      at -= all;
      continue;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, static_cast<long long>(run) > at);
    if (lane != __ffs(hit) - 1) return -1;
    at -= static_cast<long long>(run - own);
    for (int e = 0; e < E; ++e) {
      const long long w = weight(c, e);
      if (at < w) return first + c * E + e;
      at -= w;
    }
    return -1;  // not reached: the sums agree
  }
  return -1;
}

// ------------------------------------------------------------- sampling rows
template <typename T, bool VERIFY>
__global__ void __launch_bounds__(kSampleThreads) sample_rows_kernel(
    const __grid_constant__ SampleArgs a) {
  extern __shared__ __align__(16) unsigned char held[];
  __shared__ Exchange ex;
  __shared__ unsigned long long warp_mass[kSampleWarps];
  constexpr int E = Part<T>::E;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cluster = a.cluster, rank = cluster_ctarank(), r = blockIdx.x / cluster;
  int parity = 0;
  grid_dep_wait();
  grid_dep_launch();

  // the row's request, its filters, and the draft that it judges
  int q = r, draft = -1;
  bool judges = false;
  if (VERIFY) {
    int lo = 0, hi = a.B;  // the last request whose window starts at or before r
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu_in[mid] <= r) lo = mid;
      else hi = mid;
    }
    q = lo;
    const int w0 = a.cu_in[q], w1 = a.cu_in[q + 1];
    if (w0 < 0 || w0 > r || w1 <= r || w1 > a.rows) return;  // the whole cluster
    judges = r + 1 < w1;
    draft = judges ? a.ids[r + 1] : -1;
  }
  const float temp = a.temperature ? a.temperature[q] : 1.f;
  float inv = __fdiv_rn(1.f, temp);
  const bool greedy = !(temp > 0.f) || isinf(inv);
  if (greedy) inv = 0.f;
  int k = a.top_k ? a.top_k[q] : 0;
  if (k <= 0) k = a.V;
  const float p = a.top_p ? a.top_p[q] : 1.f;
  if (greedy || p <= 0.f) k = 1;  // top-p of nothing: the first token alone
  const bool by_mass = p < 1.f && p > 0.f;
  const float mp = a.min_p ? fminf(a.min_p[q], 1.f) : 0.f;  // NaN: 1, see below
  const float min_p = a.min_p && isnan(a.min_p[q]) ? 0.f : mp;

  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  const Part<T> part = part_of(row, a.V, cluster, rank);
  uint4* mine = reinterpret_cast<uint4*>(held);
  float top = -INFINITY;
  for (int c = tid; c < part.chunks; c += kSampleThreads) {
    const uint4 v = load_chunk(row, a.V, part.first + c * E);
    mine[c] = v;
    const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int e = 0; e < E; ++e) top = fmaxf(top, clean_logit(to_f<T>(t[e])));
  }
  unsigned long long x = float_order_key(top), y = 0;
  cluster_reduce<true>(ex, parity, cluster, rank, x, y);
  const RowScale sc = {key_float(static_cast<uint32_t>(x)), inv};
  const T* elems = reinterpret_cast<const T*>(held);

  // counts and sums of the tokens that a test takes
  auto sums = [&](auto&& test, unsigned long long& count, unsigned long long& mass) {
    count = mass = 0;
    for (int c = tid; c < part.chunks; c += kSampleThreads)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = raw_logit(elems + c * E + e);
        const float ev = exp_of(v, sc);
        const uint32_t w = weight_of(ev);
        if (w && test(v, ev, part.first + c * E + e)) {
          ++count;
          mass += w;
        }
      }
    cluster_reduce<false>(ex, parity, cluster, rank, count, mass);
  };
  unsigned long long positive, able, mass, count;
  sums([&](float, float, int) { return true; }, positive, mass);
  sums([&](float, float ev, int) { return ev >= min_p; }, able, mass);
  // Tokens in their order are falling 64-bit keys.  The last one of which
  // fewer than `limit` (tokens, or weight) come before:
  unsigned long long border = 0;
  const unsigned long long most = argmax_key(sc.max, 0);
  auto bisect = [&](bool by_count, double limit) {
    const unsigned long long floor_key = border;
    unsigned long long lo = 0, hi = most;
    while (lo < hi) {
      const unsigned long long mid = lo + (hi - lo) / 2;
      sums([&](float v, float ev, int id) {
        const unsigned long long key = argmax_key(v, id);
        return ev >= min_p && key >= floor_key && key > mid;
      }, count, mass);
      if (static_cast<double>(by_count ? count : mass) < limit) hi = mid;
      else lo = mid + 1;
    }
    border = hi;
  };
  const unsigned long long first_n = min(static_cast<unsigned long long>(k), able);
  if (positive) {
    const unsigned long long able_mass = mass;
    if (first_n < positive) bisect(true, static_cast<double>(first_n));
    if (by_mass) {
      mass = able_mass;
      if (border)
        sums([&](float v, float ev, int id) { return ev >= min_p && argmax_key(v, id) >= border; },
             count, mass);
      bisect(false, static_cast<double>(p) * static_cast<double>(mass));
      sums([&](float v, float ev, int id) { return argmax_key(v, id) >= border; }, count, mass);
      if (count == positive) border = 0;
    }
  }
  const float cut = border ? key_float(static_cast<uint32_t>(border >> 32)) : -INFINITY;
  const int cut_token = border ? argmax_key_index(border) : a.V - 1;

  // Draw.  A greedy draft that this row may reject has no share.
  const int left_out = VERIFY && a.greedy_drafts && draft >= 0 && draft < a.V ? draft : -1;
  auto weight = [&](int c, int e) -> uint32_t {
    const float v = raw_logit(elems + c * E + e);
    const int id = part.first + c * E + e;
    if (!is_kept(v, id, cut, cut_token) || id == left_out) return 0;
    return weight_of(exp_of(v, sc));
  };
  const Segment seg = warp_segment(part.chunks);
  unsigned long long own = 0;
  for (int c = seg.lo + lane; c < seg.hi; c += 32)
#pragma unroll
    for (int e = 0; e < E; ++e) own += weight(c, e);
  unsigned long long total = own, none = 0;
  own = warp_sum_u64(own);
  if (lane == 0) warp_mass[warp] = own;
  const int par = parity;
  cluster_reduce<false>(ex, parity, cluster, rank, total, none);
  long long all = static_cast<long long>(total);
  if (left_out >= 0) {
    const float v = raw_logit(row + left_out);
    if (is_kept(v, left_out, cut, cut_token)) all += weight_of(exp_of(v, sc));
  }
  const bool draws = total > 0 && !(VERIFY && judges && !a.greedy_drafts);
  int token = -1;
  if (draws) {
    long long at = place_of(a.u[q], static_cast<long long>(total));
    for (int i = 0; i < rank; ++i) at -= static_cast<long long>(ex.slot[par][0][i]);
    for (int i = 0; i < warp; ++i) at -= static_cast<long long>(warp_mass[i]);
    if (at >= 0 && at < static_cast<long long>(own))
      token = find_in_segment<E>(seg, at, part.first, weight);
  }
  if (token >= 0 || (!draws && rank == 0 && tid == 0)) {
    if (!VERIFY) {
      a.tokens[r] = token;
      if (a.logprobs)
        a.logprobs[r] = token >= 0 ? logprob_of(raw_logit(row + token), sc, all) : -INFINITY;
    }
    if (a.dist) {
      uint4* d = reinterpret_cast<uint4*>(a.dist + r);
      d[0] = make_uint4(__float_as_uint(sc.max), __float_as_uint(inv), __float_as_uint(cut),
                        static_cast<uint32_t>(cut_token));
      d[1] = make_uint4(static_cast<uint32_t>(all), static_cast<uint32_t>(all >> 32),
                        static_cast<uint32_t>(token), 0u);
    }
  }
}

// -------------------------------------------------------------- verification
// The weight of a token in a row that a record describes.
template <typename T>
__device__ __forceinline__ uint32_t dist_weight(float x, int id, const pe_dist& d) {
  if (!is_kept(x, id, d.cut, d.cut_token)) return 0;
  return weight_of(exp_of(x, RowScale{d.max, d.inv}));
}

// A cluster a request: its first rejected draft, and the token drawn there.
template <typename T>
__global__ void __launch_bounds__(kSampleThreads) verify_kernel(
    const __grid_constant__ VerifyArgs a) {
  __shared__ Exchange ex;
  __shared__ unsigned long long warp_mass[2][kSampleWarps];
  constexpr int E = Part<T>::E;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int cluster = a.cluster, rank = cluster_ctarank(), r = blockIdx.x / cluster;
  int parity = 0;
  grid_dep_wait();
  grid_dep_launch();
  const int w0 = a.cu_in[r], w1 = a.cu_in[r + 1], drafts = a.T - a.B;
  if (w0 < 0 || w1 <= w0 || w1 > a.T) {
    if (rank == 0 && tid == 0) {
      record_error(a.err, PE_DEV_BAD_ROW);
      a.num_accepted[r] = 0;
      a.sampled_ids[r] = -1;
    }
    return;  // the whole cluster
  }
  const T* logits = static_cast<const T*>(a.logits);
  const T* draft_logits = static_cast<const T*>(a.draft_logits);
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
      if (d < 0 || d >= a.V) {
        if (rank == 0 && warp == 0) record_error(a.err, PE_DEV_BAD_TOKEN);
      } else {
        w = dist_weight<T>(raw_logit(logits + t * a.stride + d), d, P);
        if (draft_logits && from >= 0 && from < drafts) {
          const pe_dist Q = a.draft_dist[from];
          wq = dist_weight<T>(raw_logit(draft_logits + from * a.draft_stride + d), d, Q);
          totalq = Q.total;
        }
      }
      const double u = a.accept_u[t];
      if (draft_logits)
        ok = u * static_cast<double>(wq) * static_cast<double>(P.total) <
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
  if (draft_logits && stop < w1 - 1 && P.total > 0 && from >= 0 && from < drafts) {
    // rejected: from what the target has more of than the drafter
    const pe_dist Q = a.draft_dist[from];
    const T* qrow = draft_logits + from * a.draft_stride;
    const float ap = static_cast<float>(2147483648.0 / static_cast<double>(P.total));
    const float aq =
        Q.total > 0 ? static_cast<float>(2147483648.0 / static_cast<double>(Q.total)) : 0.f;
    const Part<T> part = part_of(row, a.V, cluster, rank);
    auto weights = [&](int c, int e, uint32_t& more, uint32_t& plain) {
      const int id = part.first + c * E + e;
      more = plain = 0;
      if (id < 0 || id >= a.V) return;
      const float pw = __fmul_rn(
          static_cast<float>(dist_weight<T>(raw_logit(row + id), id, P)), ap);
      const float qw = __fmul_rn(
          static_cast<float>(dist_weight<T>(raw_logit(qrow + id), id, Q)), aq);
      plain = __float2uint_rn(pw);
      more = __float2uint_rn(fmaxf(__fsub_rn(pw, qw), 0.f));
    };
    const Segment seg = warp_segment(part.chunks);
    unsigned long long more = 0, plain = 0;
    for (int c = seg.lo + lane; c < seg.hi; c += 32)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint32_t m, n;
        weights(c, e, m, n);
        more += m;
        plain += n;
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
      token = find_in_segment<E>(seg, at, part.first, [&](int c, int e) {
        uint32_t m, n;
        weights(c, e, m, n);
        return use ? n : m;
      });
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
struct SampleShape {
  int cluster;
  size_t smem;
};
// Few rows: as many CTAs a row as a cluster has, for the shortest way; more
// rows than that fills: as few as hold the row.
static SampleShape sample_shape(int rows, int V, int elem, int sms) {
  constexpr size_t kHalf = 100 * 1024;
  auto bytes = [&](int c) {
    const int e = 16 / elem, all = (V + 2 * (e - 1)) / e;
    return static_cast<size_t>((all + c - 1) / c) * 16;
  };
  int c = 1;
  while (c < kMostCluster && bytes(c) > kHalf) c *= 2;
  while (c < kMostCluster && static_cast<long long>(rows) * c * 2 <= 2 * sms &&
         bytes(c) > 4096)
    c *= 2;
  return SampleShape{c, bytes(c)};
}

template <typename T, bool VERIFY>
static cudaError_t launch_rows(SampleArgs a, int sms, cudaStream_t s) {
  const SampleShape sh = sample_shape(a.rows, a.V, sizeof(T), sms);
  a.cluster = sh.cluster;
  auto kernel = sample_rows_kernel<T, VERIFY>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sh.smem));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(a.rows) * sh.cluster),
                            dim3(kSampleThreads), sh.smem, s, sh.cluster, a);
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

}  // namespace pe

extern "C" pe_status pe_sample(int32_t rows, int32_t vocab, int32_t dtype, const void* logits,
                               int64_t stride, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, const float* u,
                               int32_t* tokens, float* logprobs, pe_dist* dist, void* stream) {
  using namespace pe;
  if (rows < 1 || vocab < 1 || !logits_ok(logits, stride, vocab, dtype) || !u || !tokens ||
      !aligned16(dist))
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
      !accept_u || !u || !num_accepted || !sampled_ids || !dist || !aligned16(dist))
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
    // greedy drafts: nothing is left to add up
    v.cluster = draft_logits ? kMostCluster : 1;
    const dim3 grid(static_cast<unsigned>(B) * v.cluster);
    e = f32 ? launch_pdl_cluster(verify_kernel<float>, grid, dim3(kSampleThreads), 0, s, v.cluster, v)
            : launch_pdl_cluster(verify_kernel<bf16>, grid, dim3(kSampleThreads), 0, s, v.cluster, v);
  }
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
