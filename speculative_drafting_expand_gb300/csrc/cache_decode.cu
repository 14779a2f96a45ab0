// cache_decode.cu -- attention of one new token per request over a paged KV
// cache (include/peagle_cache.h):
//   out = sum_j p_j v_j,  p_j = exp(z_j - lse),  z_j = scale q.k_j,
//   lse = ln sum_j exp(z_j),
// and, where asked, each position's weight summed over the query heads of its
// kv head.
//
// One pass over K and V with a running maximum m and sum l (a new maximum
// scales what was summed by 2^(m_old - m_new); logits are kept in units of
// ln 2).  Bound by the bytes of K and V: a page row is used once per query
// head of its group, 2 flops a byte and head.
//
// Work.  The unit is one page (16 positions) of one kv head; an item is the
// run of pages of one (request, kv head, tile of query heads), and the items
// lie one after another on a line that the CTAs cut into equal pieces, and
// their warps those: every warp gets the same number of pages whatever the
// lengths are.  An item that lies in one warp's piece is finished there.
// Otherwise its parts (m, l, sum of p v) are joined: the warps' of one CTA
// through shared memory, the CTAs' by a second launch (attn_join_kernel)
// that starts as the first drains.  Joins run in the order of the positions:
// results do not depend on timing.
//
// Tiles.  A warp owns its pages alone: its lanes copy them into a ring of
// shared memory with 16-byte asynchronous copies, each lane (almost) only
// what it reads itself, so no barrier stands between copy and use.  For 16-
// and 8-bit pools S = Q K^T and O += P V are m16n8k16 matrix instructions of
// the warp: M the query heads of the group (8 used, or 16), N positions or
// elements.  A tcgen05 tile would hold 128 query rows where a group has 8;
// the warp instruction needs no staging through tensor memory, and at two
// bytes an element and 8 heads it is far from its rate.  The orders of the
// elements along k and of the positions are free as long as both operands
// share them: they are chosen such that every lane's operand is 16 contiguous
// bytes of a row.  P enters as two 16-bit numbers (value and remainder, which
// leave 2^-17 of it; fp16: 2^-22, or 2^-37 of the largest weight); with 8
// heads the remainders are the otherwise unused rows 8..15.  e4m3 pools go
// through fp16, which holds every code; q is scaled there by a power of two so
// that its largest element is in [1, 2) and fp16's range does not matter
// (elements below 2^-24 of that vanish).
//
// Measured (GB300, launches alone; 64 query heads on 8 kv heads of 64): 64
// requests of 372575 positions in all, bf16, 130 us, 5.9 TB/s of K and V (a
// copy: 6.8); 265096 positions, e4m3, with scores, 88 us, where the
// instructions of a page (half of it conversions and their shifts) bound it;
// one request of 4096 positions 9.9 us, the way from length to page ids to K
// and V to the join, and two launches.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "cache_common.cuh"
#include "pe_kernels.h"

namespace pe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLift = 4096.f;  // of weights beside e4m3 pools, see MmaTile
constexpr int kMaxWarps = 8;  // warps a CTA
constexpr int kMostCtas = 512;  // so that the join of an item over all of them fits
// Pages a warp, where there are fewer than the grid could take (one request of
// 4096: 10.3 us with 2, 11.3 with 1, 10.4 with 4; of 68: 9.3, 9.6, 13.4).
constexpr int kMinPages = 2;

// ------------------------------------------------------------------ shapes

template <int DT, int DH, int GT>
struct DecodeShape {
  static constexpr int EB = DT == PE_KV_F32 ? 4 : DT == PE_KV_BF16 ? 2 : 1;
  static constexpr int ROWB = DH * EB;
  static constexpr int PAGEB = kPage * ROWB;       // a page of one head of K or V
  static constexpr int CH = PAGEB / 512;           // 16-byte chunks a lane copies of it
  // query heads a tile: the rows of the matrix instruction that are used, or
  // what the registers of the fp32 path hold
  static constexpr int ROWS = DT == PE_KV_F32 ? (DH == 64 ? 8 : 4) : 8 * GT;
  static constexpr int WARPS = DT == PE_KV_F32 && DH == 128 ? 4 : 8;
  // pages at a time, for longer independent chains (one instead of two: e4m3
  // 158 against 153 us before the other steps, bf16 the same; four: no better)
  static constexpr int TAKE = DT == PE_KV_F32 ? 1 : 2;
  static constexpr int STAGES =  // pages in the ring
      DT == PE_KV_F32 ? 3 : PAGEB == 4096 ? 3 : 6;
  static constexpr int RING = STAGES * 2 * PAGEB;  // a warp's ring
  static constexpr int REC = ROWS * (DH + 2);      // a partial result, floats: m, l, O
  static constexpr int SCRATCH = DT == PE_KV_F32 ? (ROWS * DH + kPage * ROWS + ROWS) * 4 : 0;
  static constexpr int SMEM = WARPS * (RING + SCRATCH);
  // CTAs a SM: one of 8 warps with all the registers, or for the short e4m3
  // pages two (batch 64, bf16: 130 us with one, 135 with two and half the
  // stages; e4m3 with scores: 93.5 with one, 88.5 with two)
  static constexpr int CTAS = DT == PE_KV_E4M3 && DH == 64 ? 2 : 1;
  // the scores' kernel: K alone, two CTAs an SM
  static constexpr int S_TAKE = DT == PE_KV_F32 ? 1 : 2;
  static constexpr int S_STAGES = PAGEB == 1024 ? 8 : PAGEB == 2048 ? 6 : 3;
  static constexpr int S_RING = S_STAGES * PAGEB;
  static constexpr int S_SMEM = WARPS * (S_RING + SCRATCH);
  static_assert(REC * 4 <= S_RING, "the same without values");
  static_assert(REC * 4 <= RING, "a warp leaves its last partial in its ring");
};

struct DecodeArgs {
  CachePool pool;
  int B, Hq, Hkv, G, bt_stride, window;
  int tiles;       // tiles of query heads a kv head
  float scale;     // of the logits, with ln 2 and the K scale divided in
  float v_scale;   // divided by the lift of the weights
  const void* q;
  long long q_stride, out_stride;
  const int32_t* block_table;
  const int32_t* seq_lens;
  void* out;
  float* lse;      // caller's, or NULL
  int* err;
  // drafting step: request b's query is row q_rows[b * q_rows_stride] of
  // q_limit, and it attends seq_lens[b] + len_add positions; else NULL and 0
  const int32_t* q_rows;
  int q_rows_stride, q_limit, len_add;
  // workspace
  float* stash;    // logits of the line's first stash_pages pages, as the
                   // lanes hold them
  int stash_pages;
  float* lse_w;    // [B, Hq], in units of ln 2
  int4* meta;      // [grid]: item and flags of the CTA's first and last partial
  float* part;     // [grid][2][REC]
  float* head;     // [grid * WARPS][REC]
};

// A request's positions and pages: lo..n-1 attended, pages pf..pe-1.
struct Span {
  int n, lo, pf, pe;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b, bool record) {
  const long long cap = static_cast<long long>(a.bt_stride) * kPage;
  Span s;
  s.n = a.seq_lens[b] + a.len_add;
  if (a.q_rows &&
      static_cast<uint32_t>(a.q_rows[static_cast<size_t>(b) * a.q_rows_stride]) >=
          static_cast<uint32_t>(a.q_limit))
    s.n = 0;  // a bad row, recorded where it was made
  if (s.n < 0 || s.n > cap) {
    if (record) record_error(a.err, PE_DEV_BAD_POSITION);
    s.n = s.n < 0 ? 0 : static_cast<int>(cap);
  }
  s.lo = a.window > 0 ? max(0, s.n - a.window) : 0;
  s.pf = s.lo / kPage;
  s.pe = s.n > s.lo ? (s.n - 1) / kPage + 1 : s.pf;
  return s;
}

// Element 0 of request b's query.
template <typename A>
__device__ __forceinline__ const A* query_of(const DecodeArgs& a, int b) {
  const int row = a.q_rows ? a.q_rows[static_cast<size_t>(b) * a.q_rows_stride] : b;
  return static_cast<const A*>(a.q) + static_cast<size_t>(row) * a.q_stride;
}

// The line of pages: where unit u lies.  Every thread sums the pages of an
// equal share of the requests; the shares' prefix sums stay in shared memory
// and a warp searches them, then its share.  (The host refuses calls whose
// tables could hold 2^31 pages.)
struct Line {
  int total;  // units
  int per;    // requests a share
};
template <int THREADS>
__device__ __forceinline__ Line line_setup(const DecodeArgs& a, int heads, int* prefix) {
  __shared__ int warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  Line ln;
  ln.per = (a.B + THREADS - 1) / THREADS;
  int mine = 0;
  for (int i = 0; i < ln.per; ++i) {
    const int b = tid * ln.per + i;
    if (b < a.B) {
      const Span s = span_of(a, b, false);
      mine += s.pe - s.pf;
    }
  }
  mine *= heads;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[tid >> 5] = x;
  __syncthreads();
  int base = 0;
  ln.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int c = warp_sum[w];
    base += w < (tid >> 5) ? c : 0;
    ln.total += c;
  }
  prefix[tid] = base + x - mine;
  __syncthreads();
  return ln;
}

// Part i of `total` pages in n equal parts, the first ones a page longer
// (i >= n: nothing).
struct Share {
  int first, count;
};
__device__ __forceinline__ Share share_of(int total, int n, int i) {
  const int per = static_cast<uint32_t>(total) / static_cast<uint32_t>(n), rest = total - per * n;
  if (i >= n) return Share{0, 0};
  return Share{per * i + min(i, rest), per + (i < rest ? 1 : 0)};
}

// A place on the line: page p of head tile hh of request b.
struct Place {
  int b, hh;
  Span s;
  int p;
};
template <int THREADS>
__device__ __forceinline__ Place place_of(const DecodeArgs& a, const Line& ln, int heads,
                                          const int* prefix, int u) {
  int lo = 0, hi = min(a.B, THREADS) - 1;  // last share with prefix <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Place pl;
  int left = u - prefix[lo];
  pl.b = lo * ln.per;
  pl.s = span_of(a, pl.b, false);
  while (left >= (pl.s.pe - pl.s.pf) * heads) {
    left -= (pl.s.pe - pl.s.pf) * heads;
    pl.s = span_of(a, ++pl.b, false);
  }
  const uint32_t np = pl.s.pe - pl.s.pf;
  pl.hh = static_cast<uint32_t>(left) / np;
  pl.p = pl.s.pf + (left - pl.hh * static_cast<int>(np));
  return pl;
}
// The first page of the next item (there is one).
__device__ __forceinline__ void next_item(const DecodeArgs& a, int heads, Place& pl) {
  if (++pl.hh == heads) {
    pl.hh = 0;
    do pl.s = span_of(a, ++pl.b, false);
    while (pl.s.pe == pl.s.pf);
  }
  pl.p = pl.s.pf;
}

// ------------------------------------------------------------------ copies

// 16 bytes, or the first `bytes` of them and zeros; with an L2 policy.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes,
                                           uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(bytes), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}
// K and V pass through L2 once.  With logits to keep there (written by this
// kernel, read by the last) they are the first to leave it: batch 64, e4m3,
// with scores 91 -> 85 us, batch 16 66 -> 60; without, small caches that a
// program reads again soon may stay.  Made once, by whole warps (volatile: not
// again at a copy that some lanes skip), and the same in every lane.
__device__ __forceinline__ uint64_t kv_policy(bool first_to_leave) {
  uint64_t normal;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  const uint64_t first = l2_policy_evict_first();
  return first_to_leave ? first : normal;
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Lane (g = lane / 4, t = lane % 4) reads, of K, chunks t + 4 i of rows
// key_of(j, g), j = 0, 1, and of V chunks g + 8 i of rows t + 4 i'.  key_of()
// is the order of the positions along the logits' columns: column n of half
// j.  A page lies in the ring in its own order, but for the 16-byte chunks of
// a row, whose places are exchanged such that the eight lanes that read
// together meet all banks.
__device__ __forceinline__ int key_of(int j, int n) { return 8 * j + (n >> 1) + 4 * (n & 1); }

template <class SH>
__device__ __forceinline__ uint32_t k_place(int r, int c) {
  // rows of 64 bytes: two to the 128 bytes of all banks
  if constexpr (SH::ROWB == 64) return static_cast<uint32_t>(((r * 4 + c) ^ (r & 4)) * 16);
  else return static_cast<uint32_t>(r * SH::ROWB + (c ^ (r & 4)) * 16);
}
template <class SH>
__device__ __forceinline__ uint32_t v_place(int r, int c) {
  if constexpr (SH::ROWB == 64) return static_cast<uint32_t>(r * 64 + (c ^ (r & 2)) * 16);
  else return static_cast<uint32_t>(r * SH::ROWB + (c ^ ((r & 3) << 1)) * 16);
}

// 32 lanes copy 512 bytes in a row at a time.  Positions v_lo <= offset < v_hi
// of the page are attended; the others read as zeros whatever lies there.
template <class SH, bool WITH_V>
__device__ __forceinline__ void copy_page(uint32_t stage, const CachePool& pool, size_t page,
                                          int v_lo, int v_hi, uint64_t policy, int lane) {
  constexpr int CPR = SH::ROWB / 16;  // chunks a row
  const size_t base = page * SH::PAGEB + lane * 16;
  const char* kp = static_cast<const char*>(pool.k) + base;
  const char* vp = static_cast<const char*>(pool.v) + base;
  const bool whole = v_lo <= 0 && v_hi >= kPage;
#pragma unroll
  for (int i = 0; i < SH::CH; ++i) {
    const int r = (i * 32 + lane) / CPR, c = lane % CPR;
    const uint32_t k_at = stage + k_place<SH>(r, c);
    const uint32_t v_at = stage + SH::PAGEB + v_place<SH>(r, c);
    if (whole) {
      cp_async16(k_at, kp + i * 512, policy);
      if (WITH_V) cp_async16(v_at, vp + i * 512, policy);
    } else {
      const uint32_t n = r >= v_lo && r < v_hi ? 16u : 0u;
      cp_async16(k_at, kp + i * 512, n, policy);
      if (WITH_V) cp_async16(v_at, vp + i * 512, n, policy);
    }
  }
}

// The copying side of a warp: pages of the line in order, a commit each.
template <class SH, bool WITH_V>
struct Feeder {
  static constexpr int STAGES = WITH_V ? SH::STAGES : SH::S_STAGES;
  static constexpr int STRIDE = WITH_V ? 2 * SH::PAGEB : SH::PAGEB;
  Place pl;
  int hk;        // kv head of the place
  int left;      // units still to copy
  int ids;       // this lane's page of the 32 from ids_at on
  int ids_at;
  int stage;
  uint32_t bad;  // stages whose page is none
  uint64_t policy;

  __device__ __forceinline__ void start(const DecodeArgs& a, const Place& at, int tiles, int count,
                                        int lane) {
    pl = at;
    hk = pl.hh / tiles;
    left = count;
    stage = 0;
    bad = 0;
    policy = kv_policy(a.stash_pages > 0);
    fetch(a, lane);
  }
  __device__ __forceinline__ void fetch(const DecodeArgs& a, int lane) {
    ids_at = pl.p;
    ids = -1;
    if (pl.p + lane < pl.s.pe)
      ids = a.block_table[static_cast<size_t>(pl.b) * a.bt_stride + pl.p + lane];
  }
  // heads: items a request; tiles: items a kv head
  __device__ __forceinline__ void step(const DecodeArgs& a, int heads, int tiles, uint32_t ring,
                                       int lane, bool record) {
    if (left > 0) {
      if (pl.p == pl.s.pe) {
        next_item(a, heads, pl);
        hk = pl.hh / tiles;
        fetch(a, lane);
      } else if (pl.p - ids_at == 32) {
        fetch(a, lane);
      }
      const int blk = __shfl_sync(0xffffffffu, ids, pl.p - ids_at);
      const int first = pl.p * kPage;
      const uint32_t at = ring + stage * STRIDE;
      if (static_cast<uint32_t>(blk) < static_cast<uint32_t>(a.pool.num_blocks)) {
        bad &= ~(1u << stage);
        copy_page<SH, WITH_V>(at, a.pool, static_cast<size_t>(blk) * a.Hkv + hk, pl.s.lo - first,
                              pl.s.n - first, policy, lane);
      } else {
        if (record && lane == 0) record_error(a.err, PE_DEV_BAD_BLOCK);
        bad |= 1u << stage;
        copy_page<SH, WITH_V>(at, a.pool, 0, kPage, 0, policy, lane);  // zeros
      }
      ++pl.p;
      --left;
    }
    cp_async_commit();
    if (++stage == STAGES) stage = 0;
  }
};

// Writes a row's lse (units of ln 2 in, natural out) and returns what its sum
// of p v is multiplied by; a row without weight gives 0 and -inf.
__device__ __forceinline__ float put_lse(const DecodeArgs& a, int b, int h, float m, float l,
                                         bool write) {
  const bool none = m == -INFINITY && l == 0.f;
  if (write) {
    const float s = none ? -INFINITY : m + log2f(l);
    const size_t at = static_cast<size_t>(b) * a.Hq + h;
    a.lse_w[at] = s;
    if (a.lse) a.lse[at] = s * kLn2;
  }
  return none ? 0.f : a.v_scale / l;
}
template <int DT>
__device__ __forceinline__ void put4(void* out, size_t at, float4 v) {
  if constexpr (DT == PE_KV_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<bf16*>(out) + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// ------------------------------------------------------------ 16 and 8 bits

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == PE_KV_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two weights as a 16-bit pair and the pair of their remainders.
template <int DT>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (DT == PE_KV_BF16) {
    hi = pack_bf16x2(x, y);
    lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
  } else {
    hi = pack_f16x2(x, y);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16x2(x - f.x, y - f.y);
  }
}

// The query heads of a tile as the A operand: for each chunk of 16 bytes of
// a K row (8 or 16 elements), the words that meet its words.
template <int DT, int DH, int GT>
struct QueryTile {
  static constexpr int STEPS = DH / 16;  // k steps of 16 elements
  uint32_t a[GT][STEPS][2];
  float factor[GT];  // logit = sum * factor (units of ln 2); positive

  __device__ __forceinline__ void load(const DecodeArgs& A, int b, int h0, int rows, int lane) {
    const int g = lane >> 2, t = lane & 3;
    // the scale's sign goes to q (and all of it if it is 0), so that the
    // largest sum is the largest logit
    const uint32_t sign = A.scale < 0.f ? 0x80008000u : 0u;
    const float scale = A.scale == 0.f ? 1.f : fabsf(A.scale);
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      const int r = g + 8 * x;
      const bool on = r < rows && A.scale != 0.f;
      const bf16* q = query_of<bf16>(A, b) + static_cast<size_t>(h0 + (on ? r : 0)) * DH;
      factor[x] = scale;
      if constexpr (DT == PE_KV_BF16) {
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          uint4 v = *reinterpret_cast<const uint4*>(q + (t + 4 * i) * 8);
          if (!on) v = make_uint4(sign, sign, sign, sign);
          a[x][2 * i][0] = v.x ^ sign;
          a[x][2 * i][1] = v.y ^ sign;
          a[x][2 * i + 1][0] = v.z ^ sign;
          a[x][2 * i + 1][1] = v.w ^ sign;
        }
      } else {
        uint32_t w[STEPS][2];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < DH / 64; ++i) {
          const uint4* p = reinterpret_cast<const uint4*>(q + (t + 4 * i) * 16);
          const uint4 u = p[0], v = p[1];
          const uint32_t z[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            w[4 * i + e / 2][e & 1] = on ? z[e] ^ sign : 0u;
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(z[e] << 16)),
                                   fabsf(__uint_as_float(z[e] & 0xffff0000u))));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // biased exponent, as far as 2^ex and 2^-ex are both normal numbers: at
        // the ends q lands in [1, 4) or below 2 instead
        const uint32_t ex = min(max(__float_as_uint(top) >> 23, 1u), 253u);
        const float down = __uint_as_float((254 - ex) << 23);
        // neither 0 nor inf, which would make NaN of the masked positions' -inf
        // or of sums of 0
        factor[x] = fminf(fmaxf(factor[x] * __uint_as_float(ex << 23), FLT_MIN), FLT_MAX);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            a[x][s][e] = pack_f16x2(__uint_as_float(w[s][e] << 16) * down,
                                    __uint_as_float(w[s][e] & 0xffff0000u) * down);
      }
    }
  }

  // Sums q.k of a page: z[x][j][e], head g + 8 x, position key_of(j, 2 t + e).
  template <class SH>
  __device__ __forceinline__ void sums(uint32_t stage, int lane, float (&z)[GT][2][2]) const {
    float c[2][4] = {};
    constexpr int KI = SH::CH / 2;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        const uint4 v = lds16(stage + k_place<SH>(key_of(j, lane >> 2), (lane & 3) + 4 * i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (DT == PE_KV_BF16) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
            mma16816<DT>(c[j], a[0][2 * i + s][0], GT > 1 ? a[GT - 1][2 * i + s][0] : 0u,
                         a[0][2 * i + s][1], GT > 1 ? a[GT - 1][2 * i + s][1] : 0u, w[2 * s],
                         w[2 * s + 1]);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma16816<DT>(c[j], a[0][4 * i + s][0], GT > 1 ? a[GT - 1][4 * i + s][0] : 0u,
                         a[0][4 * i + s][1], GT > 1 ? a[GT - 1][4 * i + s][1] : 0u,
                         e4m3x2_to_f16x2(w[s]), e4m3x2_to_f16x2(w[s] >> 16));
        }
      }
#pragma unroll
    for (int x = 0; x < GT; ++x)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) z[x][j][e] = c[j][2 * x + e];
  }
};

template <int DT, int DH, int GT>
struct MmaTile {
  using SH = DecodeShape<DT, DH, GT>;
  static constexpr int NT = DH / 8;  // tiles of 8 elements
  // Weights enter P V as pairs of 16-bit numbers.  fp16 ends at 2^-24, so they
  // enter 2^12 times larger (v_scale has the inverse): one below 2^-25 of the
  // largest would be nothing there, while l counts it in full (31 positions of
  // 2^-26 beside one whose value is 0: an output of 0).  Lifted, what a pair
  // loses is at most 2^-37 of the largest.  2^4 is left below fp16's end for a
  // logit that its own rounding puts above the maximum.  A product a weight
  // (batch 64 with scores: 88.6 -> 88.9 us); a running maximum 12 lower would
  // do the same for nothing, but then l and the maximum cancel in an lse near
  // 0, whose error grows to 2^-21.
  static constexpr float LIFT = DT == PE_KV_E4M3 ? kLift : 1.f;
  QueryTile<DT, DH, GT> q;
  float m[GT], l[GT];                // head g + 8 x; l of this lane's positions
  float o[NT][4];

  __device__ __forceinline__ void start(const DecodeArgs& A, int b, int h0, int rows, char*,
                                        int lane) {
    q.load(A, b, h0, rows, lane);
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  }

  // NP pages in a row, at `stage`; positions v_lo <= i < v_hi of them are
  // attended, and bit n of `none` takes out page n.
  // stash: where the logits of the first stash_n pages go, LOGITS floats a
  // lane and page.
  static constexpr int LOGITS = 4 * GT;
  template <int NP, bool VALUES>
  __device__ __forceinline__ void pages(const uint32_t (&stage)[NP], int v_lo, int v_hi,
                                        uint32_t none, char*, float* stash, int stash_n, int lane) {
    const int t = lane & 3;
    float z[NP][GT][2][2];
#pragma unroll
    for (int n = 0; n < NP; ++n) q.template sums<SH>(stage[n], lane, z[n]);
    if (v_lo > 0 || v_hi < NP * kPage || none) {
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = n * kPage + key_of(j, 2 * t + e);
            if (r < v_lo || r >= v_hi || ((none >> n) & 1))
#pragma unroll
              for (int x = 0; x < GT; ++x) z[n][x][j][e] = -INFINITY;
          }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n)
      if (n < stash_n)
#pragma unroll
        for (int x = 0; x < GT; ++x)
          *reinterpret_cast<float4*>(stash + ((n * GT + x) * 32 + lane) * 4) =
              make_float4(z[n][x][0][0] * q.factor[x], z[n][x][0][1] * q.factor[x],
                          z[n][x][1][0] * q.factor[x], z[n][x][1][1] * q.factor[x]);
    float top[GT];
    bool grow = false;
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      top[x] = -INFINITY;
#pragma unroll
      for (int n = 0; n < NP; ++n)
        top[x] = fmax3(top[x], fmaxf(z[n][x][0][0], z[n][x][0][1]),
                       fmaxf(z[n][x][1][0], z[n][x][1][1]));
      top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
      top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2)) * q.factor[x];
      grow |= top[x] > m[x];
    }
    if (__any_sync(0xffffffffu, grow)) {
      float c[GT];
#pragma unroll
      for (int x = 0; x < GT; ++x) {
        const float mn = fmaxf(m[x], top[x]);
        c[x] = mn == -INFINITY ? 1.f : fast_exp2(m[x] - mn);
        m[x] = mn;
        l[x] *= c[x];
      }
      if (VALUES)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        o[i][0] *= c[0];
        o[i][1] *= c[0];
        o[i][2] *= c[GT - 1];
        o[i][3] *= c[GT - 1];
      }
    }
    uint32_t hi[NP][GT][2], lo[NP][GT][2];
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
      for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p0 = fast_exp2(fmaf(z[n][x][j][0], q.factor[x], -base));
          const float p1 = fast_exp2(fmaf(z[n][x][j][1], q.factor[x], -base));
          l[x] += p0 + p1;
          split2<DT>(p0 * LIFT, p1 * LIFT, hi[n][x][j], lo[n][x][j]);
        }
    }
#pragma unroll
    for (int n = 0; VALUES && n < NP; ++n)
      add_values(stage[n] + SH::PAGEB, hi[n], lo[n], lane);
  }

  // O += P V of a page
  __device__ __forceinline__ void add_values(uint32_t vs, const uint32_t (&hi)[GT][2],
                                             const uint32_t (&lo)[GT][2], int lane) {
    auto pv = [&](float (&c)[4], uint32_t b0, uint32_t b1) {
      if constexpr (GT == 1) {
        mma16816<DT>(c, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
      } else {
        mma16816<DT>(c, hi[0][0], hi[1][0], hi[0][1], hi[1][1], b0, b1);
        mma16816<DT>(c, lo[0][0], lo[1][0], lo[0][1], lo[1][1], b0, b1);
      }
    };
    if constexpr (DT == PE_KV_BF16) {
#pragma unroll
      for (int c = 0; c < DH / 64; ++c) {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 u = lds16(vs + v_place<SH>((lane & 3) + 4 * i, (lane >> 2) + 8 * c));
          w[i][0] = u.x;
          w[i][1] = u.y;
          w[i][2] = u.z;
          w[i][3] = u.w;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          pv(o[8 * c + 2 * k], __byte_perm(w[0][k], w[1][k], 0x5410),
             __byte_perm(w[2][k], w[3][k], 0x5410));
          pv(o[8 * c + 2 * k + 1], __byte_perm(w[0][k], w[1][k], 0x7632),
             __byte_perm(w[2][k], w[3][k], 0x7632));
        }
      }
    } else {
      uint32_t w[4][DH / 32];
      if constexpr (DH == 64) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 u = lds8(vs + v_place<SH>(t + 4 * i, g >> 1) + (g & 1) * 8);
          w[i][0] = u.x;
          w[i][1] = u.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 u = lds16(vs + v_place<SH>((lane & 3) + 4 * i, lane >> 2));
          w[i][0] = u.x;
          w[i][1] = u.y;
          w[i][DH / 32 - 2] = u.z;
          w[i][DH / 32 - 1] = u.w;
        }
      }
#pragma unroll
      for (int k = 0; k < DH / 32; ++k) {
        const uint32_t x0 = __byte_perm(w[0][k], w[1][k], 0x5140);
        const uint32_t x1 = __byte_perm(w[0][k], w[1][k], 0x7362);
        const uint32_t y0 = __byte_perm(w[2][k], w[3][k], 0x5140);
        const uint32_t y1 = __byte_perm(w[2][k], w[3][k], 0x7362);
        pv(o[4 * k], e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(y0));
        pv(o[4 * k + 1], e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(y0 >> 16));
        pv(o[4 * k + 2], e4m3x2_to_f16x2(x1), e4m3x2_to_f16x2(y1));
        pv(o[4 * k + 3], e4m3x2_to_f16x2(x1 >> 16), e4m3x2_to_f16x2(y1 >> 16));
      }
    }
  }

  // Element of the rows that tile i, column n holds: eight tiles hold eight
  // elements in a row.
  static __device__ __forceinline__ int elem(int i, int n) {
    if constexpr (DT == PE_KV_BF16) return (n + 8 * (i >> 3)) * 8 + (i & 7);
    else return n * NT + i;
  }
  __device__ __forceinline__ float value(int x, int i, int e) const {
    return GT == 1 ? o[i][e] + o[i][2 + e] : o[i][2 * x + e];
  }
  __device__ __forceinline__ float sum_l(int x) const {
    float s = l[x] + __shfl_xor_sync(0xffffffffu, l[x], 1);
    return s + __shfl_xor_sync(0xffffffffu, s, 2);
  }

  // The partial result as a record: m[ROWS], l[ROWS], O[ROWS][DH].
  __device__ __forceinline__ void store(float* rec, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      const float s = sum_l(x);
      const int r = g + 8 * x;
      if (t == 0) {
        rec[r] = m[x];
        rec[SH::ROWS + r] = s;
      }
      float* row = rec + 2 * SH::ROWS + r * DH;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < NT; i += 4)
          *reinterpret_cast<float4*>(row + elem(i, 2 * t + e)) =
              make_float4(value(x, i, e), value(x, i + 1, e), value(x, i + 2, e),
                          value(x, i + 3, e));
    }
  }

  // A complete item's result.
  __device__ __forceinline__ void finish(const DecodeArgs& A, int b, int h0, int rows,
                                         int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < GT; ++x) {
      const float s = sum_l(x);
      const int r = g + 8 * x;
      if (r >= rows) continue;
      const float inv = put_lse(A, b, h0 + r, m[x], s, t == 0);
      bf16* row = static_cast<bf16*>(A.out) + static_cast<size_t>(b) * A.out_stride +
                  static_cast<size_t>(h0 + r) * DH;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < NT; i += 8) {
          uint4 v;
          v.x = pack_bf16x2(value(x, i, e) * inv, value(x, i + 1, e) * inv);
          v.y = pack_bf16x2(value(x, i + 2, e) * inv, value(x, i + 3, e) * inv);
          v.z = pack_bf16x2(value(x, i + 4, e) * inv, value(x, i + 5, e) * inv);
          v.w = pack_bf16x2(value(x, i + 6, e) * inv, value(x, i + 7, e) * inv);
          *reinterpret_cast<uint4*>(row + elem(i, 2 * t + e)) = v;
        }
    }
  }
};

// ------------------------------------------------------------------ 32 bits
// No matrix instruction keeps fp32 operands: each lane sums 16 (32) elements
// of two positions for all heads of the tile, four lanes join their sums, and
// the weights go through shared memory to the lanes that hold V.

template <int DH>
struct F32Tile {
  using SH = DecodeShape<PE_KV_F32, DH, 1>;
  static constexpr int R = SH::ROWS;
  static constexpr int C = DH / 32;  // 16-byte chunks of a V row a lane
  float m[R / 4], l[R / 4];          // heads (R / 4) t + x, this lane's positions
  float o[R][C][4];                  // this lane's positions

  // scratch of the warp: q [R][DH], p [16][R], c [R]
  __device__ __forceinline__ void start(const DecodeArgs& A, int b, int h0, int rows, char* scratch,
                                        int lane) {
    float* q = reinterpret_cast<float*>(scratch);
    const float* src = query_of<float>(A, b) + static_cast<size_t>(h0) * DH;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < R * DH / 128; ++i) {
      const int e = (i * 32 + lane) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e < rows * DH) v = *reinterpret_cast<const float4*>(src + e);
      *reinterpret_cast<float4*>(q + e) =
          make_float4(v.x * A.scale, v.y * A.scale, v.z * A.scale, v.w * A.scale);
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < R / 4; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][c][e] = 0.f;
  }

  // z[x][j]: head (R / 4) t + x at position key_of(j, g)
  static __device__ __forceinline__ void logits(uint32_t stage, const char* scratch, int lane,
                                                float (&z)[R / 4][2]) {
    const float* q = reinterpret_cast<const float*>(scratch);
    const int t = lane & 3;
    constexpr int KI = SH::CH / 2;
    float s[R][2] = {};
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      float4 k[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 v = lds16(stage + k_place<SH>(key_of(j, lane >> 2), t + 4 * i));
        k[j] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                           __uint_as_float(v.w));
      }
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float4 qq = *reinterpret_cast<const float4*>(q + h * DH + (t + 4 * i) * 4);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          s[h][j] = fmaf(qq.x, k[j].x, fmaf(qq.y, k[j].y, fmaf(qq.z, k[j].z,
                                                               fmaf(qq.w, k[j].w, s[h][j]))));
      }
    }
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[h][j] += __shfl_xor_sync(0xffffffffu, s[h][j], 1);
        s[h][j] += __shfl_xor_sync(0xffffffffu, s[h][j], 2);
      }
#pragma unroll
    for (int x = 0; x < R / 4; ++x)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = s[x][j];
#pragma unroll
        for (int u = 1; u < 4; ++u) v = t == u ? s[u * (R / 4) + x][j] : v;
        z[x][j] = v;
      }
  }

  static constexpr int LOGITS = R / 2;
  template <int NP, bool VALUES>
  __device__ __forceinline__ void pages(const uint32_t (&at)[NP], int v_lo, int v_hi,
                                        uint32_t none, char* scratch, float* stash, int stash_n,
                                        int lane) {
    static_assert(NP == 1, "one page at a time");
    const uint32_t stage = at[0];
    if (none) v_lo = kPage;
    float* p = reinterpret_cast<float*>(scratch) + R * DH;
    float* cs = p + kPage * R;
    const int g = lane >> 2, t = lane & 3;
    float z[R / 4][2];
    logits(stage, scratch, lane, z);
    bool grow = false;
    float top[R / 4];
#pragma unroll
    for (int x = 0; x < R / 4; ++x) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = key_of(j, g);
        if (r < v_lo || r >= v_hi) z[x][j] = -INFINITY;
      }
      top[x] = fmaxf(z[x][0], z[x][1]);
#pragma unroll
      for (int s = 4; s < 32; s <<= 1)
        top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], s));
      grow |= top[x] > m[x];
    }
    if (stash_n > 0)
#pragma unroll
      for (int x = 0; x < R / 4; ++x)
        *reinterpret_cast<float2*>(stash + (x * 32 + lane) * 2) = make_float2(z[x][0], z[x][1]);
    const bool scale = __any_sync(0xffffffffu, grow);
    if (scale) {
#pragma unroll
      for (int x = 0; x < R / 4; ++x) {
        const float mn = fmaxf(m[x], top[x]);
        const float c = mn == -INFINITY ? 1.f : fast_exp2(m[x] - mn);
        m[x] = mn;
        l[x] *= c;
        if (g == 0) cs[t * (R / 4) + x] = c;
      }
    }
#pragma unroll
    for (int x = 0; x < R / 4; ++x) {
      const float base = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float w = fast_exp2(z[x][j] - base);
        l[x] += w;
        p[key_of(j, g) * R + t * (R / 4) + x] = w;
      }
    }
    __syncwarp();
    if (!VALUES) return;
    if (scale)
#pragma unroll
      for (int h = 0; h < R; ++h) {
        const float c = cs[h];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][i][e] *= c;
      }
    const uint32_t vs = stage + SH::PAGEB;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w[R];
#pragma unroll
      for (int h = 0; h < R; h += 4)
        *reinterpret_cast<float4*>(w + h) =
            *reinterpret_cast<const float4*>(p + (t + 4 * i) * R + h);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 v = lds16(vs + v_place<SH>(t + 4 * i, g + 8 * c));
#pragma unroll
        for (int h = 0; h < R; ++h) {
          o[h][c][0] = fmaf(w[h], __uint_as_float(v.x), o[h][c][0]);
          o[h][c][1] = fmaf(w[h], __uint_as_float(v.y), o[h][c][1]);
          o[h][c][2] = fmaf(w[h], __uint_as_float(v.z), o[h][c][2]);
          o[h][c][3] = fmaf(w[h], __uint_as_float(v.w), o[h][c][3]);
        }
      }
    }
    __syncwarp();  // p is rewritten by the next page
  }

  __device__ __forceinline__ float sum_l(int x) const {
    float s = l[x];
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    return s;
  }
  // The four lanes of a chunk hold its positions' parts; lane c % 4 ends with
  // the sum.
  __device__ __forceinline__ float4 value(int h, int c) const {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = o[h][c][e];
      v[e] += __shfl_xor_sync(0xffffffffu, v[e], 1);
      v[e] += __shfl_xor_sync(0xffffffffu, v[e], 2);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
  }

  __device__ __forceinline__ void store(float* rec, int lane) const {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < R / 4; ++x) {
      const float s = sum_l(x);
      if (g == 0) {
        rec[t * (R / 4) + x] = m[x];
        rec[R + t * (R / 4) + x] = s;
      }
    }
#pragma unroll
    for (int h = 0; h < R; ++h)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 v = value(h, c);
        if (t == (c & 3)) *reinterpret_cast<float4*>(rec + 2 * R + h * DH + (g + 8 * c) * 4) = v;
      }
  }

  __device__ __forceinline__ void finish(const DecodeArgs& A, int b, int h0, int rows,
                                         int lane) const {
    const int g = lane >> 2, t = lane & 3;
    float inv[R / 4];
#pragma unroll
    for (int x = 0; x < R / 4; ++x) {
      const float s = sum_l(x);
      const int r = t * (R / 4) + x;
      inv[x] = r < rows ? put_lse(A, b, h0 + r, m[x], s, g == 0) : 0.f;
    }
    float* out = static_cast<float*>(A.out) + static_cast<size_t>(b) * A.out_stride +
                 static_cast<size_t>(h0) * DH;
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const float f = __shfl_sync(0xffffffffu, inv[h % (R / 4)], h / (R / 4));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 v = value(h, c);
        if (t == (c & 3) && h < rows)
          *reinterpret_cast<float4*>(out + h * DH + (g + 8 * c) * 4) =
              make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
      }
    }
  }
};

template <int DT, int DH, int GT>
struct TileOf {
  using type = MmaTile<DT, DH, GT>;
};
template <int DH, int GT>
struct TileOf<PE_KV_F32, DH, GT> {
  using type = F32Tile<DH>;
};

// ----------------------------------------------------------------- results

// Joins the parts of one item inside a CTA: part[0] .. part[count - 1] in the
// order of the positions, into the result (dst NULL) or a record.
template <int DT, int DH, int GT, int W>
__device__ __forceinline__ void join_in_cta(const DecodeArgs& a, int b, int hh, int count,
                                            const float* const (&part)[W], float* dst) {
  using SH = DecodeShape<DT, DH, GT>;
  const int h0 = hh / a.tiles * a.G + (hh % a.tiles) * SH::ROWS;
  const int rows = min(SH::ROWS, a.G - (hh % a.tiles) * SH::ROWS);
#pragma unroll 1
  for (int e = threadIdx.x * 4; e < SH::ROWS * DH; e += W * 32 * 4) {
    const int r = e / DH, d = e % DH;
    float m[W], l[W];
    float4 v[W];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) {  // every load before any use; past count: the first again
      m[i] = part[i][r];
      l[i] = part[i][SH::ROWS + r];
      v[i] = *reinterpret_cast<const float4*>(part[i] + 2 * SH::ROWS + e);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) M = fmaxf(M, i < count ? m[i] : -INFINITY);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i >= count) break;
      const float c = fast_exp2(m[i] - base);
      L = fmaf(c, l[i], L);
      O = make_float4(fmaf(c, v[i].x, O.x), fmaf(c, v[i].y, O.y), fmaf(c, v[i].z, O.z),
                      fmaf(c, v[i].w, O.w));
    }
    if (dst) {
      *reinterpret_cast<float4*>(dst + 2 * SH::ROWS + e) = O;
      if (d == 0) {
        dst[r] = M;
        dst[SH::ROWS + r] = L;
      }
    } else if (r < rows) {
      const float f = put_lse(a, b, h0 + r, M, L, d == 0);
      put4<DT>(a.out, static_cast<size_t>(b) * a.out_stride + static_cast<size_t>(h0 + r) * DH + d,
               make_float4(O.x * f, O.y * f, O.z * f, O.w * f));
    }
  }
}

// A CTA's meta: of its last part, if that item began in the CTA and goes on
// after it, the request (.x, else -1), the head tile (.y) and the number of
// CTAs that have parts of it (.z).

// VALUES false: K alone, for the lse (and the logits); out gets zeros.
template <int DT, int DH, int GT, bool VALUES>
__global__ void __launch_bounds__(DecodeShape<DT, DH, GT>::WARPS * 32,
                                  DecodeShape<DT, DH, GT>::CTAS)
    attn_decode_kernel(const __grid_constant__ DecodeArgs a) {
  using SH = DecodeShape<DT, DH, GT>;
  using Tile = typename TileOf<DT, DH, GT>::type;
  using Feed = Feeder<SH, VALUES>;
  constexpr int RING = VALUES ? SH::RING : SH::S_RING;
  constexpr int W = SH::WARPS, THREADS = W * 32;
  extern __shared__ __align__(128) char smem[];
  __shared__ int prefix[THREADS];
  // a warp's parts: first (its item began before the piece), last (it goes on
  // after it)
  __shared__ int w_state[W], w_b[W][2], w_hh[W][2];
  __shared__ int after;  // pages of the CTA's last item that lie after it
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int heads = a.Hkv * a.tiles;
  const Line ln = line_setup<THREADS>(a, heads, prefix);
  // CTAs and warps take whole pages, the first ones one more; with few pages,
  // kMinPages a warp on fewer CTAs
  const int grid = min(static_cast<int>(gridDim.x),
                       max(1, static_cast<int>((static_cast<uint32_t>(ln.total) + W * kMinPages - 1) /
                                               (W * kMinPages))));
  const Share cta = share_of(ln.total, grid, blockIdx.x);
  if (cta.count == 0) {
    if (tid == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const Share mine = share_of(cta.count, W, w);
  const int working = min(cta.count, W);
  char* ring_p = smem + w * RING;
  char* scratch = smem + W * RING + w * SH::SCRATCH;
  const uint32_t ring = smem_u32(ring_p);
  float* my_last = reinterpret_cast<float*>(ring_p);
  float* my_head = a.head + (static_cast<size_t>(blockIdx.x) * W + w) * SH::REC;
  // bits of w_state: 1 a first partial in the head record, 2 it is in the
  // ring instead, 4 its item ends here, 8 a last partial in the ring
  int state = 0;
  if (mine.count > 0) {
    Place pl = place_of<THREADS>(a, ln, heads, prefix, cta.first + mine.first);
    Feed feed;
    feed.start(a, pl, a.tiles, mine.count, lane);
    int unit = cta.first + mine.first;  // of the page that is taken next
#pragma unroll 1
    for (int i = 0; i < Feed::STAGES; ++i) feed.step(a, heads, a.tiles, ring, lane, true);
    int left = mine.count, stage = 0;
    Tile tile;
    while (true) {
      const bool began = pl.p == pl.s.pf;
      const int hk = pl.hh / a.tiles, r0 = (pl.hh % a.tiles) * SH::ROWS;
      const int rows = min(SH::ROWS, a.G - r0);
      tile.start(a, pl.b, hk * a.G + r0, rows, scratch, lane);
      const int stop = min(pl.s.pe, pl.p + left);
      left -= stop - pl.p;
      auto take = [&](auto count) {
        constexpr int NP = decltype(count)::value;
        cp_async_wait<Feed::STAGES - NP>();
        __syncwarp();  // other lanes' copies, and their reads of the pages before
        uint32_t at[NP], none = 0;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          at[n] = ring + stage * Feed::STRIDE;
          none |= ((feed.bad >> stage) & 1) << n;
          if (++stage == Feed::STAGES) stage = 0;
        }
        const int first = pl.p * kPage;
        tile.template pages<NP, VALUES>(at, pl.s.lo - first, pl.s.n - first, none, scratch,
                                a.stash + static_cast<size_t>(unit) * Tile::LOGITS * 32,
                                a.stash_pages - unit, lane);
        unit += NP;
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NP; ++n) feed.step(a, heads, a.tiles, ring, lane, true);
        pl.p += NP;
      };
      if constexpr (SH::TAKE > 1)
        while (pl.p + SH::TAKE <= stop) take(std::integral_constant<int, SH::TAKE>());
      while (pl.p < stop) take(std::integral_constant<int, 1>());
      const bool ended = pl.p == pl.s.pe;
      if (left > 0) {  // more items follow in this piece
        if (began) {   // and this one is complete
          tile.finish(a, pl.b, hk * a.G + r0, rows, lane);
        } else {
          tile.store(my_head, lane);
          state |= 1 | 4;
          if (lane == 0) {
            w_b[w][0] = pl.b;
            w_hh[w][0] = pl.hh;
          }
        }
        next_item(a, heads, pl);
        continue;
      }
      cp_async_wait<0>();
      __syncwarp();
      if (began && ended) {
        tile.finish(a, pl.b, hk * a.G + r0, rows, lane);
      } else {
        tile.store(my_last, lane);
        if (w == working - 1 && lane == 0) after = pl.s.pe - pl.p;
        if (!began) {
          state |= 1 | 2 | (ended ? 4 : 0);
          if (lane == 0) {
            w_b[w][0] = pl.b;
            w_hh[w][0] = pl.hh;
          }
        }
        if (!ended) {
          state |= 8;
          if (lane == 0) {
            w_b[w][1] = pl.b;
            w_hh[w][1] = pl.hh;
          }
        }
      }
      break;
    }
  }
  if (lane == 0) w_state[w] = state;
  __syncthreads();
  // Chains of parts of one item: the warps from `from` on.  A warp's first
  // part lies in its ring (bit of in_ring) or its head record, its last part
  // in its ring.
  uint32_t in_ring = 0;
#pragma unroll
  for (int x = 0; x < W; ++x) in_ring |= ((w_state[x] >> 1) & 1) << x;
  int4 meta = make_int4(-1, 0, 0, 0);
  int from = -1;        // first warp of the open chain, its part there: last (or first)
  bool before = false;  // the chain began before this CTA
  float* part = a.part + static_cast<size_t>(blockIdx.x) * 2 * SH::REC;
#pragma unroll 1
  for (int x = 0; x <= working; ++x) {
    const int st = x < working ? w_state[x] : 0;
    if ((st & 1) && from < 0) {
      from = x;
      before = true;
    }
    const bool over = x == working;  // what is open goes on after the CTA
    if (from >= 0 && ((st & 4) || over)) {
      const int count = over ? x - from : x - from + 1;
      const float* parts[W];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i > 0 && i >= count) {
          parts[i] = parts[0];
          continue;
        }
        const int y = from + i;
        parts[i] = (i == 0 && !before) || ((in_ring >> y) & 1)
                       ? reinterpret_cast<const float*>(smem + y * RING)
                       : a.head + (static_cast<size_t>(blockIdx.x) * W + y) * SH::REC;
      }
      const int y = over ? from : x, k = over && !before ? 1 : 0;
      join_in_cta<DT, DH, GT, W>(a, w_b[y][k], w_hh[y][k], count, parts,
                                 before ? part : over ? part + SH::REC : nullptr);
      if (over && !before) {
        // how many of the next CTAs the rest of the item reaches
        meta.x = w_b[from][1];
        meta.y = w_hh[from][1];
        const Share next = share_of(ln.total, grid, min(static_cast<int>(blockIdx.x) + 1, grid - 1));
        const Share last = share_of(ln.total, grid, grid - 1);
        meta.z = 2;
        int rest = after - next.count;
        if (rest > 0) {
          // further CTAs of next.count pages, then shorter ones
          const int wide = next.count > last.count
                               ? ln.total - last.count * grid - static_cast<int>(blockIdx.x + 2)
                               : 0;
          const int of_wide = min(wide, (rest + next.count - 1) / next.count);
          rest -= of_wide * next.count;
          meta.z += of_wide;
          if (rest > 0) meta.z += (rest + last.count - 1) / last.count;
        }
      }
      from = -1;
      before = false;
    }
    if ((st & 8) && from < 0) from = x;
  }
  if (tid == 0) a.meta[blockIdx.x] = meta;
}

// Items that several CTAs share: block c joins the one whose first part is
// CTA c's last; blocks of y take a share of the rows.  The parts' m and l come
// in at once, then the products with every part's load in flight together.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 4;  // blocks of y
template <int DT, int DH, int GT>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(
    const __grid_constant__ DecodeArgs a) {
  using SH = DecodeShape<DT, DH, GT>;
  constexpr int R = SH::ROWS / kJoinRows;          // rows of this block
  constexpr int LANES = R * DH / 4;                // threads that hold the row's elements
  constexpr int WAYS = kJoinThreads / LANES;       // parts taken side by side
  constexpr int MOST = kMostCtas;
  __shared__ float wt[MOST][R], ls[MOST][R], red[2][R];
  __shared__ float4 side[WAYS > 1 ? WAYS : 1][LANES];
  grid_dep_wait();
  grid_dep_launch();
  const int c = blockIdx.x, row0 = blockIdx.y * R, tid = threadIdx.x;
  const int4 meta = __ldcg(a.meta + c);
  // rows that attend nothing
  for (int b = blockIdx.x * kJoinRows + blockIdx.y; b < a.B; b += gridDim.x * kJoinRows) {
    const Span s = span_of(a, b, tid == 0);
    if (s.pe > s.pf) continue;
    for (int e = tid * 4; e < a.Hq * DH; e += kJoinThreads * 4)
      put4<DT>(a.out, static_cast<size_t>(b) * a.out_stride + e, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = tid; h < a.Hq; h += kJoinThreads) {
      a.lse_w[static_cast<size_t>(b) * a.Hq + h] = -INFINITY;
      if (a.lse) a.lse[static_cast<size_t>(b) * a.Hq + h] = -INFINITY;
    }
  }
  if (meta.x < 0) return;
  const int b = meta.x, hh = meta.y, count = min(meta.z, MOST);
  auto rec = [&](int i) -> const float* {
    return a.part + (static_cast<size_t>(c + i) * 2 + (i == 0 ? 1 : 0)) * SH::REC;
  };
  for (int k = tid; k < count * R; k += kJoinThreads) {
    wt[k / R][k % R] = __ldcg(rec(k / R) + row0 + k % R);
    ls[k / R][k % R] = __ldcg(rec(k / R) + SH::ROWS + row0 + k % R);
  }
  __syncthreads();
  // a warp a row: the maximum, then the weights and the sum
  for (int r = tid >> 5; r < R; r += kJoinThreads / 32) {
    const int lane = tid & 31;
    float M = -INFINITY;
    for (int i = lane; i < count; i += 32) M = fmaxf(M, wt[i][r]);
#pragma unroll
    for (int k = 16; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int i = lane; i < count; i += 32) {
      const float x = fast_exp2(wt[i][r] - base);
      L = fmaf(x, ls[i][r], L);
      wt[i][r] = x;
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
    if (lane == 0) {
      red[0][r] = M;
      red[1][r] = L;
    }
  }
  __syncthreads();
  const int way = tid / LANES, e = (tid % LANES) * 4, r = e / DH;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = way; i < count; i += WAYS) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(rec(i) + 2 * SH::ROWS + row0 * DH + e));
    const float x = wt[i][r];
    O = make_float4(fmaf(x, v.x, O.x), fmaf(x, v.y, O.y), fmaf(x, v.z, O.z), fmaf(x, v.w, O.w));
  }
  if (WAYS > 1) {
    side[way][tid % LANES] = O;
    __syncthreads();
    if (way > 0) return;
#pragma unroll
    for (int k = 1; k < WAYS; ++k) {
      const float4 v = side[k][tid];
      O = make_float4(O.x + v.x, O.y + v.y, O.z + v.z, O.w + v.w);
    }
  }
  const int h0 = hh / a.tiles * a.G + (hh % a.tiles) * SH::ROWS;
  const int rows = min(SH::ROWS, a.G - (hh % a.tiles) * SH::ROWS);
  if (row0 + r >= rows) return;
  const float f = put_lse(a, b, h0 + row0 + r, red[0][r], red[1][r], e % DH == 0);
  put4<DT>(a.out,
           static_cast<size_t>(b) * a.out_stride + static_cast<size_t>(h0 + row0 + r) * DH + e % DH,
           make_float4(O.x * f, O.y * f, O.z * f, O.w * f));
}

// Adds the weights of a page's positions to the pool's scores.  v[i]: this
// lane's part of the sum at position pos[i] of four, joined over the eight
// lanes of equal t; each lane ends with one position's sum.
__device__ __forceinline__ float join_heads(const float (&v)[4], int g) {
  // three exchanges halve the four values, then the two, then add the last
  const float a0 = g & 4 ? v[2] : v[0], a1 = g & 4 ? v[3] : v[1];
  const float b0 = g & 4 ? v[0] : v[2], b1 = g & 4 ? v[1] : v[3];
  const float c0 = a0 + __shfl_xor_sync(0xffffffffu, b0, 16);
  const float c1 = a1 + __shfl_xor_sync(0xffffffffu, b1, 16);
  const float d = (g & 2 ? c1 : c0) + __shfl_xor_sync(0xffffffffu, g & 2 ? c0 : c1, 8);
  return d + __shfl_xor_sync(0xffffffffu, d, 4);  // value (g >> 1): j = g / 4, e = g / 2 % 2
}
__device__ __forceinline__ void add_scores(const DecodeArgs& a, const Span& s, int hk, int blk,
                                           int p, int r, bool mine, float v) {
  const int at = p * kPage + r;
  if (mine && blk >= 0 && blk < a.pool.num_blocks && at >= s.lo && at < s.n)
    atomicAdd(a.pool.scores + (static_cast<size_t>(blk) * a.Hkv + hk) * kPage + r, v);
}

// Weights, now that lse is known: of the pages whose logits the first kernel
// left in the workspace from those, of the others from the logits once more.
// A page of a kv head belongs to one warp, which sums its query heads in
// order; the additions are reductions in L2 because requests may share pages.
// Logits kept: 32 bytes a position and kv head of 8 query heads, written and
// read once, mostly in L2, against 64 to 256 bytes of K (16 requests of 137975
// positions, heads of 128: 78 us with K again, 65 with kept logits).
template <int DT, int DH, int GT>
__global__ void __launch_bounds__(DecodeShape<DT, DH, GT>::WARPS * 32, 2)
    attn_scores_kernel(const __grid_constant__ DecodeArgs a) {
  using SH = DecodeShape<DT, DH, GT>;
  using Feed = Feeder<SH, false>;
  using Tile = typename TileOf<DT, DH, GT>::type;
  constexpr bool F32 = DT == PE_KV_F32;
  constexpr int W = SH::WARPS, THREADS = W * 32;
  constexpr int LH = F32 ? SH::ROWS / 4 : GT;  // heads a lane
  extern __shared__ __align__(128) char smem[];
  __shared__ int prefix[THREADS];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const Line ln = line_setup<THREADS>(a, a.Hkv, prefix);
  const Share mine = share_of(ln.total, gridDim.x * W, blockIdx.x * W + w);
  if (mine.count == 0) return;
  char* scratch = smem + W * SH::S_RING + w * SH::SCRATCH;
  const uint32_t ring = smem_u32(smem + w * SH::S_RING);
  Place pl = place_of<THREADS>(a, ln, a.Hkv, prefix, mine.first);
  // a lane's row of the tile and, of the lanes that hold a sum, its position
  auto head_of = [&](int x) { return F32 ? t * LH + x : g + 8 * x; };
  const int r = F32 ? key_of(t & 1, g) : key_of(g >> 2, 2 * t + ((g >> 1) & 1));
  const bool adds = F32 ? t < 2 : (g & 1) == 0;
  float lse[LH];
  auto load_lse = [&](int r0) {
#pragma unroll
    for (int x = 0; x < LH; ++x) {
      // a row without weight, or no row
      lse[x] = -INFINITY;
      if (head_of(x) < min(SH::ROWS, a.G - r0))
        lse[x] = __ldcg(a.lse_w + static_cast<size_t>(pl.b) * a.Hq + pl.hh * a.G + r0 + head_of(x));
    }
  };
  auto weight = [&](float z, int x) {
    return lse[x] == -INFINITY ? 0.f : fast_exp2(z - lse[x]);
  };
  // ---- logits that are there
  int left = min(mine.count, max(0, a.stash_pages - mine.first));
  const int over = mine.count - left;
  if (left > 0) {
    const float* stash = a.stash + static_cast<size_t>(mine.first) * Tile::LOGITS * 32;
    load_lse(0);
    while (left > 0) {
      if (pl.p == pl.s.pe) {
        next_item(a, a.Hkv, pl);
        load_lse(0);
      }
      const int run = min(min(pl.s.pe - pl.p, left), 32);
      const int ids =
          lane < run ? a.block_table[static_cast<size_t>(pl.b) * a.bt_stride + pl.p + lane] : -1;
      constexpr int U = 4;  // pages in flight
#pragma unroll 1
      for (int i = 0; i < run; i += U) {
        float z[U][Tile::LOGITS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* from = stash + static_cast<size_t>(min(i + u, run - 1)) * Tile::LOGITS * 32;
          if constexpr (F32) {
#pragma unroll
            for (int x = 0; x < LH; ++x) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(from + (x * 32 + lane) * 2));
              z[u][2 * x] = v.x;
              z[u][2 * x + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int x = 0; x < GT; ++x) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(from + (x * 32 + lane) * 4));
              z[u][4 * x] = v.x;
              z[u][4 * x + 1] = v.y;
              z[u][4 * x + 2] = v.z;
              z[u][4 * x + 3] = v.w;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float sum;
          if constexpr (F32) {
            float v[2] = {0.f, 0.f};
#pragma unroll
            for (int x = 0; x < LH; ++x)
#pragma unroll
              for (int j = 0; j < 2; ++j) v[j] += weight(z[u][2 * x + j], x);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              v[j] += __shfl_xor_sync(0xffffffffu, v[j], 1);
              v[j] += __shfl_xor_sync(0xffffffffu, v[j], 2);
            }
            sum = t & 1 ? v[1] : v[0];
          } else {
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < GT; ++x)
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] += weight(z[u][4 * x + k], x);
            sum = join_heads(v, g);
          }
          const int blk = __shfl_sync(0xffffffffu, ids, min(i + u, 31));
          add_scores(a, pl.s, pl.hh, blk, pl.p + i + u, r, adds && i + u < run, sum);
        }
      }
      stash += static_cast<size_t>(run) * Tile::LOGITS * 32;
      pl.p += run;
      left -= run;
    }
  }
  // ---- logits once more
  if (over == 0) return;
  if (pl.p == pl.s.pe) next_item(a, a.Hkv, pl);
  left = over;
  Feed feed;
  feed.start(a, pl, 1, left, lane);
#pragma unroll 1
  for (int i = 0; i < Feed::STAGES; ++i) feed.step(a, a.Hkv, 1, ring, lane, false);
  int stage = 0;
  int have = -1;  // head tile whose query and lse are loaded
  Tile tile;
  auto take = [&](auto count) {
    constexpr int NP = decltype(count)::value;
    cp_async_wait<Feed::STAGES - NP>();
    __syncwarp();
    uint32_t at[NP];
    int blk[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
      at[n] = ring + stage * Feed::STRIDE;
      blk[n] = a.block_table[static_cast<size_t>(pl.b) * a.bt_stride + pl.p + n];
      if (++stage == Feed::STAGES) stage = 0;
    }
    float sum[NP] = {};
    for (int ht = 0; ht < a.tiles; ++ht) {
      if (have != ht) {
        const int r0 = ht * SH::ROWS;
        tile.start(a, pl.b, pl.hh * a.G + r0, min(SH::ROWS, a.G - r0), scratch, lane);
        load_lse(r0);
        have = ht;
      }
      if constexpr (F32) {
        float z[LH][2], v[2] = {0.f, 0.f};
        F32Tile<DH>::logits(at[0], scratch, lane, z);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int x = 0; x < LH; ++x) v[j] += weight(z[x][j], x);
          v[j] += __shfl_xor_sync(0xffffffffu, v[j], 1);
          v[j] += __shfl_xor_sync(0xffffffffu, v[j], 2);
        }
        sum[0] += t & 1 ? v[1] : v[0];
      } else {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
          float z[GT][2][2], v[4] = {0.f, 0.f, 0.f, 0.f};
          tile.q.template sums<SH>(at[n], lane, z);
#pragma unroll
          for (int x = 0; x < GT; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[k] += weight(z[x][k >> 1][k & 1] * tile.q.factor[x], x);
          sum[n] += join_heads(v, g);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NP; ++n) feed.step(a, a.Hkv, 1, ring, lane, false);
#pragma unroll
    for (int n = 0; n < NP; ++n) add_scores(a, pl.s, pl.hh, blk[n], pl.p + n, r, adds, sum[n]);
    pl.p += NP;
    left -= NP;
  };
  while (left > 0) {
    if (pl.p == pl.s.pe) {
      next_item(a, a.Hkv, pl);
      have = -1;
    }
    const int run = min(pl.s.pe - pl.p, left);
    if (SH::S_TAKE > 1 && run >= SH::S_TAKE) take(std::integral_constant<int, SH::S_TAKE>());
    else take(std::integral_constant<int, 1>());
  }
}

// --------------------------------------------------------------- launchers

static int sm_count(int& dev) {
  int sms = 0;
  dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

// The kernels' shared memory, asked for once per device.
template <int DT, int DH, int GT, bool VALUES>
static cudaError_t allow_smem(int dev) {
  using SH = DecodeShape<DT, DH, GT>;
  static std::atomic<uint64_t> done{0};
  if (dev < 64 && ((done.load(std::memory_order_relaxed) >> dev) & 1)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<DT, DH, GT, VALUES>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       VALUES ? SH::SMEM : SH::S_SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_scores_kernel<DT, DH, GT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SH::S_SMEM);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

template <int DT, int DH, int GT, bool VALUES>
static pe_status launch_decode(DecodeArgs& a, char* ws, char* ws_end, int dev, int sms,
                               bool accumulate, cudaStream_t s) {
  using SH = DecodeShape<DT, DH, GT>;
  const int grid = std::min(sms * SH::CTAS, kMostCtas);
  a.tiles = (a.G + SH::ROWS - 1) / SH::ROWS;
  a.lse_w = reinterpret_cast<float*>(ws);
  ws += (static_cast<size_t>(a.B) * a.Hq * 4 + 15) / 16 * 16;
  a.meta = reinterpret_cast<int4*>(ws);
  ws += static_cast<size_t>(grid) * sizeof(int4);
  a.part = reinterpret_cast<float*>(ws);
  ws += static_cast<size_t>(grid) * 2 * SH::REC * 4;
  a.head = reinterpret_cast<float*>(ws);
  ws += static_cast<size_t>(grid) * SH::WARPS * SH::REC * 4;
  // the rest of the workspace holds logits, where one tile has all heads
  a.stash = reinterpret_cast<float*>(ws);
  constexpr int page = TileOf<DT, DH, GT>::type::LOGITS * 32 * 4;
  a.stash_pages = accumulate && a.tiles == 1 && ws_end > ws
                      ? static_cast<int>(std::min<int64_t>((ws_end - ws) / page, 1 << 30))
                      : 0;
  cudaError_t e = allow_smem<DT, DH, GT, VALUES>(dev);
  if (e == cudaSuccess)
    e = launch_pdl(attn_decode_kernel<DT, DH, GT, VALUES>, dim3(grid), dim3(SH::WARPS * 32),
                   VALUES ? SH::SMEM : SH::S_SMEM, s, a);
  if (e == cudaSuccess)
    e = launch_pdl(attn_join_kernel<DT, DH, GT>, dim3(grid, kJoinRows), dim3(kJoinThreads), 0, s, a);
  if (e == cudaSuccess && accumulate)
    e = launch_pdl(attn_scores_kernel<DT, DH, GT>, dim3(2 * sms), dim3(SH::WARPS * 32), SH::S_SMEM,
                   s, a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

template <bool VALUES, int DT, int DH>
static pe_status launch_decode_heads(DecodeArgs& a, char* ws, char* ws_end, int dev, int sms,
                                     bool accumulate, cudaStream_t s) {
  if constexpr (DT != PE_KV_F32)
    if (a.G > 8) return launch_decode<DT, DH, 2, VALUES>(a, ws, ws_end, dev, sms, accumulate, s);
  return launch_decode<DT, DH, 1, VALUES>(a, ws, ws_end, dev, sms, accumulate, s);
}

// Logits that a call with accumulate may keep: more are worked out again.
constexpr int64_t kMostLogits = int64_t{1} << 30;  // bytes

// Query heads a kv head whose logits a call can keep: those of one tile.
static int most_kept_heads(int dtype, int dh) {
  if (dtype != PE_KV_F32) return DecodeShape<PE_KV_BF16, 64, 2>::ROWS;
  return dh == 64 ? DecodeShape<PE_KV_F32, 64, 1>::ROWS : DecodeShape<PE_KV_F32, 128, 1>::ROWS;
}

// The largest of the pool types: two CTAs an SM, 8 or 16 rows a tile.
static int64_t workspace_bytes_for(int64_t B, int n_heads, int n_kv_heads, int head_dim, int sms) {
  const int64_t grid = 2 * sms, rows = n_heads / n_kv_heads > 8 ? 16 : 8;
  return (B * n_heads * 4 + 15) / 16 * 16 + grid * 16 +
         grid * (2 + kMaxWarps) * rows * (head_dim + 2) * 4;
}

template <bool VALUES>
static pe_status launch_decode_pool(DecodeArgs& a, int dtype, int dh, void* workspace,
                                    int64_t workspace_bytes, int dev, int sms, bool acc,
                                    cudaStream_t s) {
  char* ws = static_cast<char*>(workspace);
  char* end = ws + workspace_bytes;
  if (dtype == PE_KV_F32)
    return dh == 64 ? launch_decode_heads<VALUES, PE_KV_F32, 64>(a, ws, end, dev, sms, acc, s)
                    : launch_decode_heads<VALUES, PE_KV_F32, 128>(a, ws, end, dev, sms, acc, s);
  if (dtype == PE_KV_BF16)
    return dh == 64 ? launch_decode_heads<VALUES, PE_KV_BF16, 64>(a, ws, end, dev, sms, acc, s)
                    : launch_decode_heads<VALUES, PE_KV_BF16, 128>(a, ws, end, dev, sms, acc, s);
  return dh == 64 ? launch_decode_heads<VALUES, PE_KV_E4M3, 64>(a, ws, end, dev, sms, acc, s)
                  : launch_decode_heads<VALUES, PE_KV_E4M3, 128>(a, ws, end, dev, sms, acc, s);
}

pe_status launch_draft_scores(const DraftScoresArgs& d, cudaStream_t s) {
  int dev;
  const int sms = sm_count(dev);
  if (sms < 1) return PE_ERR_CUDA;
  DecodeArgs a = {};
  a.pool = CachePool{d.k, d.v, d.scores, d.num_blocks};
  a.B = d.B;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.G = d.Hq / d.Hkv;
  a.bt_stride = d.bt_stride;
  const bool codes = d.dtype == PE_KV_E4M3;
  a.scale = kLog2e / std::sqrt(static_cast<float>(d.dh)) * (codes ? d.k_scale : 1.f);
  a.v_scale = codes ? d.v_scale / kLift : 1.f;
  a.q = d.q;
  a.q_stride = a.out_stride = static_cast<long long>(d.Hq) * d.dh;
  a.q_rows = d.q_rows;
  a.q_rows_stride = d.q_rows_stride;
  a.q_limit = d.rows;
  a.len_add = d.len_add;
  a.block_table = d.block_table;
  a.seq_lens = d.seq_lens;
  a.out = d.out;
  a.err = d.err;
  return launch_decode_pool<false>(a, d.dtype, d.dh, d.workspace, d.workspace_bytes, dev, sms, true, s);
}
int64_t draft_scores_workspace(int B, int Hq, int Hkv, int dh, int dtype, int bt_stride) {
  return pe_attn_decode_workspace(B, Hq, Hkv, dh,
                                  Hq / Hkv <= most_kept_heads(dtype, dh) ? bt_stride : 0);
}

}  // namespace pe

extern "C" {

int64_t pe_attn_decode_workspace(int32_t B, int32_t n_heads, int32_t n_kv_heads,
                                 int32_t head_dim, int32_t bt_stride) {
  if (B < 1 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || bt_stride < 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  int dev;
  const int sms = pe::sm_count(dev);
  if (sms < 1) return 0;
  const int64_t rows = n_heads / n_kv_heads > 8 ? 16 : 8;
  // (fp32 pools keep those of fewer heads; the type is not known here)
  const double logits = n_heads / n_kv_heads > pe::most_kept_heads(PE_KV_BF16, head_dim)
                            ? 0.0
                            : 1.0 * B * bt_stride * n_kv_heads * pe::kPage * rows * 4;
  return pe::workspace_bytes_for(B, n_heads, n_kv_heads, head_dim, sms) +
         (logits < pe::kMostLogits ? static_cast<int64_t>(logits) : pe::kMostLogits);
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
      !row_ok(out, out_stride, qw, eb) || out == q || (accumulate && !pool->scores) || !workspace ||
      !is_aligned16(workspace) || workspace_bytes <= 0)
    return PE_ERR_INVALID_ARGUMENT;
  // the pages are counted in 32 bits (a table of that size is 8 GB)
  if (static_cast<int64_t>(B) * bt_stride > 2147483647LL / n_heads) return PE_ERR_UNSUPPORTED;
  int dev;
  const int sms = sm_count(dev);
  if (sms < 1) return PE_ERR_CUDA;
  if (workspace_bytes < workspace_bytes_for(B, n_heads, pool->n_kv_heads, dh, sms))
    return PE_ERR_INVALID_ARGUMENT;
  DecodeArgs a = {};
  a.pool = CachePool{pool->k, pool->v, pool->scores, pool->num_blocks};
  a.B = B;
  a.Hq = n_heads;
  a.Hkv = pool->n_kv_heads;
  a.G = n_heads / pool->n_kv_heads;
  a.bt_stride = bt_stride;
  a.window = window;
  const bool codes = pool->dtype == PE_KV_E4M3;
  a.scale = scale * kLog2e * (codes ? pool->k_scale : 1.f);
  if (!std::isfinite(a.scale)) return PE_ERR_INVALID_ARGUMENT;
  a.v_scale = codes ? pool->v_scale / kLift : 1.f;
  a.q = q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.err = err;
  return launch_decode_pool<true>(a, pool->dtype, dh, workspace, workspace_bytes, dev, sms,
                            accumulate != 0, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
