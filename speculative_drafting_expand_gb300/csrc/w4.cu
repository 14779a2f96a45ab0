// w4.cu -- products of a few rows with 4-bit weights that have a scale for
// each group of inputs (include/peagle_w4.h).
//
// Packed layout.  The matrix is cut into tiles of 16 rows and units of 64
// inputs (groups of 128: an even number), filled up with zeros.  First the codes, [tile][unit][lane][16
// bytes]: word j of a lane is its part of the left operand of one m16n8k16
// product (inputs 16 j .. 16 j + 15 of the unit), so a warp reads a unit as
// one 512-byte line and needs no exchange.  Register i of the operand takes
// nibbles i (low half) and i + 4 (high half) of the word: one shift and one
// logic operation make a pair of bf16 numbers 128 + code, one subtraction the
// exact pair code - 8.  Then the scales, bf16, rows g and g + 8 of a tile side
// by side in a word, which is what a lane needs of a group: groups of 32, two
// words a unit, [tile][unit][g][2]; of 64, [tile][unit][g]; of 128,
// [tile][pair of units][g].
#include <algorithm>
#include <cmath>

#include "../../include/peagle_w4.h"
#include "pe_common.cuh"
#include "pe_kernels.h"

namespace pe {

constexpr int kUnit = 64;        // inputs of a unit
constexpr int kTileRows = 16;    // outputs of a tile
constexpr int kUnitBytes = 512;  // codes of a tile's unit

struct W4Shape {
  int n, k, group;
  int tiles, units, groups;
  int words;  // scale words of a tile and g
  __host__ __device__ W4Shape() {}
  __host__ __device__ W4Shape(int n_, int k_, int group_)
      : n(n_), k(k_), group(group_), tiles((n_ + kTileRows - 1) / kTileRows),
        units(group_ == 128 ? (k_ + 127) / 128 * 2 : (k_ + kUnit - 1) / kUnit),
        groups((k_ + group_ - 1) / group_),
        words(group_ == 32 ? 2 * units : group_ == 64 ? units : units / 2) {}
  __host__ __device__ long long code_bytes() const {
    return static_cast<long long>(tiles) * units * kUnitBytes;
  }
  __host__ __device__ long long bytes() const {
    return code_bytes() + static_cast<long long>(tiles) * words * (kTileRows * 2);
  }
  // bf16 element of the scale of a tile's row in a group
  __host__ __device__ long long scale_at(int tile, int row, int g32) const {
    const int w = group == 32 ? (g32 / 2 * 8 + (row & 7)) * 2 + (g32 & 1) : g32 * 8 + (row & 7);
    return (static_cast<long long>(tile) * words * 8 + w) * 2 + (row >> 3);
  }
};

// ------------------------------------------------------------------- packing
// Row and input of nibble i of word `step` of a lane, within a tile's unit.
__device__ __forceinline__ void nibble_place(int lane, int step, int i, int& row, int& in) {
  const int reg = i & 3, hi = i >> 2, g = lane / 4, t = lane % 4;
  row = g + (reg & 1) * 8;
  in = step * 16 + (reg >> 1) * 8 + 2 * t + hi;
}

struct W4PackArgs {
  W4Shape sh;
  const uint8_t* codes;
  const bf16* scales;
  const void* w;
  long long w_stride;
  void* packed;
};

// A warp a unit of a tile; done once per matrix.
__global__ void w4_pack_kernel(const __grid_constant__ W4PackArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const W4Shape sh = a.sh;
  const int lane = threadIdx.x % 32;
  const long long warps = static_cast<long long>(gridDim.x) * blockDim.x / 32;
  const long long first = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  const int row_bytes = (sh.k + 1) / 2;
  for (long long u = first; u < static_cast<long long>(sh.tiles) * sh.units; u += warps) {
    const int tile = static_cast<int>(u / sh.units), unit = static_cast<int>(u % sh.units);
    uint32_t word[4];
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      word[step] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int row, in;
        nibble_place(lane, step, i, row, in);
        row += tile * kTileRows;
        in += unit * kUnit;
        uint32_t c = 8;
        if (row < sh.n && in < sh.k)
          c = (a.codes[static_cast<long long>(row) * row_bytes + in / 2] >> (4 * (in & 1))) & 15;
        word[step] |= c << (4 * i);
      }
    }
    static_cast<uint4*>(a.packed)[u * 32 + lane] = make_uint4(word[0], word[1], word[2], word[3]);
  }
  bf16* out = reinterpret_cast<bf16*>(static_cast<char*>(a.packed) + sh.code_bytes());
  // groups past the last input have a place too (no group fills one alone: 0)
  const long long all = static_cast<long long>(sh.tiles) * sh.words * kTileRows;
  for (long long i = first * 32 + lane; i < all; i += warps * 32) {
    const int r = static_cast<int>(i % kTileRows);
    const long long tg = i / kTileRows;
    const int group = static_cast<int>(tg % sh.words), tile = static_cast<int>(tg / sh.words);
    const long long row = static_cast<long long>(tile) * kTileRows + r;
    out[sh.scale_at(tile, r, group)] = row < sh.n && group < sh.groups
                                           ? a.scales[row * sh.groups + group]
                                           : __float2bfloat16_rn(0.f);
  }
}

// A warp 16 rows of a group: the group's scale, then its codes.
template <typename T>
__global__ void w4_quantize_kernel(const __grid_constant__ W4PackArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const W4Shape sh = a.sh;
  const int lane = threadIdx.x % 32;
  const long long warps = static_cast<long long>(gridDim.x) * blockDim.x / 32;
  const long long first = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  bf16* out = reinterpret_cast<bf16*>(static_cast<char*>(a.packed) + sh.code_bytes());
  const T* w = static_cast<const T*>(a.w);
  // a work item: a tile and a span of inputs that holds whole units and groups
  const int span = max(sh.group, kUnit), spans = (sh.k + span - 1) / span;
  for (long long item = first; item < static_cast<long long>(sh.tiles) * spans; item += warps) {
    const int tile = static_cast<int>(item / spans), s0 = static_cast<int>(item % spans) * span;
    float scale[2][2] = {};  // rows g and g + 8 of up to two groups of the span
    for (int r = 0; r < kTileRows; ++r) {
      const long long row = static_cast<long long>(tile) * kTileRows + r;
      for (int gi = 0; gi * sh.group < span; ++gi) {
        const int lo = s0 + gi * sh.group, hi = min(lo + sh.group, sh.k);
        float most = 0.f;
        if (row < sh.n)
          for (int j = lo + lane; j < hi; j += 32)
            most = fmaxf(most, fabsf(to_f<T>(w[row * a.w_stride + j])));
#pragma unroll
        for (int m = 16; m; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
        const bf16 sc = __float2bfloat16_rn(__fdiv_rn(most, 7.f));
        if (lane == 0)
          out[sh.scale_at(tile, r, lo / sh.group)] = sc;
        if (lane / 4 == (r & 7)) {
          if (r < 8) scale[gi & 1][0] = __bfloat162float(sc);
          else scale[gi & 1][1] = __bfloat162float(sc);
        }
      }
    }
    for (int unit = s0 / kUnit; unit < sh.units && unit * kUnit < s0 + span; ++unit) {
      uint32_t word[4];
#pragma unroll
      for (int step = 0; step < 4; ++step) {
        word[step] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          int r, in;
          nibble_place(lane, step, i, r, in);
          in += unit * kUnit;
          const long long row = static_cast<long long>(tile) * kTileRows + r;
          const float s = scale[((in - s0) / sh.group) & 1][r >> 3];
          int c = 8;
          if (row < sh.n && in < sh.k && s > 0.f)
            c = 8 + static_cast<int>(fminf(
                        fmaxf(rintf(__fdiv_rn(to_f<T>(w[row * a.w_stride + in]), s)), -8.f), 7.f));
          word[step] |= static_cast<uint32_t>(c) << (4 * i);
        }
      }
      static_cast<uint4*>(a.packed)[(static_cast<long long>(tile) * sh.units + unit) * 32 + lane] =
          make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
}

// ------------------------------------------------------------------- product
struct W4Args {
  W4Shape sh;
  int rows;  // of this launch, at most 8 NT
  int cluster;
  int whole;  // tiles that one warp each takes; the rest are taken by
  int split;  // this many warps each
  const void* packed;
  const void* x;
  long long x_stride;
  void* y;
  long long y_stride;
};

constexpr int kW4Threads = 512;
constexpr int kW4Warps = kW4Threads / 32;
// Units on their way to a warp, and CTAs an SM: with one column tile, 64
// registers and 32 warps an SM; with more, half the warps and more ahead.
template <int NT>
struct W4Tune {
  static constexpr int AHEAD = NT == 1 ? 4 : NT == 2 ? 8 : 6;
  static constexpr int CTAS = NT == 1 ? 2 : 1;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Pairs of codes - 8, exact: 0x4300 is 128 in bf16, whose last bit is 1.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(v) : "r"(w >> (4 * i)));
    asm("sub.bf16x2 %0, %1, %2;" : "=r"(a[i]) : "r"(v), "r"(0x43084308u));
  }
}

// x in shared memory, as the products' right operand: [unit][part][half][row][t][16
// bytes], 16 bytes being the four registers of lane (row, t) for the two
// 16-input steps of half a unit.  A lane whose column is past the last row
// reads the last row again; its column of the result is not used.
template <typename TX, int PARTS>
__device__ __forceinline__ void stage_x(const W4Args& a, uint32_t* xs, int unit0, int units) {
  const int eights = units * (kUnit / 8);  // a thread takes eight inputs of a row
  const TX* x = static_cast<const TX*>(a.x);
  const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                    a.x_stride * static_cast<long long>(sizeof(TX)) % 16 == 0;
  for (int r = 0; r < a.rows; ++r)
    for (int i = threadIdx.x; i < eights; i += blockDim.x) {
      const int unit = i / 8, in = i % 8 * 8;  // of the unit
      const int j = (unit0 + unit) * kUnit + in;
      const TX* from = x + r * a.x_stride + j;
      float v[8];
      if (wide && j + 8 <= a.sh.k) {
        if constexpr (sizeof(TX) == 4) {
          const float4 lo = __ldg(reinterpret_cast<const float4*>(from));
          const float4 hi = __ldg(reinterpret_cast<const float4*>(from) + 1);
          v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
          v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        } else {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(from));
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = j + e < a.sh.k ? to_f<TX>(from[e]) : 0.f;
      }
      const int half = in / 32, reg = in / 16 % 2 * 2 + in / 8 % 2;
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        uint32_t* to = xs + (((unit * PARTS + part) * 2 + half) * a.rows + r) * 16 + reg;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t word = pack_bf16x2(v[2 * t], v[2 * t + 1]);
          to[t * 4] = word;
          if (part + 1 < PARTS) {
            v[2 * t] -= __uint_as_float(word << 16);
            v[2 * t + 1] -= __uint_as_float(word & 0xffff0000u);
          }
        }
      }
    }
}

// y[r, i]: rows r in columns of the products, outputs i in their rows.  A
// cluster holds x once, each CTA a range of the inputs.  Most tiles are a
// warp's own; the last ones, fewer than there are warps, are shared by `split`
// warps each, a range of the CTA's inputs to a warp.  Partial results meet in
// shared memory and are added in the order of the inputs.
template <typename TX, typename TY, int NT, int GROUP>
__global__ void __launch_bounds__(kW4Threads, W4Tune<NT>::CTAS)
    w4_linear_kernel(const __grid_constant__ W4Args a) {
  constexpr int PARTS = sizeof(TX) == 4 ? 3 : 1;
  constexpr int GRAIN = GROUP > kUnit ? GROUP / kUnit : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int cluster = a.cluster, rank = cluster > 1 ? cluster_ctarank() : 0;
  const W4Shape sh = a.sh;
  // Ranges of inputs start at whole groups: pairs of units for groups of 128.
  auto range = [&](int units, int parts, int i, int& lo, int& hi) {
    const int per = ((units + GRAIN - 1) / GRAIN + parts - 1) / parts * GRAIN;
    lo = min(i * per, units);
    hi = min(lo + per, units);
  };
  int u0, u1, none, longest;
  range(sh.units, cluster, rank, u0, u1);
  range(sh.units, cluster, 0, none, longest);  // partial results start alike in all CTAs
  uint32_t* xs = reinterpret_cast<uint32_t*>(smem);
  float* partial = reinterpret_cast<float*>(
      smem + static_cast<size_t>(longest) * PARTS * a.rows * (kUnit * 2));
  grid_dep_wait();
  grid_dep_launch();
  stage_x<TX, PARTS>(a, xs, u0, u1 - u0);
  __syncthreads();

  const int clusters = gridDim.x / cluster, me = blockIdx.x / cluster;
  const uint4* codes = static_cast<const uint4*>(a.packed) + lane;
  const uint32_t* scales =
      reinterpret_cast<const uint32_t*>(static_cast<const char*>(a.packed) + sh.code_bytes()) +
      g * (GROUP == 32 ? 2 : 1);
  const uint4* xl = reinterpret_cast<const uint4*>(xs) + t;
  int xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xrow[nt] = min(nt * 8 + g, a.rows - 1) * 4;
  TY* y = static_cast<TY*>(a.y);

  // a warp's part of a tile: `units` units from v0 of the CTA's range
  auto product = [&](int tile, int v0, int units, float (&sum)[NT][4]) {
    constexpr int AHEAD = W4Tune<NT>::AHEAD, WORDS = GROUP == 32 ? 2 : 1;
    const uint4* src = codes + (static_cast<long long>(tile) * sh.units + u0 + v0) * 32;
    const uint32_t* sc = scales + (static_cast<long long>(tile) * sh.words * 8 +
                                   (u0 + v0) * (GROUP == 32 ? 16 : GROUP == 64 ? 8 : 4));
    const uint4* xu = xl + v0 * (PARTS * 2) * a.rows * 4;
    uint4 code[AHEAD];
    uint32_t scale[GROUP == 128 ? AHEAD / 2 : AHEAD][WORDS];
    // a unit's codes, and scales where it starts a group
    auto fetch = [&](int i, int ahead) {
      code[i] = __ldcs(src + (i + ahead) * 32);
      if constexpr (GROUP == 32) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(sc + (i + ahead) * 16));
        scale[i][0] = v.x;
        scale[i][1] = v.y;
      } else if constexpr (GROUP == 64) {
        scale[i][0] = __ldcs(sc + (i + ahead) * 8);
      } else if (i % 2 == 0) {
        scale[i / 2][0] = __ldcs(sc + (i + ahead) * 4);
      }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (i < units) fetch(i, 0);
    float acc[NT][4];
    for (int base = 0; base < units; base += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (base + i >= units) break;
        const uint32_t word[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
        const uint32_t sc2[2] = {scale[GROUP == 128 ? i / 2 : i][0],
                                 scale[GROUP == 128 ? i / 2 : i][WORDS - 1]};
        if (base + i + AHEAD < units) {
          if (GROUP == 128 && i % 2 == 0) code[i] = __ldcs(src + (i + AHEAD) * 32);
          else fetch(i, AHEAD);
          // a pair's scale is still needed by its second unit
          if (GROUP == 128 && i % 2 == 1) scale[i / 2][0] = __ldcs(sc + (i - 1 + AHEAD) * 4);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a0[4], a1[4];
          codes_to_bf16(word[2 * half], a0);
          codes_to_bf16(word[2 * half + 1], a1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (GROUP == 32 || (half == 0 && (GROUP == 64 || i % 2 == 0)))
              acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              const uint4 b = xu[(part * 2 + half) * a.rows * 4 + xrow[nt]];
              mma_bf16(acc[nt], a0, b.x, b.y);
              mma_bf16(acc[nt], a1, b.z, b.w);
            }
          }
          // the scales of a group whose last product this was
          if (GROUP == 32 || (half == 1 && (GROUP == 64 || i % 2 == 1))) {
            const float lo = __uint_as_float(sc2[half] << 16);
            const float hi = __uint_as_float(sc2[half] & 0xffff0000u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              sum[nt][0] = fmaf(acc[nt][0], lo, sum[nt][0]);
              sum[nt][1] = fmaf(acc[nt][1], lo, sum[nt][1]);
              sum[nt][2] = fmaf(acc[nt][2], hi, sum[nt][2]);
              sum[nt][3] = fmaf(acc[nt][3], hi, sum[nt][3]);
            }
          }
        }
        xu += PARTS * 2 * a.rows * 4;
      }
      src += AHEAD * 32;
      sc += AHEAD * (GROUP == 32 ? 16 : GROUP == 64 ? 8 : 4);
    }
  };
  auto store = [&](int r, int i, float v) {
    if (r < a.rows && i < sh.n) y[r * a.y_stride + i] = from_f<TY>(v);
  };
  // where partial results meet: those of `split` warps a tile
  auto meet = [&](int round, int split, const float (&sum)[NT][4]) {
    // partial[warp][nt * 8 + column][16 outputs]
    float* own = partial + warp * (NT * 128);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        own[(nt * 8 + 2 * t + (e & 1)) * 16 + g + (e >> 1) * 8] = sum[nt][e];
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
    // this CTA's share of the cluster's results
    const int results = kW4Warps / split * (NT * 128);
    for (int z = rank * kW4Threads + static_cast<int>(threadIdx.x); z < results;
         z += cluster * kW4Threads) {
      const int w = z / (NT * 128), r = z / 16 % (NT * 8), i = (round + w) * kTileRows + z % 16;
      if (r >= a.rows) continue;
      float v = 0.f;
      for (int c = 0; c < cluster; ++c) {
        const float* from = partial + w * split * (NT * 128) + z % (NT * 128);
        if (cluster > 1) from = cluster_pointer(from, c);
        for (int s = 0; s < split; ++s) v += from[s * (NT * 128)];
      }
      store(r, i, v);
    }
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
  };
  // whole tiles first, then the shared ones
  int split = 1, end = a.whole, round = me * kW4Warps;
  int v0 = 0, v1 = u1 - u0;
  while (true) {
    if (round >= end) {
      if (end == sh.tiles) break;
      split = a.split;
      end = sh.tiles;
      round = a.whole + me * (kW4Warps / split);
      range(u1 - u0, split, warp % split, v0, v1);
      continue;
    }
    const int tile = round + warp / split;
    float sum[NT][4] = {};
    if (tile < end) product(tile, v0, v1 - v0, sum);
    if (cluster > 1 || split > 1) {
      meet(round, split, sum);
    } else if (tile < end) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          store(nt * 8 + 2 * t + (e & 1), tile * kTileRows + g + (e >> 1) * 8, sum[nt][e]);
    }
    round += clusters * (kW4Warps / split);
  }
}

struct W4Plan {
  int cluster, whole, split, ctas;
  size_t smem;
};
constexpr size_t kW4MostShared = 220 * 1024;

static int w4_grain(const W4Shape& sh) { return sh.group > kUnit ? sh.group / kUnit : 1; }
static int w4_longest(const W4Shape& sh, int units, int parts) {
  const int grain = w4_grain(sh);
  return ((units + grain - 1) / grain + parts - 1) / parts * grain;
}
static size_t w4_held(const W4Shape& sh, int rows, int parts, int nt, int cluster) {
  return static_cast<size_t>(w4_longest(sh, sh.units, cluster)) * parts * rows * (kUnit * 2) +
         static_cast<size_t>(kW4Warps) * nt * 128 * 4;
}

// Steps that the slowest warp takes, in units: rounds of whole tiles, then
// rounds of shared ones, each with what meeting costs; and the time that x
// takes into shared memory.  The cheapest of the few choices is taken.
static W4Plan w4_plan(const W4Shape& sh, int rows, int parts, int nt, int sms) {
  W4Plan best = {};
  double least = 1e30;
  for (int cluster = 1; cluster <= 8; cluster *= 2) {
    const size_t held = w4_held(sh, rows, parts, nt, cluster);
    const int per_sm = nt == 1 && held <= kW4MostShared / 2 ? 2 : 1;
    if (held > kW4MostShared) continue;
    const int most = per_sm * sms / cluster;  // clusters
    const int units = w4_longest(sh, sh.units, cluster);
    const long long warps = static_cast<long long>(most) * kW4Warps;
    const int full = static_cast<int>(sh.tiles / warps);
    const long long left = sh.tiles - full * warps;
    for (int split = 1; split <= kW4Warps; split *= 2) {
      const int at_once = kW4Warps / split;
      const long long groups = (left + at_once - 1) / at_once;
      const long long rounds = (groups + most - 1) / most;
      const double meet = cluster > 1 ? 6.0 : 3.0;
      const double cost = full * (units + (cluster > 1 ? meet : 0.0)) +
                          rounds * (w4_longest(sh, units, split) + meet) +
                          static_cast<double>(held) / 8192.0;
      if (cost < least) {
        least = cost;
        const long long ctas = full ? most : std::min<long long>(groups, most);
        best = W4Plan{cluster, static_cast<int>(full * warps), split,
                      static_cast<int>(ctas) * cluster, held};
      }
    }
  }
  return best;
}

template <typename TX, typename TY, int NT, int GROUP>
static cudaError_t launch_w4(W4Args a, int sms, cudaStream_t s) {
  const W4Plan p = w4_plan(a.sh, a.rows, sizeof(TX) == 4 ? 3 : 1, NT, sms);
  if (p.ctas == 0) return cudaErrorInvalidValue;  // not reached: w4_rows_at_once
  a.cluster = p.cluster;
  a.whole = p.whole;
  a.split = p.split;
  auto kernel = w4_linear_kernel<TX, TY, NT, GROUP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(p.smem));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(p.ctas), dim3(kW4Threads), p.smem, s, p.cluster, a);
}
template <typename TX, typename TY, int NT>
static cudaError_t launch_w4(const W4Args& a, int sms, cudaStream_t s) {
  return a.sh.group == 32   ? launch_w4<TX, TY, NT, 32>(a, sms, s)
         : a.sh.group == 64 ? launch_w4<TX, TY, NT, 64>(a, sms, s)
                            : launch_w4<TX, TY, NT, 128>(a, sms, s);
}

// Rows of one pass over the weights: what 32 columns of products take and the
// shared memory of a cluster of eight holds.
static int w4_rows_at_once(const W4Shape& sh, int parts) {
  int rows = 32;
  while (rows > 1 &&
         w4_held(sh, rows, parts, rows <= 8 ? 1 : rows <= 16 ? 2 : 4, 8) > kW4MostShared)
    rows /= 2;
  return rows;
}

template <typename TX, typename TY>
static cudaError_t run_w4(W4Args a, int sms, cudaStream_t s) {
  const int most = w4_rows_at_once(a.sh, sizeof(TX) == 4 ? 3 : 1), all = a.rows;
  for (int r = 0; r < all; r += most) {
    W4Args b = a;
    b.rows = std::min(most, all - r);
    b.x = static_cast<const TX*>(a.x) + r * a.x_stride;
    b.y = static_cast<TY*>(a.y) + r * a.y_stride;
    const cudaError_t e = b.rows <= 8    ? launch_w4<TX, TY, 1>(b, sms, s)
                          : b.rows <= 16 ? launch_w4<TX, TY, 2>(b, sms, s)
                                         : launch_w4<TX, TY, 4>(b, sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

static pe_status w4_sizes(int32_t n, int32_t k, int32_t group) {
  if (n < 1 || k < 1 || (group != 32 && group != 64 && group != 128))
    return PE_ERR_INVALID_ARGUMENT;
  if (k > (1 << 18) || n > (1 << 24)) return PE_ERR_UNSUPPORTED;
  return PE_OK;
}
static bool w4_aligned(const void* p, size_t to) {
  return p && reinterpret_cast<uintptr_t>(p) % to == 0;
}
static cudaError_t w4_sm_count(int& sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return e;
}
// Blocks of eight warps, a warp an item, four blocks an SM at most.
static dim3 pack_grid(long long items, int sms) {
  return dim3(static_cast<unsigned>(std::min<long long>((items + 7) / 8, 4LL * sms)));
}

}  // namespace pe

extern "C" int64_t pe_w4_bytes(int32_t n, int32_t k, int32_t group) {
  if (pe::w4_sizes(n, k, group) != PE_OK) return 0;
  return pe::W4Shape(n, k, group).bytes();
}

extern "C" pe_status pe_w4_pack(const uint8_t* codes, const void* scales, int32_t n, int32_t k,
                                int32_t group, void* packed, void* stream) {
  using namespace pe;
  if (const pe_status st = w4_sizes(n, k, group); st != PE_OK) return st;
  if (!codes || !w4_aligned(scales, 2) || !w4_aligned(packed, 16)) return PE_ERR_INVALID_ARGUMENT;
  W4PackArgs a = {};
  a.sh = W4Shape(n, k, group);
  a.codes = codes;
  a.scales = static_cast<const bf16*>(scales);
  a.packed = packed;
  int sms = 0;
  cudaError_t e = w4_sm_count(sms);
  if (e == cudaSuccess)
    e = launch_pdl(w4_pack_kernel, pack_grid(static_cast<long long>(a.sh.tiles) * a.sh.units, sms),
                   dim3(256), 0, static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

extern "C" pe_status pe_w4_quantize(const void* w, int32_t dtype, int64_t w_stride, int32_t n,
                                    int32_t k, int32_t group, void* packed, void* stream) {
  using namespace pe;
  if (const pe_status st = w4_sizes(n, k, group); st != PE_OK) return st;
  if ((dtype != PE_DTYPE_BF16 && dtype != PE_DTYPE_F32) || w_stride < k ||
      !w4_aligned(w, dtype == PE_DTYPE_F32 ? 4 : 2) || !w4_aligned(packed, 16))
    return PE_ERR_INVALID_ARGUMENT;
  W4PackArgs a = {};
  a.sh = W4Shape(n, k, group);
  a.w = w;
  a.w_stride = w_stride;
  a.packed = packed;
  int sms = 0;
  cudaError_t e = w4_sm_count(sms);
  const int span = std::max(group, kUnit);
  const dim3 grid = pack_grid(static_cast<long long>(a.sh.tiles) * ((k + span - 1) / span), sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = dtype == PE_DTYPE_F32 ? launch_pdl(w4_quantize_kernel<float>, grid, dim3(256), 0, s, a)
                              : launch_pdl(w4_quantize_kernel<bf16>, grid, dim3(256), 0, s, a);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}

extern "C" pe_status pe_w4_linear(const void* packed, int32_t n, int32_t k, int32_t group,
                                  int32_t rows, int32_t x_dtype, const void* x, int64_t x_stride,
                                  int32_t y_dtype, void* y, int64_t y_stride, void* stream) {
  using namespace pe;
  if (const pe_status st = w4_sizes(n, k, group); st != PE_OK) return st;
  const bool xf = x_dtype == PE_DTYPE_F32, yf = y_dtype == PE_DTYPE_F32;
  if ((!xf && x_dtype != PE_DTYPE_BF16) || (!yf && y_dtype != PE_DTYPE_BF16) || (xf && !yf) ||
      rows < 1 || x_stride < k || y_stride < n || !w4_aligned(packed, 16) ||
      !w4_aligned(x, xf ? 4 : 2) || !w4_aligned(y, yf ? 4 : 2))
    return PE_ERR_INVALID_ARGUMENT;
  W4Args a = {};
  a.sh = W4Shape(n, k, group);
  a.rows = rows;
  a.packed = packed;
  a.x = x;
  a.x_stride = x_stride;
  a.y = y;
  a.y_stride = y_stride;
  int sms = 0;
  cudaError_t e = w4_sm_count(sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = xf ? run_w4<float, float>(a, sms, s)
           : yf ? run_w4<bf16, float>(a, sms, s) : run_w4<bf16, bf16>(a, sms, s);
  return e == cudaSuccess ? PE_OK : PE_ERR_CUDA;
}
