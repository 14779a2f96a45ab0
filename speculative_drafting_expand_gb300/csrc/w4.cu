// w4.cu -- products of a few rows with 4-bit weights that have a scale for
// each group of inputs (include/peagle_w4.h).
//
// Packed layout.  The matrix is cut into tiles of 16 rows and units of 64
// inputs (groups of 128: an even number), filled up with zeros.  First the
// codes, [tile][unit][lane][16 bytes]: word j of a lane is its part of the left
// operand of one m16n8k16 product (inputs 16 j .. 16 j + 15 of the unit), so a
// warp reads a unit as one 512-byte line and needs no exchange.  Register i of
// the operand takes nibbles i (low half) and i + 4 (high half) of the word, from
// which a logic operation and an addition make a pair of fp16 numbers code - 8,
// exact.  Then the scales, bf16, rows g and g + 8 of a tile side by side in a
// word, which is what a lane needs of a group: groups of 32, two words a unit,
// [tile][unit][g][2]; of 64, [tile][unit][g]; of 128, [tile][pair of units][g].
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_fp16.h>

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
  int chunk;  // tiles of a cluster that meet at once
  int ring;   // where the warps' rings start in shared memory
  const void* packed;
  const void* x;
  long long x_stride;
  void* y;
  long long y_stride;
};

constexpr int kW4Threads = 512;
constexpr int kW4Warps = kW4Threads / 32;
// CTAs an SM: with one column tile 64 registers and 32 warps an SM, with more
// half the warps.
template <int NT>
struct W4Tune {
  static constexpr int CTAS = NT == 1 ? 2 : 1;
  static constexpr int AHEAD = NT == 1 ? 3 : 4;  // pairs of units in a warp's ring
};
// A ring's slot: a pair of units and their scales.
__host__ __device__ constexpr int w4_slot(int group) {
  return 2 * kUnitBytes + (group == 32 ? 128 : group == 64 ? 64 : 32);
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Pairs of codes - 8 in fp16, exact, by the published method of kernels with 4-bit
// weights, whose constants follow from the format.  0x6400 is 1024, whose last bit
// is 1: the low nibble of each half gives 1024 + code, the next one 1024 + 16 code.
// (bf16 has room for one nibble a half and takes two instructions a pair of
// additions: 115 instructions a unit over a launch instead of 103.)
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&a)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    const uint32_t v = i ? w >> 8 : w;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(lo) : "r"(v));
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(hi) : "r"(v));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(a[2 * i]) : "r"(lo), "r"(0x64086408u));  // - 1032
    asm("fma.rn.f16x2 %0, %1, %2, %3;"  // / 16 - 72
        : "=r"(a[2 * i + 1])
        : "r"(hi), "r"(0x2c002c00u), "r"(0xd480d480u));
  }
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes of a row from element j on, zeros past the last.
template <typename TX>
__device__ __forceinline__ uint4 load_inputs(const TX* from, int j, int k, bool wide) {
  constexpr int E = 16 / static_cast<int>(sizeof(TX));
  if (wide && j + E <= k) return __ldg(reinterpret_cast<const uint4*>(from));
  uint32_t w[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    if constexpr (sizeof(TX) == 4) {
      w[n] = j + n < k ? __float_as_uint(from[n]) : 0u;
    } else {
      const uint32_t lo = j + 2 * n < k ? __bfloat16_as_ushort(from[2 * n]) : 0u;
      const uint32_t hi = j + 2 * n + 1 < k ? __bfloat16_as_ushort(from[2 * n + 1]) : 0u;
      w[n] = lo | hi << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x in shared memory, as the products' right operand: [unit][part][half][row][t][16
// bytes], 16 bytes being the four registers of lane (row, t) for the two
// 16-input steps of half a unit.  A lane whose column is past the last row
// reads the last row again; its column of the result is not used.
// fp16 has bf16's bits and more, but not its range: each row (of this CTA's
// inputs) is multiplied by the power of two, an even one, that brings its
// largest to 2^13 .. 2^15.  fp16 ends on a grid of 2^-24 there, so what is not on it
// is off by 2^-25 at most, 2^-38 of the largest: bf16 elements below 2^-30 of that.
// fp32 x is taken as three fp16 parts, which hold all 24 bits of an element down to
// 2^-14 of the largest and end on the same grid (to go below it takes a further part
// on a grid of its own, a third more products).  16-bit x is put in place as it is
// while the largest are found, and turned there, FLY loads of a thread at a time;
// fp32 x is read twice.
template <typename TX, int PARTS, int FLY>
__device__ __forceinline__ void stage_x(const W4Args& a, uint32_t* xs, int unit0, int units,
                                        uint32_t* largest, float* unscale) {
  constexpr int E = 16 / static_cast<int>(sizeof(TX));  // elements a thread takes at a time
  const int chunks = units * (kUnit / E), all = chunks * a.rows;
  const TX* x = static_cast<const TX*>(a.x);
  const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                    a.x_stride * static_cast<long long>(sizeof(TX)) % 16 == 0;
  // word of the pair of inputs `in` (of its unit) in part 0
  auto place = [&](int r, int unit, int in) {
    return ((unit * PARTS * 2 + in / 32) * a.rows + r) * 16 + in / 2 % 4 * 4 + in / 16 % 2 * 2 +
           in / 8 % 2;
  };
  const int part_words = 2 * a.rows * 16;
  if (threadIdx.x < 32) largest[threadIdx.x] = 0;
  __syncthreads();
  for (int i0 = threadIdx.x - threadIdx.x % 32; i0 < all; i0 += FLY * kW4Threads) {
    uint4 q[FLY];
    int row[FLY], at[FLY];
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      const int i = i0 + f * kW4Threads + static_cast<int>(threadIdx.x) % 32;
      row[f] = i < all ? i / chunks : -1;
      at[f] = (i - row[f] * chunks) * E;
      if (row[f] >= 0)
        q[f] = load_inputs<TX>(x + row[f] * a.x_stride + unit0 * kUnit + at[f],
                               unit0 * kUnit + at[f], a.sh.k, wide);
    }
#pragma unroll
    for (int f = 0; f < FLY; ++f) {
      if (i0 + f * kW4Threads >= all) break;  // (for the whole warp)
      uint32_t top = 0;
      if (row[f] >= 0) {
        const uint32_t w[4] = {q[f].x, q[f].y, q[f].z, q[f].w};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          top = max(top, w[n] & (sizeof(TX) == 4 ? 0x7fffffffu : 0x7fff0000u));
          if constexpr (sizeof(TX) == 2) {
            top = max(top, (w[n] & 0x7fffu) << 16);
            xs[place(row[f], at[f] / kUnit, at[f] % kUnit + 2 * n)] = w[n];
          }
        }
      }
      // mostly a warp's inputs are of one row
      const int r0 = __shfl_sync(0xffffffffu, row[f], 0);
      if (__all_sync(0xffffffffu, row[f] == r0)) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (threadIdx.x % 32 == 0) atomicMax(&largest[r0], top);
      } else if (row[f] >= 0) {
        atomicMax(&largest[row[f]], top);
      }
    }
  }
  __syncthreads();
  // half of the power: its square may be past what fp32 has
  auto half_shift = [&](int r) {
    const int e = static_cast<int>(largest[r] >> 23);
    return e == 255 ? 0 : (14 + 127 - e) >> 1;
  };
  auto scale_of = [&](int r) { return __uint_as_float((127 + half_shift(r)) << 23); };
  if (threadIdx.x < a.rows)
    unscale[threadIdx.x] = __uint_as_float((127 - half_shift(threadIdx.x)) << 23);
  if constexpr (sizeof(TX) == 2) {
    uint4* xq = reinterpret_cast<uint4*>(xs);
    for (int c = threadIdx.x; c < all; c += kW4Threads) {
      const float scale = scale_of(c / 4 % a.rows);
      const uint4 q = xq[c];
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int n = 0; n < 4; ++n)
        w[n] = pack_f16x2(__uint_as_float(w[n] << 16) * scale * scale,
                          __uint_as_float(w[n] & 0xffff0000u) * scale * scale);
      xq[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll 2
    for (int i = threadIdx.x; i < all; i += kW4Threads) {
      const int r = i / chunks, at = (i - r * chunks) * E, j = unit0 * kUnit + at;
      const float scale = scale_of(r);
      const uint4 q = load_inputs<TX>(x + r * a.x_stride + j, j, a.sh.k, wide);
      float v[4] = {__uint_as_float(q.x) * scale * scale, __uint_as_float(q.y) * scale * scale,
                    __uint_as_float(q.z) * scale * scale, __uint_as_float(q.w) * scale * scale};
#pragma unroll
      for (int n = 0; n < 4; n += 2) {
        uint32_t* to = xs + place(r, at / kUnit, at % kUnit + n);
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          const uint32_t word = pack_f16x2(v[n], v[n + 1]);
          to[part * part_words] = word;
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&word));
          v[n] -= f.x;
          v[n + 1] -= f.y;
        }
      }
    }
  }
}

// y[r, i] in 64 bits and from the numbers as they came, by one thread.  For a
// row of finite x whose sum left fp32's range: it is taken of x brought to 2^13
// .. 2^15 and times scales of up to 2^128, so it can where the result itself has
// room (2^17 inputs of weight -8 at most: with scales above 2^92).  No model has
// such scales; what the others pay is a comparison a result when it is stored
// (taking the row's power back before the scale instead costs a multiplication a
// result and group).
template <typename TX, typename TY>
__device__ __noinline__ void store_by_64_bits(const W4Args& a, int r, int i) {
  const W4Shape sh = a.sh;
  const int tile = i / kTileRows, row = i % kTileRows;
  const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
  const uint32_t* codes = static_cast<const uint32_t*>(a.packed);
  const bf16* scales =
      reinterpret_cast<const bf16*>(static_cast<const char*>(a.packed) + sh.code_bytes());
  double sum = 0.0;
  for (int j = 0; j < sh.k; ++j) {
    // (nibble_place, the other way round)
    const int in = j % 16, nibble = (in & 1) * 4 + in / 8 * 2 + (row >> 3);
    const int lane = (row & 7) * 4 + in % 8 / 2;
    const long long word =
        ((static_cast<long long>(tile) * sh.units + j / kUnit) * 32 + lane) * 4 + j % kUnit / 16;
    const int code = static_cast<int>(codes[word] >> (4 * nibble) & 15) - 8;
    const float scale = __bfloat162float(scales[sh.scale_at(tile, row, j / sh.group)]);
    sum += static_cast<double>(to_f<TX>(x[j])) * code * scale;
  }
  static_cast<TY*>(a.y)[r * a.y_stride + i] = from_f<TY>(static_cast<float>(sum));
}

// y[r, i]: rows r in columns of the products, outputs i in their rows.  A
// cluster holds x once, each CTA a range of the inputs, and has a run of tiles.
// The warps of a CTA divide the units of its run evenly: a warp has the end of
// one tile, some whole ones and the start of another.  What does not end where
// a tile ends meets in shared memory and is added in the order of the inputs.
// Products of 8 columns and not tcgen05 tiles: codes would have to be written to
// shared memory as 16-bit operands of 128 rows, four times their bytes, for one
// to eight columns of use.  The codes go from the ring into registers and from
// there into the product; what bounds that is the issue of instructions, in three
// quarters of the slots (201,088 x 2880 in groups of 32, one row: 66 us, 4.92 TB/s,
// 103 warp instructions a unit over the launch; 151,936 x 2048 in groups of 128,
// eight rows: 40 us, 4.2 TB/s, 114 a unit).  64 registers, which two CTAs an SM
// leave a thread, are short: 12 to 76 bytes of them are spilled and loaded again.
// Small matrices are bound by the way from the launch through x and the ring's
// first pairs to the meeting (5120 x 2880, one row: 8.6 us).
template <typename TX, typename TY, int NT, int GROUP>
__global__ void __launch_bounds__(kW4Threads, W4Tune<NT>::CTAS)
    w4_linear_kernel(const __grid_constant__ W4Args a) {
  constexpr int PARTS = sizeof(TX) == 4 ? 3 : 1;
  constexpr int GRAIN = GROUP > kUnit ? GROUP / kUnit : 1;
  constexpr int RES = NT * 128;  // results of a tile
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int cluster = a.cluster, rank = cluster > 1 ? cluster_ctarank() : 0;
  const W4Shape sh = a.sh;
  // Ranges of inputs start at whole groups: pairs of units for groups of 128.
  const int longest = ((sh.units + GRAIN - 1) / GRAIN + cluster - 1) / cluster * GRAIN;
  const int u0 = min(rank * longest, sh.units), units_here = min(longest, sh.units - u0);
  uint32_t* xs = reinterpret_cast<uint32_t*>(smem);
  // (meeting places start alike in all CTAs)
  float* heads = reinterpret_cast<float*>(
      smem + static_cast<size_t>(longest) * PARTS * a.rows * (kUnit * 2));
  float* mains = heads + kW4Warps * RES;  // of warps, or of the cluster's tiles
  constexpr int AHEAD = W4Tune<NT>::AHEAD, SLOT = w4_slot(GROUP);
  unsigned char* ring = smem + a.ring + warp * (AHEAD * SLOT);
  __shared__ uint32_t largest[32];
  __shared__ __align__(8) float unscale[32];
  const int clusters = gridDim.x / cluster, me = blockIdx.x / cluster;
  const uint4* xl = reinterpret_cast<const uint4*>(xs) + t;
  int xrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) xrow[nt] = min(nt * 8 + g, a.rows - 1) * 4;
  TY* y = static_cast<TY*>(a.y);

  bool over = false;  // a result is infinite or NaN
  auto store = [&](int r, int i, float v) {
    if (r < a.rows && i < sh.n) {
      y[r * a.y_stride + i] = from_f<TY>(v);
      over = over || !(fabsf(v) < INFINITY);
    }
  };
  // The same result again, where x is not why
  auto again = [&](int r, int i) {
    if (r >= a.rows || i >= sh.n || fabsf(to_f<TY>(y[r * a.y_stride + i])) < INFINITY) return;
    for (int c = 0; c < cluster; ++c)
      if ((cluster > 1 ? *cluster_pointer(largest + r, c) : largest[r]) >= 0x7f800000u) return;
    store_by_64_bits<TX, TY>(a, r, i);
  };
  // place[column][16 outputs]
  auto put = [&](float* place, const float (&sum)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        place[(nt * 8 + 2 * t + (e & 1)) * 16 + g + (e >> 1) * 8] = sum[nt][e];
  };
  const int run0 = static_cast<int>(static_cast<long long>(sh.tiles) * me / clusters);
  const int run1 = static_cast<int>(static_cast<long long>(sh.tiles) * (me + 1) / clusters);
  for (int tile0 = run0; tile0 < run1; tile0 += a.chunk) {
    const int tiles = min(a.chunk, run1 - tile0);
    // where a warp's units start, counted from the first tile's (fewer than
    // 2^28: 2^20 tiles of all clusters, 2^11 units)
    const unsigned all = static_cast<unsigned>(tiles) * units_here;
    auto start = [&](int w) { return static_cast<int>(all * w / kW4Warps / GRAIN * GRAIN); };
    const int from = start(warp), mine = start(warp + 1) - from;
    int j = from / max(units_here, 1);  // tile of the run
    int v = from - j * units_here;      // its next unit
    bool begun = v > 0;                 // the tile was begun by an earlier warp
    // What is fetched next, in pairs that end where a tile ends: a warp's units
    // come from one run of memory, but for the other CTAs' inputs between tiles.
    const char* code = static_cast<const char*>(a.packed) + lane * 16 +
                       (static_cast<long long>(tile0 + j) * sh.units + u0 + v) * kUnitBytes;
    const char* scale = static_cast<const char*>(a.packed) + sh.code_bytes() + lane * 4 +
                        (static_cast<long long>(tile0 + j) * sh.words +
                         (GROUP == 32 ? 2 * (u0 + v) : GROUP == 64 ? u0 + v : (u0 + v) / 2)) * 32;
    int to_fetch = mine, fv = v;
    if (tile0 == run0) {  // (every run has a tile)
      // here, where the first address is known, and not at the start: a call of
      // 5120 x 2880 takes 8.5 us for 9.4 (the codes' first lines brought into L2
      // before the wait: no change)
      grid_dep_wait();
      grid_dep_launch();
    }
    const uint32_t ring_at = smem_u32(ring);
    uint32_t fill = ring_at;
    auto fetch = [&]() {
      if (to_fetch > 0) {
        const int n = min(min(units_here - fv, to_fetch), 2);
        copy_async16(fill + lane * 16, code);
        if (n == 2) copy_async16(fill + kUnitBytes + lane * 16, code + kUnitBytes);
        constexpr int LANES = GROUP == 32 ? 16 : 8;  // that a unit's scales take
        if (lane < (GROUP == 128 ? LANES : n * LANES))
          copy_async4(fill + 2 * kUnitBytes + lane * 4, scale);
        code += n * kUnitBytes;
        scale += GROUP == 128 ? 32 : n * LANES * 4;
        to_fetch -= n;
        fv += n;
        if (fv == units_here) {
          fv = 0;
          if (cluster > 1) {
            code += static_cast<long long>(sh.units - units_here) * kUnitBytes;
            const int words = GROUP == 32 ? 2 * units_here : GROUP == 64 ? units_here : units_here / 2;
            scale += static_cast<long long>(sh.words - words) * 32;
          }
        }
        fill = fill == ring_at + (AHEAD - 1) * SLOT ? ring_at : fill + SLOT;
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD - 1; ++i) fetch();
    if (tile0 == run0) {
      stage_x<TX, PARTS, NT == 1 ? 2 : 8>(a, xs, u0, units_here, largest, unscale);
      __syncthreads();
    }
    const unsigned char* slot = ring;
    const int xhalf = a.rows * 4;  // 16-byte chunks of half a unit and a part
    const uint4* xu = xl + v * (PARTS * 2) * xhalf;
    float sum[NT][4] = {}, acc[NT][4];
    auto product = [&](const uint4& w4, bool odd, uint32_t s0, uint32_t s1) {
      const uint32_t word[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t a0[4], a1[4];
        codes_to_f16(word[2 * half], a0);
        codes_to_f16(word[2 * half + 1], a1);
        const bool first = GROUP == 32 || (half == 0 && (GROUP == 64 || !odd));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) {
            const uint4 b = xu[(part * 2 + half) * xhalf + xrow[nt]];
            if (first && part == 0) mma_f16_first(acc[nt], a0, b.x, b.y);
            else mma_f16(acc[nt], a0, b.x, b.y);
            mma_f16(acc[nt], a1, b.z, b.w);
          }
        // the scales of a group whose last product this was
        if (GROUP == 32 || (half == 1 && (GROUP == 64 || odd))) {
          const uint32_t s2 = half ? s1 : s0;
          const float lo = __uint_as_float(s2 << 16), hi = __uint_as_float(s2 & 0xffff0000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            sum[nt][0] = fmaf(acc[nt][0], lo, sum[nt][0]);
            sum[nt][1] = fmaf(acc[nt][1], lo, sum[nt][1]);
            sum[nt][2] = fmaf(acc[nt][2], hi, sum[nt][2]);
            sum[nt][3] = fmaf(acc[nt][3], hi, sum[nt][3]);
          }
        }
      }
      xu += PARTS * 2 * xhalf;
    };
    // the scale words of a slot's unit
    auto scale_of = [&](int i, uint32_t& s0, uint32_t& s1) {
      const unsigned char* p = slot + 2 * kUnitBytes;
      if constexpr (GROUP == 32) {
        const uint2 two = reinterpret_cast<const uint2*>(p)[i * 8 + g];
        s0 = two.x;
        s1 = two.y;
      } else {
        s0 = s1 = reinterpret_cast<const uint32_t*>(p)[(GROUP == 64 ? i * 8 : 0) + g];
      }
    };
    for (int left = mine; left > 0;) {
      // the warp's units of tile j
      int units = min(units_here - v, left);
      left -= units;
      v += units;
      for (; units > 0; units -= 2) {
        copy_wait<AHEAD - 2>();
        __syncwarp();
        const uint4 w0 = reinterpret_cast<const uint4*>(slot)[lane];
        uint32_t s0, s1;
        scale_of(0, s0, s1);
        if (GROUP == 128 || units > 1) {
          const uint4 w1 = reinterpret_cast<const uint4*>(slot + kUnitBytes)[lane];
          uint32_t s2, s3;
          scale_of(1, s2, s3);
          fetch();  // into the slot before this one, which every lane has read
          product(w0, false, s0, s1);
          product(w1, true, s2, s3);
        } else {
          fetch();
          product(w0, false, s0, s1);
        }
        slot = slot == ring + (AHEAD - 1) * SLOT ? ring : slot + SLOT;
      }
      // (columns past the last row have no scale, and no use)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 back = *reinterpret_cast<const float2*>(unscale + nt * 8 + 2 * t);
        sum[nt][0] = sum[nt][0] * back.x * back.x;
        sum[nt][1] = sum[nt][1] * back.y * back.y;
        sum[nt][2] = sum[nt][2] * back.x * back.x;
        sum[nt][3] = sum[nt][3] * back.y * back.y;
      }
      if (begun) {
        put(heads + warp * RES, sum);
      } else if (cluster > 1) {
        put(mains + j * RES, sum);
      } else if (v < units_here) {
        put(mains + warp * RES, sum);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            store(nt * 8 + 2 * t + (e & 1), (tile0 + j) * kTileRows + g + (e >> 1) * 8, sum[nt][e]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sum[nt][0] = sum[nt][1] = sum[nt][2] = sum[nt][3] = 0.f;
      ++j;
      v = 0;
      begun = false;
      xu = xl;
    }
    copy_wait<0>();
    __syncthreads();
    if (cluster == 1) {
      // a warp's last tile, where other warps go on with it
      for (int z = threadIdx.x; z < kW4Warps * RES; z += kW4Threads) {
        const int w = z / RES, e = z % RES, r = e / 16;
        const int b0 = start(w), b1 = start(w + 1);
        if (b0 == b1 || r >= a.rows) continue;
        const int jw = b1 / units_here, begin = jw * units_here;
        if (b1 == begin || b0 > begin) continue;  // it ends here, or starts with an earlier warp
        float sumv = mains[z];
        for (int o = w + 1; o < kW4Warps; ++o) {
          const int s0 = start(o);
          if (s0 >= begin + units_here) break;
          if (s0 < start(o + 1)) sumv += heads[o * RES + e];
        }
        store(r, (tile0 + jw) * kTileRows + e % 16, sumv);
      }
      if (__syncthreads_or(over))
        for (int z = threadIdx.x; z < tiles * RES; z += kW4Threads)
          again(z % RES / 16, (tile0 + z / RES) * kTileRows + z % 16);
    } else {
      // tiles in one piece, then the pieces of all ranges of the inputs
      if (units_here == 0)
        for (int z = threadIdx.x; z < tiles * RES; z += kW4Threads) mains[z] = 0.f;
      for (int o = 1; o < kW4Warps && units_here; ++o) {
        const int b0 = start(o);
        if (b0 < start(o + 1) && b0 % units_here)
          for (int e = threadIdx.x; e < RES; e += kW4Threads)
            mains[b0 / units_here * RES + e] += heads[o * RES + e];
      }
      cluster_barrier();
      for (int z = rank * kW4Threads + static_cast<int>(threadIdx.x); z < tiles * RES;
           z += cluster * kW4Threads) {
        const int e = z % RES, r = e / 16;
        if (r >= a.rows) continue;
        float sumv = 0.f;
        for (int c = 0; c < cluster; ++c) sumv += *cluster_pointer(mains + z, c);
        store(r, (tile0 + z / RES) * kTileRows + e % 16, sumv);
      }
      if (over)  // this thread's own
        for (int z = rank * kW4Threads + static_cast<int>(threadIdx.x); z < tiles * RES;
             z += cluster * kW4Threads)
          again(z % RES / 16, (tile0 + z / RES) * kTileRows + z % 16);
      cluster_barrier();
    }
    __syncthreads();
  }
}

struct W4Plan {
  int cluster, chunk, ctas;
  size_t smem;
};
constexpr size_t kW4MostShared = 220 * 1024;
// tiles that a cluster's CTAs put together at once
static int w4_chunk(int nt) { return 32 / nt; }

// Shared memory: x, the places where results meet, the warps' rings.
static size_t w4_ring_at(const W4Shape& sh, int rows, int parts, int nt, int cluster) {
  const int grain = sh.group > kUnit ? sh.group / kUnit : 1;
  const int longest = ((sh.units + grain - 1) / grain + cluster - 1) / cluster * grain;
  return static_cast<size_t>(longest) * parts * rows * (kUnit * 2) +
         static_cast<size_t>(kW4Warps + (cluster > 1 ? w4_chunk(nt) : kW4Warps)) * nt * 128 * 4;
}
static size_t w4_held(const W4Shape& sh, int rows, int parts, int nt, int cluster) {
  return w4_ring_at(sh, rows, parts, nt, cluster) +
         static_cast<size_t>(kW4Warps) * w4_slot(sh.group) *
             (nt == 1 ? W4Tune<1>::AHEAD : nt == 2 ? W4Tune<2>::AHEAD : W4Tune<4>::AHEAD);
}

// Clusters of one kernel that are resident at a time: a GPC's SMs need not be a
// multiple of the cluster.  Asked once a process, device and shape.
template <typename TX, typename TY, int NT, int GROUP>
static int resident_clusters(int cluster, int per_sm, size_t smem, int sms) {
  if (cluster == 1) return per_sm * sms;
  static std::atomic<int> known[16][2][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const int c = cluster == 2 ? 1 : cluster == 4 ? 2 : 3;
  std::atomic<int>* place = dev < 16 ? &known[dev][per_sm - 1][c] : nullptr;
  int n = place ? place->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  auto kernel = w4_linear_kernel<TX, TY, NT, GROUP>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kW4Threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kW4MostShared)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
    n = std::max(1, per_sm * sms / cluster / 2);
  else if (place)
    place->store(n, std::memory_order_relaxed);
  return n;
}

// The time that the busiest CTA takes, by the number of CTAs that share the
// inputs, in microseconds as measured (0.3 a unit of each of its warps, 32 KB of
// x into shared memory in one, 1.5 a meeting of a cluster): the cheapest of the
// four choices is taken.
template <typename TX, typename TY, int NT, int GROUP>
static W4Plan w4_plan(const W4Shape& sh, int rows, int sms) {
  constexpr int nt = NT, parts = sizeof(TX) == 4 ? 3 : 1;
  W4Plan best = {};
  double least = 1e30;
  for (int cluster = 1; cluster <= 8; cluster *= 2) {
    const size_t held = w4_held(sh, rows, parts, nt, cluster);
    if (held > kW4MostShared) continue;
    const int per_sm = nt == 1 && held <= kW4MostShared / 2 ? 2 : 1;
    const int most = resident_clusters<TX, TY, NT, GROUP>(cluster, per_sm, held, sms);
    const int tiles = (sh.tiles + most - 1) / most;        // of a cluster
    // few tiles: no more clusters than it takes for every one to have as many
    const int clusters = tiles > 4 ? std::min(most, sh.tiles) : (sh.tiles + tiles - 1) / tiles;
    const double units = static_cast<double>(tiles) * ((sh.units + cluster - 1) / cluster);
    const double share = std::max(1.0, static_cast<double>(clusters) * cluster / sms);
    const double x = static_cast<double>(sh.k) / cluster * parts * rows * 2;
    const double cost = std::ceil(units / kW4Warps) * 0.3 * share + x / 32768.0 +
                        (cluster > 1 ? 1.5 * ((tiles + w4_chunk(nt) - 1) / w4_chunk(nt)) : 0.0);
    if (cost < least) {
      least = cost;
      best = W4Plan{cluster, cluster > 1 ? w4_chunk(nt) : tiles, clusters * cluster, held};
    }
  }
  return best;
}

template <typename TX, typename TY, int NT, int GROUP>
static cudaError_t launch_w4(W4Args a, int sms, cudaStream_t s) {
  const W4Plan p = w4_plan<TX, TY, NT, GROUP>(a.sh, a.rows, sms);
  if (p.ctas == 0) return cudaErrorInvalidValue;  // not reached: w4_rows_at_once
  a.cluster = p.cluster;
  a.chunk = p.chunk;
  a.ring = static_cast<int>(w4_ring_at(a.sh, a.rows, sizeof(TX) == 4 ? 3 : 1, NT, p.cluster));
  auto kernel = w4_linear_kernel<TX, TY, NT, GROUP>;
  // (always the same limit: another thread's call may lie between this and the launch)
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kW4MostShared));
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
  if (k > (1 << 17) || n > (1 << 24)) return PE_ERR_UNSUPPORTED;
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
