// w4.cu -- products of a few rows with 4-bit weights that have a scale for
// each group of inputs (include/peagle_w4.h).
//
// Packed layout.  The matrix is cut into tiles of 16 rows and units of 64
// inputs, filled up with zeros.  First the codes, [tile][unit][lane][16
// bytes]: word j of a lane is its part of the left operand of one m16n8k16
// product (inputs 16 j .. 16 j + 15 of the unit), so a warp reads a unit as
// one 512-byte line and needs no exchange.  Register i of the operand takes
// nibbles i (low half) and i + 4 (high half) of the word: one shift and one
// logic operation make a pair of bf16 numbers 128 + code, one subtraction the
// exact pair code - 8.  Then the scales, [tile][group][16 rows] bf16, rows g
// and g + 8 side by side, which is what a lane needs.
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
  __host__ __device__ W4Shape() {}
  __host__ __device__ W4Shape(int n_, int k_, int group_)
      : n(n_), k(k_), group(group_), tiles((n_ + kTileRows - 1) / kTileRows),
        units((k_ + kUnit - 1) / kUnit), groups((k_ + group_ - 1) / group_) {}
  __host__ __device__ long long code_bytes() const {
    return static_cast<long long>(tiles) * units * kUnitBytes;
  }
  __host__ __device__ long long bytes() const {
    return code_bytes() + static_cast<long long>(tiles) * groups * (kTileRows * 2);
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
  const long long all = static_cast<long long>(sh.tiles) * sh.groups * kTileRows;
  for (long long i = first * 32 + lane; i < all; i += warps * 32) {
    const int r = static_cast<int>(i % kTileRows);
    const long long tg = i / kTileRows;
    const int group = static_cast<int>(tg % sh.groups);
    const long long row = tg / sh.groups * kTileRows + (r >> 1) + (r & 1) * 8;
    out[i] = row < sh.n ? a.scales[row * sh.groups + group] : __float2bfloat16_rn(0.f);
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
    const int s1 = min(s0 + span, sh.k);
    float scale[2][2] = {};  // rows g and g + 8 of up to two groups of the span
    for (int r = 0; r < kTileRows; ++r) {
      const long long row = static_cast<long long>(tile) * kTileRows + r;
      for (int gi = 0; s0 + gi * sh.group < s1; ++gi) {
        const int lo = s0 + gi * sh.group, hi = min(lo + sh.group, sh.k);
        float most = 0.f;
        if (row < sh.n)
          for (int j = lo + lane; j < hi; j += 32)
            most = fmaxf(most, fabsf(to_f<T>(w[row * a.w_stride + j])));
#pragma unroll
        for (int m = 16; m; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
        const bf16 sc = __float2bfloat16_rn(__fdiv_rn(most, 7.f));
        if (lane == 0)
          out[(static_cast<long long>(tile) * sh.groups + lo / sh.group) * kTileRows +
              2 * (r & 7) + (r >> 3)] = sc;
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
  int split;  // warps that share a tile's inputs
  const void* packed;
  const void* x;
  long long x_stride;
  void* y;
  long long y_stride;
};

constexpr int kW4Threads = 256;
constexpr int kW4Warps = kW4Threads / 32;
constexpr int kW4Ahead = 4;  // units on their way to a warp

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
  const int pairs = units * (kUnit / 2);
  const TX* x = static_cast<const TX*>(a.x);
  for (int i = threadIdx.x; i < pairs * a.rows; i += blockDim.x) {
    const int r = i / pairs, pr = i % pairs;
    const int unit = pr / 32, in = pr % 32 * 2;  // of the unit
    const long long j = static_cast<long long>(unit0 + unit) * kUnit + in;
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) v[e] = j + e < a.sh.k ? to_f<TX>(x[r * a.x_stride + j + e]) : 0.f;
    const int step = in / 16, t = in % 8 / 2, reg = in % 16 / 8;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      const uint32_t word = pack_bf16x2(v[0], v[1]);
      v[0] -= __uint_as_float(word << 16);
      v[1] -= __uint_as_float(word & 0xffff0000u);
      xs[((((unit * PARTS + part) * 2 + step / 2) * a.rows + r) * 4 + t) * 4 + step % 2 * 2 + reg] =
          word;
    }
  }
}

// y[r, i]: rows r in columns of the products, outputs i in their rows.  A
// cluster holds x once, each CTA a range of the inputs; in a CTA `split` warps
// share a tile's range, and the other warps take other tiles.  Partial
// results meet in shared memory and are added in the order of the inputs.
template <typename TX, typename TY, int NT>
__global__ void __launch_bounds__(kW4Threads) w4_linear_kernel(const __grid_constant__ W4Args a) {
  constexpr int PARTS = sizeof(TX) == 4 ? 3 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int cluster = a.cluster, rank = cluster > 1 ? cluster_ctarank() : 0;
  const W4Shape sh = a.sh;
  // Ranges of inputs start at whole groups: pairs of units for groups of 128.
  const int grain = sh.group > kUnit ? sh.group / kUnit : 1;
  auto range = [&](int units, int parts, int i, int& lo, int& hi) {
    const int per = ((units + grain - 1) / grain + parts - 1) / parts * grain;
    lo = min(i * per, units);
    hi = min(lo + per, units);
  };
  int u0, u1;
  range(sh.units, cluster, rank, u0, u1);
  const int split = a.split, tiles_at_once = kW4Warps / split;
  int v0, v1;
  range(u1 - u0, split, warp % split, v0, v1);
  v0 += u0;
  v1 += u0;
  uint32_t* xs = reinterpret_cast<uint32_t*>(smem);
  grid_dep_wait();
  grid_dep_launch();
  stage_x<TX, PARTS>(a, xs, u0, u1 - u0);
  int longest, none;  // the first range: partial results start alike in all CTAs
  range(sh.units, cluster, 0, none, longest);
  float* partial = reinterpret_cast<float*>(
      smem + static_cast<size_t>(longest) * PARTS * a.rows * (kUnit * 2));
  __syncthreads();

  const int clusters = gridDim.x / cluster, me = blockIdx.x / cluster;
  const uint4* codes = static_cast<const uint4*>(a.packed);
  const uint32_t* scales = reinterpret_cast<const uint32_t*>(
      static_cast<const char*>(a.packed) + sh.code_bytes());
  const bool meet = split > 1 || cluster > 1;
  const int steps = sh.group / 16;  // products of a group
  for (int round = me * tiles_at_once; round < sh.tiles; round += clusters * tiles_at_once) {
    const int tile = round + warp / split;
    float sum[NT][4] = {};
    if (tile < sh.tiles) {
      const uint4* src = codes + static_cast<long long>(tile) * sh.units * 32 + lane;
      const uint32_t* sc = scales + static_cast<long long>(tile) * sh.groups * 8 + g;
      uint4 ahead[kW4Ahead];
#pragma unroll
      for (int i = 0; i < kW4Ahead; ++i)
        if (v0 + i < v1) ahead[i] = __ldcs(src + (v0 + i) * 32);
      float acc[NT][4] = {};
      for (int base = v0; base < v1; base += kW4Ahead) {
#pragma unroll
        for (int i = 0; i < kW4Ahead; ++i) {
          const int unit = base + i;
          if (unit >= v1) break;
          const uint4 w4 = ahead[i];
          if (unit + kW4Ahead < v1) ahead[i] = __ldcs(src + (unit + kW4Ahead) * 32);
          const uint32_t word[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t a0[4], a1[4];
            codes_to_bf16(word[2 * half], a0);
            codes_to_bf16(word[2 * half + 1], a1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int part = 0; part < PARTS; ++part) {
                const int r = min(nt * 8 + g, a.rows - 1);
                const uint4 b = *reinterpret_cast<const uint4*>(
                    xs + (((((unit - u0) * PARTS + part) * 2 + half) * a.rows + r) * 4 + t) * 4);
                mma_bf16(acc[nt], a0, b.x, b.y);
                mma_bf16(acc[nt], a1, b.z, b.w);
              }
            const int done = unit * 4 + half * 2 + 2;
            if (done % steps == 0 || (half == 1 && unit + 1 == v1)) {
              // the group's scales, once its last product is in
              const int group = min((done - 1) / steps, sh.groups - 1);
              const uint32_t s2 = sc[group * 8];
              const float lo = __uint_as_float(s2 << 16), hi = __uint_as_float(s2 & 0xffff0000u);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                sum[nt][0] = fmaf(acc[nt][0], lo, sum[nt][0]);
                sum[nt][1] = fmaf(acc[nt][1], lo, sum[nt][1]);
                sum[nt][2] = fmaf(acc[nt][2], hi, sum[nt][2]);
                sum[nt][3] = fmaf(acc[nt][3], hi, sum[nt][3]);
                acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
              }
            }
          }
        }
      }
    }
    TY* y = static_cast<TY*>(a.y);
    if (!meet) {
      if (tile < sh.tiles)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = nt * 8 + 2 * t + (e & 1), i = tile * kTileRows + g + (e >> 1) * 8;
            if (r < a.rows && i < sh.n) y[r * a.y_stride + i] = from_f<TY>(sum[nt][e]);
          }
      continue;
    }
    // partial[warp][nt * 8 + column][16 outputs]
    float* own = partial + warp * (NT * 128);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        own[(nt * 8 + 2 * t + (e & 1)) * 16 + g + (e >> 1) * 8] = sum[nt][e];
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();
    // this CTA's share of the cluster's results
    const int results = tiles_at_once * NT * 128;
    for (int z = rank * kW4Threads + static_cast<int>(threadIdx.x); z < results;
         z += cluster * kW4Threads) {
      const int w = z / (NT * 128), r = z / 16 % (NT * 8), i = (round + w) * kTileRows + z % 16;
      float v = 0.f;
      for (int c = 0; c < cluster; ++c)
        for (int s = 0; s < split; ++s) {
          float* from = partial + (w * split + s) * (NT * 128) + z % (NT * 128);
          v += cluster > 1 ? ld_shared_cluster_f32(cluster_map_shared(smem_u32(from), c)) : *from;
        }
      if (r < a.rows && i < sh.n) y[r * a.y_stride + i] = from_f<TY>(v);
    }
    if (cluster > 1) cluster_sync_all();
    else __syncthreads();
  }
}

struct W4Plan {
  int cluster, split, ctas;
  size_t smem;
};
constexpr size_t kW4MostShared = 220 * 1024;

// Enough CTAs a cluster that x fits beside the partial results; then as many
// warps a tile as keep every warp of the GPU busy.
static W4Plan w4_plan(const W4Shape& sh, int rows, int parts, int nt, int sms) {
  const int grain = sh.group > kUnit ? sh.group / kUnit : 1;
  const size_t meet = static_cast<size_t>(kW4Warps) * nt * 128 * 4;
  auto held = [&](int cluster) {
    const int per = ((sh.units + grain - 1) / grain + cluster - 1) / cluster * grain;
    return static_cast<size_t>(per) * parts * rows * (kUnit * 2) + meet;
  };
  W4Plan p = {1, 1, 0, 0};
  while (p.cluster < 8 && held(p.cluster) > kW4MostShared / 2) p.cluster *= 2;
  p.smem = held(p.cluster);
  const int per_sm = p.smem <= kW4MostShared / 2 ? 2 : 1;
  const int most = per_sm * sms / p.cluster * p.cluster;
  while (p.split < kW4Warps &&
         static_cast<long long>(sh.tiles) * p.split * 2 <= static_cast<long long>(most) / p.cluster * kW4Warps)
    p.split *= 2;
  const int at_once = kW4Warps / p.split;
  const long long want = static_cast<long long>((sh.tiles + at_once - 1) / at_once) * p.cluster;
  p.ctas = static_cast<int>(std::min<long long>(want, most));
  return p;
}

template <typename TX, typename TY, int NT>
static cudaError_t launch_w4(W4Args a, int sms, cudaStream_t s) {
  const W4Plan p = w4_plan(a.sh, a.rows, sizeof(TX) == 4 ? 3 : 1, NT, sms);
  if (p.smem > kW4MostShared) return cudaErrorInvalidValue;
  a.cluster = p.cluster;
  a.split = p.split;
  auto kernel = w4_linear_kernel<TX, TY, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(p.smem));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(p.ctas), dim3(kW4Threads), p.smem, s, p.cluster, a);
}

// Rows of one pass over the weights: what 32 columns of products take and the
// shared memory of a cluster of eight holds.
static int w4_rows_at_once(const W4Shape& sh, int parts) {
  int rows = 32;
  auto held = [&](int r) {
    const int grain = sh.group > kUnit ? sh.group / kUnit : 1;
    const int per = ((sh.units + grain - 1) / grain + 7) / 8 * grain;
    return static_cast<size_t>(per) * parts * r * (kUnit * 2) +
           static_cast<size_t>(kW4Warps) * (r <= 8 ? 1 : r <= 16 ? 2 : 4) * 512;
  };
  while (rows > 1 && held(rows) > kW4MostShared) rows /= 2;
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
