// cache_common.cuh -- what the paged KV cache operators share: the pool as
// the kernels see it, argument checks, rotary phases in fixed point.
#pragma once

#include <cmath>

#include "../../include/peagle_cache.h"
#include "fp8_common.cuh"
#include "pe_common.cuh"

namespace pe {

constexpr int kPage = 16;  // positions a page

// ------------------------------------------------------------------- pools
struct CachePool {
  void* k;
  void* v;
  float* scores;
  int num_blocks;
};

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int kv_elem_bytes(int dtype) {
  return dtype == PE_KV_F32 ? 4 : dtype == PE_KV_BF16 ? 2 : 1;
}
inline int act_elem_bytes(int dtype) { return dtype == PE_KV_F32 ? 4 : 2; }

inline pe_status check_pool(const pe_kv_pool* p) {
  if (!p || !p->k || !p->v || !is_aligned16(p->k) || !is_aligned16(p->v) ||
      (p->scores && !is_aligned16(p->scores)) || p->num_blocks < 1 || p->n_kv_heads < 1)
    return PE_ERR_INVALID_ARGUMENT;
  if (p->dtype != PE_KV_BF16 && p->dtype != PE_KV_F32 && p->dtype != PE_KV_E4M3)
    return PE_ERR_INVALID_ARGUMENT;
  if (p->dtype == PE_KV_E4M3 && !(std::isfinite(p->k_scale) && p->k_scale > 0.f &&
                                  std::isfinite(p->v_scale) && p->v_scale > 0.f))
    return PE_ERR_INVALID_ARGUMENT;
  if (p->head_dim != 64 && p->head_dim != 128) return PE_ERR_UNSUPPORTED;
  return PE_OK;
}

// rows [n, heads, dh] of the activation type, `stride` elements apart
inline bool row_ok(const void* p, int64_t stride, int64_t width, int elem_bytes) {
  return p && is_aligned16(p) && stride >= width && (stride * elem_bytes) % 16 == 0;
}

// ------------------------------------------------------------------ rotary
// Turns per position of every pair, as a 64-bit fraction of a turn: position
// times step, modulo 2^64, is the angle's fraction of a turn, negative
// differences included, but for the step's own error times the position.  The
// steps are products of doubles: off by less than 2^-53 of a turn for theta
// from 10 on, 2^-51 from 1 on (more below, where turns per position exceed 1).
// No fp64 arithmetic and no range reduction is left to the kernel.
struct RopeSteps {
  uint64_t step[64];
  int on;
};

inline RopeSteps rope_steps(float theta, int head_dim) {
  RopeSteps r = {};
  r.on = theta > 0.f ? 1 : 0;
  if (!r.on) return r;
  const int half = head_dim / 2;
  double f[64];
  f[0] = 1.0;
  f[1] = std::pow(static_cast<double>(theta), -1.0 / half);
  for (int i = 2; i < half; ++i) f[i] = f[i >> 1] * f[i >> 1] * ((i & 1) ? f[1] : 1.0);
  for (int i = 0; i < half; ++i) {
    double turns = f[i] * 0.15915494309189533576888376337251;  // 1 / (2 pi)
    turns -= std::floor(turns);
    r.step[i] = static_cast<uint64_t>(turns * 18446744073709551616.0);  // < 2^64: turns < 1
  }
  return r;
}

// cos and sin of pos * step: the top 32 bits of the product are the angle in
// 2^-32 turns, as a signed number in half turns for sincospif.  The float of
// them has 24 bits, which leaves 2^-26 of a turn (1.6 half steps of fp32 in
// cos and sin).
__device__ __forceinline__ void rope_cos_sin(uint64_t step, long long pos, float& c, float& s) {
  const uint64_t turn = step * static_cast<uint64_t>(pos);
  const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

// The same for results that are rounded to 16 bits or fewer (FAST): the
// hardware's sine and cosine, whose error on half a turn either way is 2^-21,
// next to half a step of 2^-9 of the result.
template <bool FAST>
__device__ __forceinline__ void rope_turn(uint64_t step, long long pos, float& c, float& s) {
  if constexpr (FAST) {
    const uint64_t turn = step * static_cast<uint64_t>(pos);
    const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
    __sincosf(static_cast<float>(top) * 1.4629180792671596e-9f, &s, &c);  // 2 pi 2^-32
  } else {
    rope_cos_sin(step, pos, c, s);
  }
}

// The element type's chunk of 16 bytes as floats and back.
template <typename S>
struct Chunk;
template <>
struct Chunk<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Chunk<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Chunk<uint8_t> {
  static constexpr int N = 16;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[16]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t h = e4m3x2_to_f16x2(w[i] >> (16 * k));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[4 * i + 2 * k] = f.x;
        x[4 * i + 2 * k + 1] = f.y;
      }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[16]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32x2_to_e4m3x2(x[4 * i], x[4 * i + 1]) |
             (static_cast<uint32_t>(f32x2_to_e4m3x2(x[4 * i + 2], x[4 * i + 3])) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ uint4 shfl_xor16(uint4 v, int m) {
  v.x = __shfl_xor_sync(0xffffffffu, v.x, m);
  v.y = __shfl_xor_sync(0xffffffffu, v.y, m);
  v.z = __shfl_xor_sync(0xffffffffu, v.z, m);
  v.w = __shfl_xor_sync(0xffffffffu, v.w, m);
  return v;
}

}  // namespace pe
