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
// times step, modulo 2^64, is the angle's fraction of a turn exactly to the
// step's own rounding (double: 2^-53 of it), at any position and for
// negative differences too.  No fp64 arithmetic and no range reduction is
// left to the kernel.
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
// 2^-32 turns, as a signed number in half turns for sincospif.
__device__ __forceinline__ void rope_cos_sin(uint64_t step, long long pos, float& c, float& s) {
  const uint64_t turn = step * static_cast<uint64_t>(pos);
  const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
}

}  // namespace pe
