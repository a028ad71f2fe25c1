// The int8 quantiser's arithmetic, shared by int8_quantize and the linear that
// quantises its tokens itself.
#pragma once

#include <algorithm>

#include "fused.h"

namespace mxmoe {

// The largest magnitude of 8 bf16, as bits (their order is the magnitudes').
__device__ __forceinline__ uint32_t amax8(const u32x4_any& u) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = std::max(m, u[i] & 0x7fffu);
    m = std::max(m, (u[i] >> 16) & 0x7fffu);
  }
  return m;
}

// Four codes as bytes: adding 3 * 2^22 leaves the nearest integer, ties to even,
// in the sum's last bits (|v| < 2^22).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  constexpr float kMagic = 12582912.0f;
  const uint32_t ua = __float_as_uint(a + kMagic), ub = __float_as_uint(b + kMagic);
  const uint32_t uc = __float_as_uint(c + kMagic), ud = __float_as_uint(d + kMagic);
  const uint32_t lo = __builtin_amdgcn_perm(ub, ua, 0x0c0c0400);   // bytes 0 of ua and ub
  const uint32_t hi = __builtin_amdgcn_perm(ud, uc, 0x04000c0c);
  return lo | hi;
}

// Eight bf16 times r as codes.
__device__ __forceinline__ u32x2_any int8_codes8(const u32x4_any& u, float r) {
  float v[8];
  unpack_bf16x8(make_uint4(u.x, u.y, u.z, u.w), v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r;
  return u32x2_any{codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7])};
}

// int8_quantize's scale of a row from the bits of its largest magnitude (a NaN's lie
// above infinity's and stay one; a NaN's last byte, its code, is 0).
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  const float s = bf16_to_f32(amax_bits) * (1.0f / 127.0f);
  return s < 0x1p-126f ? 0x1p-126f : s;
}

template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return std::max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRowMask, 0xf, false));
}
// Maximum over the 64 lanes of a wave (all active), by wave_sum's moves.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = dpp_max<0x111>(x);        // row_shr:1
  x = dpp_max<0x112>(x);        // row_shr:2
  x = dpp_max<0x114>(x);        // row_shr:4
  x = dpp_max<0x118>(x);        // row_shr:8
  x = dpp_max<0x142, 0xa>(x);   // row_bcast:15
  x = dpp_max<0x143, 0xc>(x);   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

}  // namespace mxmoe
