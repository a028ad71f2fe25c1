// Helpers of the operators around the expert layer (norm.hip,
// linear_fused.hip): wave reductions by DPP, bf16 packing, and the host check
// that outputs overlap nothing.
#pragma once

#include "common.h"

namespace mxmoe {

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

// A byte range an entry point reads or writes (bytes = 0: absent).
struct Span {
  const void* p;
  uint64_t bytes;
};

inline bool overlaps(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y ? y - x < a.bytes : x - y < b.bytes;
}

// ---------------------------------------------------------------------------
// device
// ---------------------------------------------------------------------------

// Two floats -> two bf16 (round to nearest even) packed low/high.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const bf16x2_t v = __builtin_convertvector((f32x2_t){lo, hi}, bf16x2_t);
  return __builtin_bit_cast(uint32_t, v);
}

// x from another lane, by DPP; lanes whose source lies outside their row (or
// outside kRowMask) get `old`.
template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ float dpp_f32(float old, float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), kCtrl, kRowMask, 0xf, false));
}

// Sum over the 64 lanes of a wave (all active), the same value in every lane:
// shifts by 1, 2, 4 and 8 lanes within each row of 16, lane 15 of rows 0 and 2
// into rows 1 and 3, lane 31 into rows 2 and 3; lane 63 then holds the sum.
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_f32<0x111>(0.0f, x);        // row_shr:1
  x += dpp_f32<0x112>(0.0f, x);        // row_shr:2
  x += dpp_f32<0x114>(0.0f, x);        // row_shr:4
  x += dpp_f32<0x118>(0.0f, x);        // row_shr:8
  x += dpp_f32<0x142, 0xa>(0.0f, x);   // row_bcast:15
  x += dpp_f32<0x143, 0xc>(0.0f, x);   // row_bcast:31
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// 16 and 8 bytes on a boundary of their elements only: gfx950 loads and stores
// them in one instruction all the same.
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// e4m3x4 with its saturation in one instruction per value (finite inputs).
__device__ __forceinline__ uint32_t e4m3x4_sat(float a, float b, float c, float d) {
  a = __builtin_amdgcn_fmed3f(a, -448.0f, 448.0f);
  b = __builtin_amdgcn_fmed3f(b, -448.0f, 448.0f);
  c = __builtin_amdgcn_fmed3f(c, -448.0f, 448.0f);
  d = __builtin_amdgcn_fmed3f(d, -448.0f, 448.0f);
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// Maximum over a quad of lanes (quad_perm [1, 0, 3, 2], then [2, 3, 0, 1]).
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, dpp_f32<0xb1>(x, x));
  return fmaxf(x, dpp_f32<0x4e>(x, x));
}

}  // namespace mxmoe
