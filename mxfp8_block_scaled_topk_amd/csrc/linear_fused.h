// Shared by the kernels of mx_linear_fused: parameters, the direct
// global->LDS loads and the epilogue's arithmetic.
#pragma once

#include <type_traits>

#include "fused.h"

namespace mxmoe {

struct LinParams {
  const uint8_t* x;    // [T, K] e4m3
  const uint8_t* xs;   // [T, s_stride] e8m0
  const uint8_t* w;    // [N, K] e4m3
  const uint8_t* ws;   // [N, s_stride] e8m0
  const void* bias;    // [N] bf16 or fp32, or null
  const uint16_t* res; // [T, N] bf16, or null
  uint16_t* y;         // [T, N] bf16, or null: then yq and ys
  uint8_t* yq;         // [T, N] e4m3
  uint8_t* ys;         // [T, ys_stride] e8m0
  int64_t T, K, N;
  int64_t s_stride, ys_stride;
  int nk;              // 128-element k stages, the last one with
  int tail_blocks;     // this many 32-element blocks (1 .. 4)
  int bias_f32;
  int act;             // mx_activation
  uint32_t n_tiles, t_tiles;   // lin_stream_kernel's tiles along N and T
  uint32_t first8;             // its launch's first workgroup, over 8
  int stream_res;      // the residual is too large to be left in the memory-side cache
};

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kStageK = 128;   // elements (bytes) of a row per k stage

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const lds_u8*)p;
}
// Direct global->LDS loads: lane l's bytes land at lds + l * 16 (or * 4).  The
// compiler keeps the wait states that a memory instruction needs after a vector
// instruction wrote its scalar operands (5: v_readlane of a spilled base) or a
// scalar one wrote m0 (1), but it cannot see one in inline assembly: the s_nop
// stands for them.
// Uniform base plus a per-lane 32-bit offset:
__device__ __forceinline__ void load_lds16(uint32_t voff, const void* sbase, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(sbase), "{m0}"(lds) : "memory");
}
// Per-lane addresses:
__device__ __forceinline__ void load_lds4(const uint8_t* p, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
// two bytes per lane, zero-extended to the lane's LDS word
__device__ __forceinline__ void load_lds2(const uint8_t* p, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_ushort %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {   // at most N loads outstanding
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// every LDS read of this wave has returned
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// erfc(x) / 2 for x >= 0, as t exp(g(t) - x^2) with t = 1 / (1 + x / 2): g is
// the degree-9 polynomial through log(erfc(x) exp(x^2) / (2 t)) at Chebyshev
// nodes in t over 0 <= x <= 12.  Its relative error is under 4e-7 in fp32 up to
// the exponential's own, so gelu keeps its digits in the left tail, where
// 1 + erf(x) would cancel.
__device__ __forceinline__ float half_erfc(float x) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.5f, x, 1.0f));
  float g = 0.15775100886821747f;
  g = fmaf(g, t, -0.7501815557479858f);
  g = fmaf(g, t, 1.3186529874801636f);
  g = fmaf(g, t, -0.909740686416626f);
  g = fmaf(g, t, 0.09432142972946167f);
  g = fmaf(g, t, -0.09025566279888153f);
  g = fmaf(g, t, 0.06523264944553375f);
  g = fmaf(g, t, 0.3803541362285614f);
  g = fmaf(g, t, 0.9993481040000916f);
  g = fmaf(g, t, -1.9586294889450073f);
  return t * __expf(fmaf(-x, x, g));
}

// The activation of n values (act is uniform over the launch).  The hardware
// exp and reciprocal are good to about 1 ulp; every form below is a product
// whose factors keep their relative accuracy until the exponential leaves the
// normal floats (results below about 1e-36 become 0).
template <int n>
__device__ __forceinline__ void activate(float (&z)[n], int act) {
  switch (act) {
    case MX_ACT_RELU:   // (a maximum with 0 would turn NaN into 0)
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = z[i] <= 0.0f ? 0.0f : z[i];
      break;
    case MX_ACT_SILU:   // z / (1 + e^-z)
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] *= __builtin_amdgcn_rcpf(1.0f + __expf(-z[i]));
      break;
    case MX_ACT_GELU:   // z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float e = half_erfc(fabsf(z[i]) * 0.70710678118654752f);
        z[i] *= z[i] > 0.0f ? 1.0f - e : e;
      }
      break;
    case MX_ACT_GELU_TANH:   // (z / 2)(1 + tanh u) = z / (1 + e^-2u)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        constexpr float c = -2.0f * 0.79788456080286536f * 1.4426950408889634f;   // exponents of 2
        const float u2 = z[i] * fmaf(z[i] * z[i], c * 0.044715f, c);
        z[i] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u2));
      }
      break;
    default:
      break;
  }
}

__device__ __forceinline__ float bias_at(const LinParams& p, int64_t n) {
  return p.bias_f32 ? static_cast<const float*>(p.bias)[n] : bf16_to_f32(static_cast<const uint16_t*>(p.bias)[n]);
}

// ---- the epilogue of 8 consecutive features n .. of a token -------------------------
// n is a multiple of 8; cnt (at most 8) of the features exist, none when cnt <=
// 0.  The four lanes of a quad hold one 32-feature block of one token.

// their bias (0 where there is none)
__device__ __forceinline__ void epilogue_bias(const LinParams& p, int64_t n, int cnt, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.0f;
  if (!p.bias || cnt <= 0) return;
  if (cnt >= 8) {
    if (p.bias_f32) {
      __builtin_memcpy(b, static_cast<const float*>(p.bias) + n, 32);
    } else {
      uint4 u;
      __builtin_memcpy(&u, static_cast<const uint16_t*>(p.bias) + n, 16);
      unpack_bf16x8(u, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const float v = bias_at(p, n + (i < cnt ? i : 0));
      b[i] = i < cnt ? v : 0.0f;
    }
  }
}

// Where they lie: element el + lane_el of y, yq and the residual, scale byte s
// + lane_s of ys.  With el and s uniform over the wave the addresses take a
// scalar base and one 32-bit register.
struct Place {
  int64_t el, s;
  uint32_t lane_el, lane_s;
};
template <class T>
__device__ __forceinline__ T* at(T* base, int64_t el, uint32_t lane_el) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(const_cast<typename std::remove_const<T>::type*>(base + el)) +
                              (uint32_t)(lane_el * (uint32_t)sizeof(T)));
}

// The residual of the 8 features as 16 bytes (zeros past cnt).
template <bool kStream>
__device__ __forceinline__ uint4 load_res8(const uint16_t* r, int cnt) {
  uint4 u;
  if (cnt >= 8) {
    const u32x4_any* src = reinterpret_cast<const u32x4_any*>(r);
    const u32x4_any v = kStream ? __builtin_nontemporal_load(src) : *src;
    u = make_uint4(v.x, v.y, v.z, v.w);
  } else {
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = r[i < cnt ? i : 0];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < cnt ? e[i] : 0;
    u = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16, e[4] | (uint32_t)e[5] << 16,
                   e[6] | (uint32_t)e[7] << 16);
  }
  return u;
}

// res: load_res8's (zeros without a residual)
__device__ __forceinline__ void epilogue8(const LinParams& p, const Place& pl, int64_t n, int cnt, const float (&b)[8],
                                          const uint4& res, float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
  activate(z, p.act);
  float r[8];
  unpack_bf16x8(res, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += r[i];
  if (p.y) {
    if (cnt <= 0) return;
    const uint4 o = make_uint4(bf16x2(z[0], z[1]), bf16x2(z[2], z[3]), bf16x2(z[4], z[5]), bf16x2(z[6], z[7]));
    uint16_t* y = at(p.y, pl.el, pl.lane_el);
    if (cnt >= 8) {
      // written once: past the caches, which hold the operands of the tiles to come
      const u32x4_any v = {o.x, o.y, o.z, o.w};
      __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(y));
    } else {
      const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < cnt) y[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    if (cnt < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = i < cnt ? z[i] : 0.0f;
    }
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(z[i]));
    a = quad_max(a);
    if (cnt <= 0) return;
    const uint32_t sb = e8m0_from_amax(a);
    const float inv = e8m0_inverse(sb);
    const uint2 o = make_uint2(e4m3x4_sat(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv),
                               e4m3x4_sat(z[4] * inv, z[5] * inv, z[6] * inv, z[7] * inv));
    uint8_t* q = at(p.yq, pl.el, pl.lane_el);
    if (cnt >= 8) {
      const u32x2_any v = {o.x, o.y};
      __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(q));
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < cnt) q[i] = static_cast<uint8_t>((i < 4 ? o.x : o.y) >> (8 * (i & 3)));
    }
    if ((n & 31) == 0) {
      uint8_t* s = at(p.ys, pl.s, pl.lane_s);
      s[0] = static_cast<uint8_t>(sb);
      if (n + 32 >= p.N && (n & 32) == 0) s[1] = 0;   // the last of an odd count: its pair's padding
    }
  }
}

}  // namespace mxmoe
