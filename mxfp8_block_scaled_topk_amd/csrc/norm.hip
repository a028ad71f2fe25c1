// mx_add_rmsnorm: residual addition, root-mean-square norm and MX
// quantisation of its result, one pass over the rows:
//
//   h[r]  = x[r] + residual[r]                       fp32 (h = x without one)
//   n[r]  = h[r] / sqrt(mean(h[r]^2) + eps) * weight fp32
//   residual_out = bf16(h),  y = bf16(n),  (q, s) = MX quantisation of n
//
// Each output is rounded once, from the fp32 value: q is not the quantisation
// of y, and the norm reads h before h is rounded to bf16.
//
// A lane owns chunks of 8 consecutive elements (16 bytes of bf16), so a quad
// of lanes owns one 32-element MX block and its amax is two DPP exchanges.  W
// waves share a row, chunk c of lane t covering elements 8 (64 W c + t) .. + 8:
// the loads and stores of a wave are contiguous.  The row stays in registers
// between the sum of squares and the outputs (up to 32 elements a lane);
// the sum is a tree over the lane's elements, the wave (DPP) and the W waves
// (LDS).  Rows longer than 32768 (16384 when they are not aligned) are read twice
// (add_rmsnorm_long).
// HBM-bound: 2 bytes per element in (4 with a residual), 1 + 1/32 out (2 more
// for each of residual_out and y).  16384 x 2048 with all of them takes 58 us,
// 303 MB at 5.2 TB/s (a copy of 256 MB: 5.5); 1031 x 4304 6.9 us; one row of 2048
// 2.7 us, of which the launch is 1.7.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "fused.h"

namespace mxmoe {

namespace {

struct NormParams {
  const uint16_t* x;
  const uint16_t* res;     // or null
  const void* weight;      // bf16 or fp32 [K]
  uint16_t* res_out;       // or null
  uint16_t* y;             // or null
  uint8_t* q;              // or null
  uint8_t* s;
  int64_t rows, K, ldx, ldr;
  int64_t s_stride;        // scale bytes per row
  int nb;                  // scales per row, without the padding
  int w_f32;
  float eps;
};

// The first n (1 .. 7) of the 16-byte window's 8 elements that ends n elements
// into the window (elements before a row's last chunk are readable): moved to
// the front, zeros behind them.
__device__ __forceinline__ uint4 window8(const u32x4_any& u, int n) {
  const uint64_t lo = (uint64_t)u.y << 32 | u.x, hi = (uint64_t)u.w << 32 | u.z;
  const int s = 16 * (8 - n);
  const uint64_t a = s < 64 ? lo >> s | hi << (64 - s) : hi >> (s - 64);
  const uint64_t b = s < 64 ? hi >> s : 0;
  return make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
}

// Eight bf16 at p as floats, the n first of them (the rest 0).  kVec: n = 8.
// kTiny: the row may be shorter than 8 elements.
template <bool kVec, bool kTiny>
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[8]) {
  if (kVec || n >= 8) {
    const u32x4_any u = *reinterpret_cast<const u32x4_any*>(p);
    unpack_bf16x8(make_uint4(u.x, u.y, u.z, u.w), v);
  } else if constexpr (kTiny) {
    uint16_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = p[i < n ? i : 0];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(t[i]) : 0.0f;
  } else {
    unpack_bf16x8(window8(*reinterpret_cast<const u32x4_any*>(p + n - 8), n), v);
  }
}

template <bool kVec, bool kTiny>
__device__ __forceinline__ void load_weight8(const NormParams& p, int64_t e, int n, float (&w)[8]) {
  if (p.w_f32) {
    const float* f = static_cast<const float*>(p.weight) + e;
    if (kVec || n >= 8) {
      const u32x4_any a = *reinterpret_cast<const u32x4_any*>(f), b = *reinterpret_cast<const u32x4_any*>(f + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __uint_as_float(a[i]);
        w[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = f[i < n ? i : 0];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < n ? w[i] : 0.0f;
    }
  } else {
    load8<kVec, kTiny>(static_cast<const uint16_t*>(p.weight) + e, n, w);
  }
}

// The first `bytes` (1 .. 15) of the 16 in (lo, hi).
__device__ __forceinline__ void store_part(uint8_t* p, uint64_t lo, uint64_t hi, int bytes) {
  if (bytes & 8) {
    __builtin_memcpy(p, &lo, 8);
    p += 8;
    lo = hi;
  }
  if (bytes & 4) {
    const uint32_t v = (uint32_t)lo;
    __builtin_memcpy(p, &v, 4);
    p += 4;
    lo >>= 32;
  }
  if (bytes & 2) {
    const uint16_t v = (uint16_t)lo;
    __builtin_memcpy(p, &v, 2);
    p += 2;
    lo >>= 16;
  }
  if (bytes & 1) *p = (uint8_t)lo;
}

// Whole pieces of an output go past this XCD's L2: they are written once, for a
// kernel on any XCD (16384 x 2048 with three outputs 71 -> 61 us, rows of 1001
// 52 -> 35).
template <bool kVec>
__device__ __forceinline__ void store_bf16x8(uint16_t* p, int n, const float (&v)[8]) {
  const u32x4_any u = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
  if (kVec || n >= 8)
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any*>(p));
  else
    store_part(reinterpret_cast<uint8_t*>(p), (uint64_t)u.y << 32 | u.x, (uint64_t)u.w << 32 | u.z, 2 * n);
}

// y, q and s of 8 elements e .. of row r from h and rstd (n of them exist;
// lanes with n <= 0 only take part in the quad's exchange).
template <bool kVec>
__device__ __forceinline__ void emit8(const NormParams& p, int64_t r, int64_t e, int n, const float (&h)[8],
                                      const float (&w)[8], float rstd) {
  float v[8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = h[i] * rstd * w[i];
    amax = fmaxf(amax, fabsf(v[i]));
  }
  if (p.y && n > 0) store_bf16x8<kVec>(p.y + r * p.K + e, n, v);
  if (!p.q) return;
  amax = quad_max(amax);
  if (n <= 0) return;
  const uint32_t sb = e8m0_from_amax(amax);
  const float inv = e8m0_inverse(sb);
  const uint32_t lo = e4m3x4_sat(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  const uint32_t hi = e4m3x4_sat(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  uint8_t* d = p.q + r * p.K + e;
  const u32x2_any u = {lo, hi};
  if (kVec || n >= 8)
    __builtin_nontemporal_store(u, reinterpret_cast<u32x2_any*>(d));
  else
    store_part(d, (uint64_t)hi << 32 | lo, 0, n);
  if ((threadIdx.x & 3) == 0) {
    const int b = static_cast<int>(e >> 5);
    uint8_t* sr = p.s + r * p.s_stride;
    sr[b] = static_cast<uint8_t>(sb);
    if ((p.nb & 1) && b == p.nb - 1) sr[p.nb] = 0;
  }
}

// Sum of x over the W waves that share a row (each wave's partial in LDS).
template <int W>
__device__ __forceinline__ float row_sum(float x, float* part) {
  x = wave_sum(x);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();   // the previous row's partials are read
    if ((threadIdx.x & 63) == 0) part[wave] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += part[i];
  }
  return x;
}

// 1 / sqrt(m).  The hardware's root is good to 1 ulp; a Newton step takes it to
// about half.
__device__ __forceinline__ float recip_root(float m) {
  const float r = rsqrtf(m);
  return r > 0.0f ? fmaf(0.5f * r, fmaf(-m * r, r, 1.0f), r) : r;   // (an infinite element gives 0)
}

// Squares of a row can add up past fp32 (elements over 1.8e19 / sqrt K).  The row
// then comes again, scaled by kFar: its sum of squares lies between 2^-64 and
// 2^89, and elements whose scaled square underflows are below 2^-85 of it.  The
// branch is taken by whole rows; residual_out is stored ahead of it (behind it,
// one row of 2048 takes 2.8 us instead of 2.7 and 16384 x 2048 62 instead of 58).
constexpr float kFar = 0x1p-96f;

// sum: of the row's squares, the same in all lanes that share it; sum_far(): of
// those of the row times kFar
template <class F>
__device__ __forceinline__ float rstd_of(float sum, const NormParams& p, F sum_far) {
  const float k = static_cast<float>(p.K);
  if (__builtin_expect(__builtin_amdgcn_readfirstlane(__float_as_int(sum)) == 0x7f800000, 0))   // infinity
    return recip_root(sum_far() / k + p.eps * kFar * kFar) * kFar;
  return recip_root(sum / k + p.eps);
}

// Sum of the squares of 8 elements times k.
__device__ __forceinline__ float squares8(const float (&h)[8], float k) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = h[2 * i] * k, b = h[2 * i + 1] * k;
    t[i] = a * a + b * b;
  }
  return (t[0] + t[1]) + (t[2] + t[3]);
}

// W waves per row (kR = max(1, 4 / W) rows per workgroup), C chunks per lane.
// kTiny: rows of fewer than 8 elements.
template <int W, int C, bool kVec, bool kTiny>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void add_rmsnorm_kernel(NormParams p) {
  constexpr int kRows = W < 4 ? 4 / W : 1;
  static_assert(W == 1 || W >= 4, "one wave per row, or the workgroup's waves share one");
  __shared__ float part[W];
  const int lane = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t first = (int64_t)blockIdx.x * kRows + (W == 1 ? threadIdx.x >> 6 : 0);
  for (int64_t r = first; r < p.rows; r += (int64_t)gridDim.x * kRows) {
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t e = 8 * (int64_t)(64 * W * c + lane);
      const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
      if (n > 0) {
        load8<kVec, kTiny>(p.x + r * p.ldx + e, n, h[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = 0.0f;
      }
    }
    if (p.res) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t e = 8 * (int64_t)(64 * W * c + lane);
        const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
        if (n > 0) {
          float a[8];
          load8<kVec, kTiny>(p.res + r * p.ldr + e, n, a);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[c][i] += a[i];
        }
      }
    }
    auto row_squares = [&](float k) __attribute__((always_inline)) {
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) sum += squares8(h[c], k);
      return sum;
    };
    const float sum = row_squares(1.0f);
    // the weight: with few chunks per lane (few or short rows, where latency
    // counts) requested before the sum's exchange
    constexpr bool kEarly = C <= 2;
    float w[kEarly ? C : 1][8] = {};
    auto load_w = [&](int c, float (&v)[8]) __attribute__((always_inline)) {
      const int64_t e = 8 * (int64_t)(64 * W * c + lane);
      const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
      if (n > 0) load_weight8<kVec, kTiny>(p, e, n, v);
    };
    if constexpr (kEarly) {
#pragma unroll
      for (int c = 0; c < C; ++c) load_w(c, w[c]);
    }
    const float total = row_sum<W>(sum, part);
    // ahead of the root and its branch
    if (p.res_out) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t e = 8 * (int64_t)(64 * W * c + lane);
        const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
        if (n > 0) store_bf16x8<kVec>(p.res_out + r * p.K + e, n, h[c]);
      }
    }
    const float rstd = rstd_of(total, p, [&]() __attribute__((always_inline)) {
      return row_sum<W>(row_squares(kFar), part);
    });
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t e = 8 * (int64_t)(64 * W * c + lane);
      const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
      if constexpr (!kEarly) load_w(c, w[0]);
      emit8<kVec>(p, r, e, n, h[c], w[kEarly ? c : 0], rstd);
    }
  }
}

constexpr int kLongWaves = 16;

// Rows of any length: the row is read once for its sum of squares and again
// for the outputs.  A thread reads and writes the same chunks both times, so
// an output may still take its input's place.
template <bool kVec>
__global__ __launch_bounds__(64 * kLongWaves) void add_rmsnorm_long(NormParams p) {
  __shared__ float part[kLongWaves];
  constexpr int64_t kStep = 8 * 64 * kLongWaves;
  const int64_t steps = (p.K + kStep - 1) / kStep;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    auto load_h = [&](int64_t e, int n, float (&h)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = 0.0f;
      if (n <= 0) return;
      load8<kVec, false>(p.x + r * p.ldx + e, n, h);
      if (p.res) {
        float a[8];
        load8<kVec, false>(p.res + r * p.ldr + e, n, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += a[i];
      }
    };
    auto row_squares = [&](float scale) __attribute__((always_inline)) {
      // 16 chunks at a time, 16 of these at a time: of up to 2048 chunks none
      // goes through more than 42 additions (one running sum would be off by
      // 2^-15 where all roundings fall to one side)
      float sum = 0.0f, sum256 = 0.0f, sum16 = 0.0f;
      for (int64_t k = 0; k < steps; ++k) {
        const int64_t e = k * kStep + 8 * (int64_t)threadIdx.x;
        const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
        float h[8];
        load_h(e, n, h);
        sum16 += squares8(h, scale);
        if ((k & 15) != 15) continue;
        sum256 += sum16;
        sum16 = 0.0f;
        if ((k & 255) != 255) continue;
        sum += sum256;
        sum256 = 0.0f;
      }
      return sum + (sum256 + sum16);
    };
    const float rstd = rstd_of(row_sum<kLongWaves>(row_squares(1.0f), part), p, [&]() __attribute__((always_inline)) {
      return row_sum<kLongWaves>(row_squares(kFar), part);
    });
    for (int64_t k = 0; k < steps; ++k) {
      const int64_t e = k * kStep + 8 * (int64_t)threadIdx.x;
      const int n = static_cast<int>(std::min<int64_t>(p.K - e, 8));
      float h[8], w[8] = {};
      load_h(e, n, h);
      if (n > 0) load_weight8<kVec, false>(p, e, n, w);
      if (p.res_out && n > 0) store_bf16x8<kVec>(p.res_out + r * p.K + e, n, h);
      emit8<kVec>(p, r, e, n, h, w, rstd);
    }
  }
}

template <bool kVec>
void launch_norm(const NormParams& p, hipStream_t stream) {
  const int64_t cap = (int64_t)num_cus() * 32;
  const int64_t chunks = (p.K + 7) / 8;   // of a row
#define MX_NORM_LAUNCH_T(W, C, kTiny)                                                                          \
  do {                                                                                                         \
    const int64_t per = W < 4 ? 4 / W : 1;                                                                     \
    const int64_t grid = std::min(cap, (p.rows + per - 1) / per);                                              \
    add_rmsnorm_kernel<W, C, kVec, kTiny><<<dim3((unsigned)grid), dim3(64 * (W < 4 ? 4 : W)), 0, stream>>>(p); \
  } while (0)
#define MX_NORM_LAUNCH(W, C) MX_NORM_LAUNCH_T(W, C, false)
#define MX_NORM_LAUNCH_VEC(W, C)              \
  do {                                        \
    if constexpr (kVec) MX_NORM_LAUNCH(W, C); \
  } while (0)
#define MX_NORM_LONG()                                                                         \
  add_rmsnorm_long<kVec><<<dim3((unsigned)std::min<int64_t>((int64_t)num_cus() * 2, p.rows)), \
                           dim3(64 * kLongWaves), 0, stream>>>(p)
  if (p.K < 8) {
    if constexpr (!kVec) MX_NORM_LAUNCH_T(1, 1, true);
  } else if (p.rows <= num_cus()) {
    // a row's latency counts, not the waves it takes (1 row of 2048: 4.8 us with
    // one wave of 4 chunks a lane, 2.7 with 4 waves)
    if (chunks <= 64) MX_NORM_LAUNCH(1, 1);
    else if (chunks <= 256) MX_NORM_LAUNCH(4, 1);
    else if (chunks <= 512) MX_NORM_LAUNCH(8, 1);
    else if (chunks <= 1024) MX_NORM_LAUNCH(16, 1);
    else if (chunks <= 2048) MX_NORM_LAUNCH(16, 2);
    else if (kVec && chunks <= 4096) MX_NORM_LAUNCH_VEC(16, 4);
    else MX_NORM_LONG();
  } else if (chunks <= 64) MX_NORM_LAUNCH(1, 1);
  else if (chunks <= 128) MX_NORM_LAUNCH(1, 2);
  else if (chunks <= 256) MX_NORM_LAUNCH(1, 4);
  else if (chunks <= 512) MX_NORM_LAUNCH(4, 2);
  else if (chunks <= 1024) MX_NORM_LAUNCH(4, 4);
  else if (chunks <= 2048) MX_NORM_LAUNCH(8, 4);
  else if (kVec && chunks <= 4096) MX_NORM_LAUNCH_VEC(16, 4);
  else MX_NORM_LONG();
#undef MX_NORM_LONG
#undef MX_NORM_LAUNCH_VEC
#undef MX_NORM_LAUNCH
#undef MX_NORM_LAUNCH_T
}

}  // namespace

}  // namespace mxmoe

extern "C" int mx_add_rmsnorm(const void* x_bf16, int64_t ldx, const void* residual_bf16, int64_t ldr,
                              const void* weight, int weight_type, float eps, int64_t rows, int64_t kd,
                              void* residual_out_bf16, void* y_bf16, void* q_u8, void* s_u8, void* stream) {
  using namespace mxmoe;
  if (rows < 0 || kd <= 0 || ldx < kd || (residual_bf16 && ldr < kd))
    return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: bad sizes rows=%lld kd=%lld ldx=%lld ldr=%lld", (long long)rows,
                (long long)kd, (long long)ldx, (long long)ldr);
  if (!dims_in_range({rows, ldx, residual_bf16 ? ldr : 0}))
    return fail(MX_ERR_UNSUPPORTED, "mx_add_rmsnorm: rows, ldx or ldr above 2^31 - 1");
  if (kd > (int64_t)1 << 24) return fail(MX_ERR_UNSUPPORTED, "mx_add_rmsnorm: kd=%lld > 2^24", (long long)kd);
  if (weight_type != MX_TYPE_BF16 && weight_type != MX_TYPE_F32)
    return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: weight_type must be MX_TYPE_BF16 or MX_TYPE_F32, got %d",
                weight_type);
  if (!(eps >= FLT_MIN) || !std::isfinite(eps))
    return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: eps must be a positive normal float");
  if (!q_u8 != !s_u8) return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: q and s go together");
  if (residual_out_bf16 && !residual_bf16)
    return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: residual_out without a residual");
  if (rows == 0) return MX_OK;
  if (!x_bf16 || !weight || (!q_u8 && !y_bf16))
    return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: null pointer");
  if (reinterpret_cast<uintptr_t>(x_bf16) % 2 || reinterpret_cast<uintptr_t>(residual_bf16) % 2 ||
      reinterpret_cast<uintptr_t>(weight) % (weight_type == MX_TYPE_F32 ? 4 : 2) ||
      reinterpret_cast<uintptr_t>(residual_out_bf16) % 2 || reinterpret_cast<uintptr_t>(y_bf16) % 2)
    return fail(MX_ERR_UNSUPPORTED, "mx_add_rmsnorm: misaligned pointer");
  NormParams p{};
  p.x = static_cast<const uint16_t*>(x_bf16);
  p.res = static_cast<const uint16_t*>(residual_bf16);
  p.weight = weight;
  p.res_out = static_cast<uint16_t*>(residual_out_bf16);
  p.y = static_cast<uint16_t*>(y_bf16);
  p.q = static_cast<uint8_t*>(q_u8);
  p.s = static_cast<uint8_t*>(s_u8);
  p.rows = rows;
  p.K = kd;
  p.ldx = ldx;
  p.ldr = residual_bf16 ? ldr : kd;
  p.nb = (int)((kd + 31) / 32);
  p.s_stride = 2 * ((kd + 63) / 64);
  p.w_f32 = weight_type == MX_TYPE_F32;
  p.eps = eps;
  // No output may overlap another one or an input, except that residual_out
  // or y may take the place of x or of the residual, row for row.
  const uint64_t dense = (uint64_t)rows * (uint64_t)kd * 2;
  const Span in[3] = {{x_bf16, ((uint64_t)(rows - 1) * (uint64_t)ldx + (uint64_t)kd) * 2},
                      {residual_bf16, ((uint64_t)(rows - 1) * (uint64_t)p.ldr + (uint64_t)kd) * 2},
                      {weight, (uint64_t)kd * (p.w_f32 ? 4 : 2)}};
  const int64_t ld[3] = {ldx, p.ldr, -1};
  const Span out[4] = {{residual_out_bf16, dense},
                       {y_bf16, dense},
                       {q_u8, (uint64_t)rows * (uint64_t)kd},
                       {s_u8, (uint64_t)rows * (uint64_t)p.s_stride}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i) {
      const bool in_place = o < 2 && out[o].p == in[i].p && (ld[i] == kd || (rows == 1 && i < 2));
      if (!in_place && overlaps(out[o], in[i]))
        return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: an output overlaps an input");
    }
    for (int i = o + 1; i < 4; ++i)
      if (overlaps(out[o], out[i])) return fail(MX_ERR_INVALID_ARG, "mx_add_rmsnorm: two outputs overlap");
  }
  const uintptr_t align_or = reinterpret_cast<uintptr_t>(x_bf16) | reinterpret_cast<uintptr_t>(residual_bf16) |
                             reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(residual_out_bf16) |
                             reinterpret_cast<uintptr_t>(y_bf16);
  const bool vec = align_or % 16 == 0 && reinterpret_cast<uintptr_t>(q_u8) % 8 == 0 && kd % 8 == 0 && ldx % 8 == 0 &&
                   p.ldr % 8 == 0;
  if (vec) launch_norm<true>(p, as_stream(stream));
  else launch_norm<false>(p, as_stream(stream));
  return check_launch("mx_add_rmsnorm");
}
