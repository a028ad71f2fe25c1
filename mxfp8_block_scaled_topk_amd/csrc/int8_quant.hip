// int8_quantize: bf16 rows to int8 with one fp32 scale per row (a token, or an
// output channel of a weight):
//
//   s[r] = max(fl(amax[r] fl(1 / 127)), 2^-126)     amax: the row's largest |x|
//   q[r] = rne(fl(x[r] fl(1 / s[r])))               fl: rounded to fp32
//
// The reciprocal is taken once a row, so an element costs a product and a
// rounding; the floor of the scale keeps it finite (2^126 at most) and gives a
// row of zeros the scale 2^-126.  |x| fl(1 / s) is at most 127 (1 + 3 2^-24), so
// nothing saturates.
//
// A lane owns chunks of 8 consecutive elements (16 bytes in, 8 out); W waves
// share a row, chunk c of lane t covering elements 8 (64 W c + t) .. + 8, and the
// row stays in registers between its maximum and its codes.  Rows longer than
// that are read twice (int8_quantize_long).  HBM bounds it, or the launch: 16384
// rows of 2048 19 us (5.3 TB/s; a copy's rate is 5.1), 196608 of 2048 214 us (5.6), one
// row of 4096 2.3 us.
#include <algorithm>

#include "int8_codes.h"

namespace mxmoe {

namespace {

struct QuantParams {
  const uint16_t* x;
  int8_t* q;
  float* s;
  int64_t rows, K, ldx;
};

// Chunks start at element 8 i, a row's last one (K >= 8) at K - 8: its first
// elements then come twice, with the same codes.
__device__ __forceinline__ int64_t chunk_at(int64_t e, int64_t K) { return std::min<int64_t>(e, K - 8); }

__device__ __forceinline__ void store_codes8(int8_t* d, const u32x4_any& u, float r) {
  __builtin_nontemporal_store(int8_codes8(u, r), reinterpret_cast<u32x2_any*>(d));
}

template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part) {
  m = wave_max(m);
  if constexpr (W > 1) {
    __syncthreads();   // the previous row's partials are read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) m = std::max(m, part[i]);
  }
  return m;
}

// W waves per row (4 / W rows per workgroup for one wave), C chunks per lane.
template <int W, int C>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void int8_quantize_kernel(QuantParams p) {
  constexpr int kRows = W < 4 ? 4 / W : 1;
  static_assert(W == 1 || W >= 4, "one wave per row, or the workgroup's waves share one");
  __shared__ uint32_t part[W];
  const int lane = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t first = (int64_t)blockIdx.x * kRows + (W == 1 ? threadIdx.x >> 6 : 0);
  for (int64_t r = first; r < p.rows; r += (int64_t)gridDim.x * kRows) {
    u32x4_any u[C];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t e = 8 * (int64_t)(64 * W * c + lane);
      u[c] = u32x4_any{0, 0, 0, 0};
      if (e < p.K) u[c] = *reinterpret_cast<const u32x4_any*>(p.x + r * p.ldx + chunk_at(e, p.K));
    }
#pragma unroll
    for (int c = 0; c < C; ++c) m = std::max(m, amax8(u[c]));
    const float s = int8_scale(row_max<W>(m, part));
    if (lane == 0) p.s[r] = s;
    const float inv = 1.0f / s;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t e = 8 * (int64_t)(64 * W * c + lane);
      if (e < p.K) store_codes8(p.q + r * p.K + chunk_at(e, p.K), u[c], inv);
    }
  }
}

constexpr int kLongWaves = 16;

__global__ __launch_bounds__(64 * kLongWaves) void int8_quantize_long(QuantParams p) {
  __shared__ uint32_t part[kLongWaves];
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const uint16_t* x = p.x + r * p.ldx;
    uint32_t m = 0;
    for (int64_t e = 8 * (int64_t)threadIdx.x; e < p.K; e += 8 * 64 * kLongWaves)
      m = std::max(m, amax8(*reinterpret_cast<const u32x4_any*>(x + chunk_at(e, p.K))));
    const float s = int8_scale(row_max<kLongWaves>(m, part));
    if (threadIdx.x == 0) p.s[r] = s;
    const float inv = 1.0f / s;
    for (int64_t e = 8 * (int64_t)threadIdx.x; e < p.K; e += 8 * 64 * kLongWaves)
      store_codes8(p.q + r * p.K + chunk_at(e, p.K), *reinterpret_cast<const u32x4_any*>(x + chunk_at(e, p.K)), inv);
  }
}

// Rows of fewer than 8 elements: a thread each.
__global__ __launch_bounds__(256) void int8_quantize_tiny(QuantParams p) {
  for (int64_t r = blockIdx.x * (int64_t)256 + threadIdx.x; r < p.rows; r += (int64_t)gridDim.x * 256) {
    const uint16_t* x = p.x + r * p.ldx;
    uint32_t m = 0;
    for (int i = 0; i < (int)p.K; ++i) m = std::max<uint32_t>(m, x[i] & 0x7fffu);
    const float s = int8_scale(m);
    p.s[r] = s;
    const float inv = 1.0f / s;
    for (int i = 0; i < (int)p.K; ++i)
      p.q[r * p.K + i] = static_cast<int8_t>(codes4(bf16_to_f32(x[i]) * inv, 0.0f, 0.0f, 0.0f) & 0xff);
  }
}

}  // namespace

int launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t kd, int64_t ld, int8_t* q, float* s,
                         hipStream_t stream) {
  const QuantParams p{x, q, s, rows, kd, ld};
  const int64_t cap = (int64_t)num_cus() * 32;
  const int64_t chunks = (kd + 7) / 8;   // of a row
#define MX_QUANT_LAUNCH(W, C)                                                                             \
  do {                                                                                                    \
    const int64_t per = W < 4 ? 4 / W : 1;                                                                \
    const int64_t grid = std::min(cap, (rows + per - 1) / per);                                           \
    int8_quantize_kernel<W, C><<<dim3((unsigned)grid), dim3(64 * (W < 4 ? 4 : W)), 0, stream>>>(p);       \
  } while (0)
  // Rows of up to 2048 elements: 4 waves each for few rows, whose loads are then all in
  // flight (64 rows of 2048: 2.4 us, a wave each 2.6; 300: 2.45, 2.7), a wave each for
  // many (16384 of 2048: 19.0, 4 waves 19.4; 4096 of 1024: 4.1, 5.0).  Longer rows as many
  // waves as hold them, up to 32768 elements.
  if (kd < 8) int8_quantize_tiny<<<dim3((unsigned)std::min(cap, (rows + 255) / 256)), dim3(256), 0, stream>>>(p);
  else if (chunks <= 64) MX_QUANT_LAUNCH(1, 1);
  else if (chunks <= 256 && rows > 4 * num_cus()) MX_QUANT_LAUNCH(1, 4);
  else if (chunks <= 256) MX_QUANT_LAUNCH(4, 1);
  else if (chunks <= 1024) MX_QUANT_LAUNCH(4, 4);
  else if (chunks <= 4096) MX_QUANT_LAUNCH(16, 4);
  else int8_quantize_long<<<dim3((unsigned)std::min<int64_t>((int64_t)num_cus() * 2, rows)), dim3(64 * kLongWaves), 0, stream>>>(p);
#undef MX_QUANT_LAUNCH
  return check_launch("int8_quantize");
}

int check_int8_quantize(const char* name, int64_t rows, int64_t kd, int64_t ld) {
  if (rows < 0 || kd <= 0 || ld < kd)
    return fail(MX_ERR_INVALID_ARG, "%s: bad sizes rows=%lld kd=%lld ld=%lld", name, (long long)rows, (long long)kd,
                (long long)ld);
  if (!dims_in_range({rows, ld})) return fail(MX_ERR_UNSUPPORTED, "%s: rows or ld above 2^31 - 1", name);
  if (kd > (int64_t)1 << 24) return fail(MX_ERR_UNSUPPORTED, "%s: kd=%lld > 2^24", name, (long long)kd);
  return MX_OK;
}

}  // namespace mxmoe

extern "C" int int8_quantize(const void* x_bf16, int64_t rows, int64_t kd, int64_t ld, void* q_i8, float* s,
                             void* stream) {
  using namespace mxmoe;
  int rc = check_int8_quantize("int8_quantize", rows, kd, ld);
  if (rc) return rc;
  if (rows == 0) return MX_OK;
  if (!x_bf16 || !q_i8 || !s) return fail(MX_ERR_INVALID_ARG, "int8_quantize: null pointer");
  if (reinterpret_cast<uintptr_t>(x_bf16) % 2 || reinterpret_cast<uintptr_t>(s) % 4)
    return fail(MX_ERR_UNSUPPORTED, "int8_quantize: misaligned pointer");
  const Span in = {x_bf16, ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)kd) * 2};
  const Span out[2] = {{q_i8, (uint64_t)rows * (uint64_t)kd}, {s, (uint64_t)rows * 4}};
  if (overlaps(out[0], in) || overlaps(out[1], in) || overlaps(out[0], out[1]))
    return fail(MX_ERR_INVALID_ARG, "int8_quantize: an output overlaps the input or the other output");
  return launch_int8_quantize(static_cast<const uint16_t*>(x_bf16), rows, kd, ld, static_cast<int8_t*>(q_i8), s,
                              as_stream(stream));
}
