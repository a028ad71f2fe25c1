// Shared by the kernels of int8_linear and gmm_int8: parameters, the groups'
// tables and the matrix instructions' types.
#pragma once

#include "int8_codes.h"
#include "linear_fused.h"

namespace mxmoe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

constexpr int kInt8MaxE = 1024;

struct Int8Params {
  LinParams e;           // sizes (T rows, K, N, nk) and the epilogue's operands
  const int8_t* x;       // [T, K]
  const float* xs;       // [T]
  const int8_t* w;       // [E, rows, K]
  const float* ws;       // [E, rows]
  const int64_t* gl;     // [E], or null: one group of all rows
  int gl_type, E;
  int64_t rows;          // weight rows per expert (2 N with swiglu)
  int present;           // 16-byte chunks of a row in its last 128-element stage
  int swiglu;
  int cached;            // outputs through the caches (see store8_bits)
};

// Stages are 128 bytes of each row; chunk c (16 bytes) of LDS row r lies at chunk
// c ^ ((r / 2) % 8), so that the 16 lanes of one LDS access (consecutive rows, one
// chunk) hit distinct banks.
__device__ __forceinline__ int chunk_offset(int r, int c) { return r * kStageK + ((c ^ ((r >> 1) & 7)) << 4); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class P>
__device__ __forceinline__ P* uniform(P* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
  return reinterpret_cast<P*>(((uint64_t)hi << 32) | lo);
}

// The experts' rows and tiles of kBM rows, by the workgroup's first wave, from the
// group list (counts, or cumulative), clamped to the T rows there are: expert e
// owns rows row0[e] .. row0[e + 1] and tiles tile0[e] .. tile0[e + 1].
template <int kBM>
__device__ __forceinline__ void group_tables(const Int8Params& p, int* tile0, int* row0) {
  constexpr int kPer = kInt8MaxE / 64;
  const int lane = threadIdx.x & 63, E = p.E, per = (E + 63) >> 6;
  const int64_t T = p.e.T;
  // a lane's experts are lane * per + i
  int64_t n[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * per + i;
    n[i] = 0;
    if (i < per && e < E) {
      int64_t v = p.gl[e];
      if (p.gl_type == 0 && e > 0) v = (int64_t)((uint64_t)v - (uint64_t)p.gl[e - 1]);
      n[i] = std::min<int64_t>(std::max<int64_t>(v, 0), T);
    }
    mine += n[i];
  }
  int64_t before = mine;   // at most 2^10 * 2^31
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t v = __shfl_up(before, off);
    if (lane >= off) before += v;
  }
  before -= mine;
  int tiles = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * per + i;
    const int r0 = (int)std::min(before, T), r1 = (int)std::min(before + n[i], T);
    before += n[i];
    n[i] = ((int64_t)r1 - r0 + kBM - 1) / kBM;
    tiles += (int)n[i];
    if (i < per && e < E) row0[e] = r0;
    if (i < per && e == E - 1) row0[E] = r1;
  }
  int first = wave_inclusive_scan(tiles) - tiles;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * per + i;
    if (i < per && e < E) tile0[e] = first;
    first += (int)n[i];
    if (i < per && e == E - 1) tile0[E] = first;
  }
}

// The expert that owns tile t < tile0[E]: the last e with tile0[e] <= t.
__device__ __forceinline__ int expert_of(const int* tile0, int E, int t) {
  const int lane = threadIdx.x & 63, per = (E + 63) >> 6;
  // lanes whose first expert starts at or before t: all up to the owner's lane
  const int at = lane * per;
  const int block = __popcll(__ballot(at < E && tile0[std::min(at, E)] <= t)) - 1;
  if (per == 1) return uniform(block);
  const int e = block * per + std::min(lane, per - 1);
  return uniform(block * per + __popcll(__ballot(lane < per && e < E && tile0[std::min(e, E)] <= t)) - 1);
}

// 8 consecutive features of a token, the first cnt of which exist, to element el +
// lane_el of y: as bf16, or rounded here.  They are written once: past the caches,
// which hold the operands of the tiles to come, but for gmm_int8's rows that do not
// lie on 64 bytes, where the parts of a line that neighbouring tiles write meet in
// the L2 (8 experts, 44922 rows, K = 640: N = 704 43 / 44 us past / through the
// caches, N = 706 72 / 51; 64 experts, 32768 rows, K = 1024, N = 4104: 257 / 235).
// int8_linear's tiles gain less by that on some widths than they lose on others (T =
// 8192, K = 1024: N = 3080 62 / 58, N = 4104 66 / 78), SwiGLU's gain nothing.
__device__ __forceinline__ void store8_bits(uint16_t* y, int64_t el, uint32_t lane_el, int cnt, const u32x4_any& o,
                                            bool cached = false) {
  if (cnt <= 0) return;
  y = at(y, el, lane_el);
  if (cnt >= 8) {
    if (cached) {
      asm volatile("" ::: "memory");   // keeps the two stores apart: merged, the hint is lost
      *reinterpret_cast<u32x4_any*>(y) = o;
    } else {
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any*>(y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < cnt) y[i] = static_cast<uint16_t>(o[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(uint16_t* y, int64_t el, uint32_t lane_el, int cnt, const float (&z)[8],
                                       bool cached = false) {
  store8_bits(y, el, lane_el, cnt,
              u32x4_any{bf16x2(z[0], z[1]), bf16x2(z[2], z[3]), bf16x2(z[4], z[5]), bf16x2(z[6], z[7])}, cached);
}
// The linear's epilogue: bias, activation, residual (load_res8's), then store8.
__device__ __forceinline__ void finish8(const LinParams& p, int64_t el, uint32_t lane_el, int cnt, const float (&b)[8],
                                        const uint4& res, float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += b[i];
  activate(z, p.act);
  float r[8];
  unpack_bf16x8(res, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] += r[i];
  store8(p.y, el, lane_el, cnt, z);
}

// silu(g) u with the hardware exp and reciprocal (about 1 ulp each)
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

}  // namespace mxmoe
