// The tile kernel of mx_linear_fused: batches whose arithmetic, not the weight
// stream, sets the time.
//
// A workgroup of WN x WM waves computes a BN (weight rows) x BM (tokens) tile,
// each wave NA x NB fragments of 32 x 32.  The pipeline is the grouped GEMMs'
// one for a single group of rows: K advances 128 elements per stage through a
// two-slot LDS ring filled by direct global->LDS loads; a stage is two 64-wide
// sub-steps; every operand fragment is reloaded for the next sub-step right
// after its last MFMA, so the LDS reads overlap the matrix work; one barrier
// per stage sits between the sub-steps, and the loads of the stage after next
// follow it into the slot it frees.  The kernel is persistent and the stage
// stream runs across tile boundaries: a tile's epilogue runs while the next
// tile's first stage is already in LDS.
//
// Three shapes, by how much of the card the tiles fill and what a stage costs:
//   256 x 256, two slots    1.4 us a stage (3.0 PFLOP/s), the least operand
//                           traffic; 8 waves, all 256 registers
//   256 x 128, three slots  0.9 us a stage (2.4 PFLOP/s), half the epilogue
//   128 x 128, two slots    two workgroups per CU, so that one's epilogue and
//                           first loads run beside the other's products
// Measured: T = 16384, K = N = 4096 with bias and residual 251 - 263 us, 2.1 -
// 2.2 PFLOP/s (the same product in 256 x 256 tiles without a residual 235 us,
// 2.34; the library's fp8 product without any epilogue 224 us).  What bounds it:
// operands arriving in LDS, 64 KB a stage at about 47 GB/s per CU (the matrix
// units are busy half of the time, at 2.1 GHz), then the residual and the output
// of all CUs in one burst per tile.  T = 2048, K = 2048,
// N = 4096 to MXFP8 with gelu_tanh 27 - 30 us: 15 us of stages, the rest one tile's
// launch, first loads and epilogue with nothing beside them.
#include <algorithm>
#include <type_traits>

#include "linear_fused.h"

namespace mxmoe {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const volatile u32x4 lds_u32x4_v;
typedef __attribute__((address_space(3))) const volatile uint8_t lds_u8_v;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

// at most n (wave-uniform) loads outstanding; 0 where n is not among the cases
__device__ __forceinline__ void wait_loads_le(int n) {
  switch (n) {
#define MX_WAIT(N) case N: wait_loads<N>(); break;
    MX_WAIT(16) MX_WAIT(15) MX_WAIT(14) MX_WAIT(13) MX_WAIT(12) MX_WAIT(11) MX_WAIT(10) MX_WAIT(9) MX_WAIT(8) MX_WAIT(7) MX_WAIT(6) MX_WAIT(5)
#undef MX_WAIT
    default: wait_loads<0>(); break;
  }
}
// Workgroup barrier that first drains this wave's LDS accesses.
__device__ __forceinline__ void drain_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ int opaque(int v) {   // keeps address arithmetic where it is used
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class P>
__device__ __forceinline__ P* uniptr(P* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
  return reinterpret_cast<P*>(((uint64_t)hi << 32) | lo);
}

// Tiles are dealt in bands of this many n-tiles, m-tile after m-tile within a
// band, so the tiles that the CUs of one XCD hold at a time share both operands.
constexpr int kBand = 8;

// kG: k stages per scale load.  4 (K a multiple of 512, scale tensors on
// 16-byte boundaries): 16 scale bytes per row at a group's first stage, into a
// double-buffered ring of their own.  1: the stage's 4 bytes per row.  kTail
// (with kG = 1): K is not a multiple of 128; see lin_stream_kernel.
template <int NA, int NB, int WN, int WM, int S, int kG, bool kTail>
__global__ __launch_bounds__(64 * WN * WM) void lin_tile_kernel(LinParams p, int m_tiles, int n_tiles) {
  constexpr int kWaves = WN * WM;
  constexpr int BN = 32 * NA * WN, BM = 32 * NB * WM;
  constexpr int kRowsA = BN / kWaves, kRowsB = BM / kWaves;   // rows each wave fetches
  constexpr int kOpsA = kRowsA / 8, kOpsB = kRowsB / 8;
  constexpr int kScaleWavesA = BN / 64, kScaleWaves = (BN + BM) / 64;   // 64 scale rows per wave, weights' first
  static_assert(kScaleWaves <= kWaves && (S == 2 || S == 3), "scale rows and ring slots");
  static_assert(kG == 1 || !kTail, "scale groups need whole stages");
  constexpr int kSlotData = (BN + BM) * kStageK;
  constexpr int kSlot = kSlotData + (kG == 1 ? (BN + BM) * (kTail ? 8 : 4) : 0);
  constexpr int kScBuf = (BN + BM) * 16;   // one group's scales
  __shared__ __attribute__((aligned(16))) uint8_t ring[S * kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t s_sc[kG == 4 ? 2 * kScBuf : 16];
  __shared__ __attribute__((aligned(16))) float s_bias[BN];   // the tile's, 0 where there is none

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const int li = lane & 31, lg = lane >> 5;
  const int nk = p.nk;
  const int64_t K = p.K, srow = p.s_stride;
  const int total = m_tiles * n_tiles;
  const int G = gridDim.x, GX = G >> 3;   // G is a multiple of 8 (host)
  // XCD x holds workgroups x, x + 8, ...: round j gives it the GX consecutive
  // tiles from j G + x GX on
  const int first_tile = (blockIdx.x & 7) * GX + (blockIdx.x >> 3);
  if (first_tile >= total) return;
  const int my_tiles = (total - first_tile + G - 1) / G;

  struct Tile {
    int64_t n0, t0;
    int rows_n, rows_t;   // that exist
  };
  auto tile_at = [&](int j) __attribute__((always_inline)) -> Tile {
    const int t = first_tile + j * G;
    const int band = t / (kBand * m_tiles);
    const int r = t - band * (kBand * m_tiles);
    const int w = std::min(kBand, n_tiles - band * kBand);
    const int mt = uni(r / w), nt = uni(band * kBand + r % w);
    Tile ti;
    ti.n0 = (int64_t)nt * BN;
    ti.t0 = (int64_t)mt * BM;
    ti.rows_n = uni((int)std::min<int64_t>(BN, p.N - ti.n0));
    ti.rows_t = uni((int)std::min<int64_t>(BM, p.T - ti.t0));
    return ti;
  };

  // ---- loads ------------------------------------------------------------------------
  // An instruction fills 8 rows of 128 bytes: lane l row l / 8, chunk position
  // l % 8, holding chunk (l % 8) ^ ((row / 2) % 8).
  const int drow = lane >> 3;
  const int ch_even = (lane & 7) ^ (lane >> 4), ch_odd = ch_even ^ 4;   // rows 8 j + .., j even and odd
  const uint32_t ring0 = lds_offset(ring), sc0 = lds_offset(s_sc);
  struct Src {
    const uint8_t* w;      // weight row n0
    const uint8_t* x;      // token row t0
    const uint8_t* sc;     // the scale rows this wave fetches (64 of them)
    int last_n, last_t, last_s;
  };
  auto src_of = [&](const Tile& ti) __attribute__((always_inline)) -> Src {
    Src s;
    s.w = uniptr(p.w + ti.n0 * K);
    s.x = uniptr(p.x + ti.t0 * K);
    s.last_n = ti.rows_n - 1;
    s.last_t = ti.rows_t - 1;
    s.sc = wave < kScaleWavesA ? uniptr(p.ws + ti.n0 * srow) : uniptr(p.xs + ti.t0 * srow);
    s.last_s = wave < kScaleWavesA ? s.last_n : s.last_t;
    return s;
  };
  const int srow_local = 64 * (wave < kScaleWavesA ? wave : wave - kScaleWavesA) + lane;
  const uint32_t row0_a = (uint32_t)((kRowsA * wave + drow) * K), row0_b = (uint32_t)((kRowsB * wave + drow) * K);
  constexpr int kLoadOps = kOpsA + kOpsB + 1;
  // S = 2: a stage's loads go out over the first MFMAs of one sub-step (5 behind
  // the first, the rest behind the second: spread wider, the last ones are late).
  // S = 3: half of them over that sub-step's MFMAs, half over the next one's.
  constexpr int kFirst = S == 2 ? kLoadOps : (kLoadOps + 1) / 2;
  constexpr int kPer = S == 2 ? 5 : (kFirst + NA * NB - 1) / (NA * NB);
  const bool sc_wave = kScaleWaves == kWaves || wave < kScaleWaves;
  auto slot_of = [](int gs) __attribute__((always_inline)) -> int {
    if constexpr (S == 2) return gs & 1;
    else return (int)((unsigned)gs % 3u);
  };
  // memory instructions of this wave for tile stage ks (S = 3 leaves the latest stage's in flight)
  auto ops_of = [&](int ks) __attribute__((always_inline)) -> int {
    return kOpsA + kOpsB + (sc_wave && (kG == 1 || (ks & 3) == 0) ? (kTail ? 2 : 1) : 0);
  };
  auto load_part = [&](int i, const Src& s, int ks, int gs) __attribute__((always_inline)) {
    const uint32_t base = ring0 + (uint32_t)slot_of(gs) * (uint32_t)kSlot;
    const int present = kTail && ks == nk - 1 ? 2 * p.tail_blocks : 8;   // 16-byte chunks
    if (i < kOpsA + kOpsB) {
      const bool is_w = i < kOpsA;
      const int j = is_w ? i : i - kOpsA;
      int c = (j & 1) ? ch_odd : ch_even;
      if (kTail && c >= present) c &= 1;
      // rows past the last repeat it
      const uint32_t row = std::min((is_w ? row0_a : row0_b) + (uint32_t)(8 * j) * (uint32_t)K,
                                    (uint32_t)(is_w ? s.last_n : s.last_t) * (uint32_t)K);
      const uint32_t voff = row + (uint32_t)(c * 16) + (uint32_t)(ks * kStageK);
      load_lds16(voff, is_w ? s.w : s.x,
                 base + (uint32_t)((is_w ? 0 : BN * kStageK) + ((is_w ? kRowsA : kRowsB) * wave + 8 * j) * kStageK));
    } else if (sc_wave) {
      const uint32_t off = (uint32_t)std::min(srow_local, s.last_s) * (uint32_t)srow;
      const uint32_t rows = (uint32_t)(wave < kScaleWavesA ? 64 * wave : BN + 64 * (wave - kScaleWavesA));
      if constexpr (kG == 4) {
        if ((ks & 3) == 0)
          load_lds16(off + (uint32_t)(ks * 4), s.sc, sc0 + (uint32_t)(((gs >> 2) & 1) * kScBuf) + rows * 16);
      } else if constexpr (kTail) {
        // two pairs of scale bytes, each pair's rows together; an absent pair repeats the first
        const uint8_t* q = s.sc + off + ks * 4;
        load_lds2(q, base + (uint32_t)kSlotData + rows * 4);
        load_lds2(present > 4 ? q + 2 : q, base + (uint32_t)kSlotData + (uint32_t)((BN + BM) * 4) + rows * 4);
      } else {
        load_lds4(s.sc + off + ks * 4, base + (uint32_t)kSlotData + rows * 4);
      }
    }
  };
  auto load_stage = [&](const Src& s, int ks, int gs) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoadOps; ++i) load_part(i, s, ks, gs);
  };

  // ---- fragments --------------------------------------------------------------------
  const int sw = (li >> 1) & 7;
  const uint32_t rd_a = (uint32_t)((32 * NA * wn + li) * kStageK);
  const uint32_t rd_b = (uint32_t)((BN + 32 * NB * wm + li) * kStageK);
  const uint32_t row_a = (uint32_t)(32 * NA * wn + li), row_b = (uint32_t)(BN + 32 * NB * wm + li);
  uint32_t chk[4];   // byte offset of chunk 2 c + lg within a row
#pragma unroll
  for (int c = 0; c < 4; ++c) chk[c] = (uint32_t)(((2 * c + lg) ^ sw) << 4);
  auto slot_ptr = [&](int gs) __attribute__((always_inline)) {
    uint32_t b = ring0 + (uint32_t)slot_of(gs) * (uint32_t)kSlot;
    asm("" : "+s"(b));
    return (const lds_u8*)(uintptr_t)b;
  };
  auto group_ptr = [&](int gs) __attribute__((always_inline)) {
    uint32_t b = sc0 + (uint32_t)(((gs >> 2) & 1) * kScBuf + (gs & 3) * 4);
    asm("" : "+s"(b));
    return (const lds_u8*)(uintptr_t)b;
  };
  auto scale_at = [&](int gs, int s, uint32_t row) __attribute__((always_inline)) -> int {
    if constexpr (kG == 4) return (int)*reinterpret_cast<lds_u8_v*>(group_ptr(gs) + row * 16 + 2 * s + lg);
    const lds_u8* sl = slot_ptr(gs) + kSlotData;
    if constexpr (kTail) return (int)*reinterpret_cast<lds_u8_v*>(sl + s * ((BN + BM) * 4) + row * 4 + lg);
    return (int)*reinterpret_cast<lds_u8_v*>(sl + row * 4 + 2 * s + lg);
  };
  auto frag_at = [&](int gs, int s, uint32_t rd) __attribute__((always_inline)) -> v8i {
    const lds_u8* sl = slot_ptr(gs) + rd;
    const u32x4 a0 = *reinterpret_cast<lds_u32x4_v*>(sl + chk[2 * s]);
    const u32x4 a1 = *reinterpret_cast<lds_u32x4_v*>(sl + chk[2 * s + 1]);
    return v8i{(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
  };

  // prologue: the first S stages (S = 3 needs as many per tile, host)
  const Src first = src_of(tile_at(0));
  load_stage(first, 0, 0);
  if constexpr (S == 3) {
    int later = 0;
#pragma unroll
    for (int i = 1; i < S; ++i) {
      load_stage(first, i, i);
      later += ops_of(i);
    }
    wait_loads_le(later);
  } else {
    if (nk > 1) load_stage(first, 1, 1);
    else if (my_tiles > 1) load_stage(src_of(tile_at(1)), 0, 1);
    wait_loads<0>();
  }
  drain_barrier();

  int g = 0;   // stages so far: stage g is in slot g % S
  int latest = S == 3 ? ops_of(S - 1) : 0;   // S = 3: memory instructions of the latest stage's loads, at a tile's start
  for (int cj = 0; cj < my_tiles; ++cj) {
    const Tile cur = tile_at(cj);
    const Src csrc = src_of(cur);
    const bool has_next = cj + 1 < my_tiles;
    const Src nsrc = has_next ? src_of(tile_at(cj + 1)) : csrc;
    // waves with no row that exists compute nothing, but load their share and meet the barriers
    const bool active = 32 * NA * wn < cur.rows_n && 32 * NB * wm < cur.rows_t;
    v8i fa[NA], fb[NB];
    int sa[NA], sb[NB];
    v16f acc[NA][NB];
    auto load_a = [&](int gs, int s, int f) __attribute__((always_inline)) {
      fa[f] = frag_at(gs, s, rd_a + f * 32 * kStageK);
      sa[f] = scale_at(gs, s, row_a + 32 * f);
    };
    // ks: the stage in memory (only looked at when kTail)
    auto load_b = [&](int gs, int s, int f, int ks) __attribute__((always_inline)) {
      fb[f] = frag_at(gs, s, rd_b + f * 32 * kStageK);
      sb[f] = scale_at(gs, s, row_b + 32 * f);
      if (kTail && ks == nk - 1) {
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (2 * s + (v >> 2) >= p.tail_blocks) fb[f][v] = 0;
      }
    };
    auto substep = [&](int gs, int ns, int nks, auto kReload, auto extra) __attribute__((always_inline)) {
      if (!active) {
#pragma unroll
        for (int m = 0; m < NA * NB; ++m) extra(m);
        return;
      }
#pragma unroll
      for (int m = 0; m < NA * NB; ++m) {
        const int fm = m / NA, fn = m % NA;
        acc[fn][fm] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[fn], fb[fm], acc[fn][fm], 0, 0, 0, sa[fn], 0,
                                                                      sb[fm]);
        // keeps the MFMA here, among the loads it overlaps; with 512 registers a
        // wave (4 waves) the accumulators live in the upper half
        if constexpr (kWaves > 4) asm volatile("" : "+v"(acc[fn][fm]));
        else asm volatile("" : "+a"(acc[fn][fm]));
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(kReload)::value) {
          if (fm == NB - 1) load_a(gs, ns, fn);
          if (fn == NA - 1) load_b(gs, ns, fm, nks);
        }
        extra(m);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[a][c][v] = 0.0f;
    if (active) {
#pragma unroll
      for (int f = 0; f < NA; ++f) load_a(g, 0, f);
#pragma unroll
      for (int f = 0; f < NB; ++f) load_b(g, 0, f, 0);
    }
    // the loads that stage ks of this tile starts: stage ks + S of the tile, else
    // of the next one, else a repeat of the last that is never read
    auto target = [&](int ks, Src& t) __attribute__((always_inline)) -> int {
      const bool in_tile = ks + S < nk;
      t.w = in_tile ? csrc.w : nsrc.w;
      t.x = in_tile ? csrc.x : nsrc.x;
      t.sc = in_tile ? csrc.sc : nsrc.sc;
      t.last_n = in_tile ? csrc.last_n : nsrc.last_n;
      t.last_t = in_tile ? csrc.last_t : nsrc.last_t;
      t.last_s = in_tile ? csrc.last_s : nsrc.last_s;
      return in_tile ? ks + S : (has_next ? (S == 2 ? 0 : ks + S - nk) : nk - 1);
    };
    auto stage = [&](int ks, auto kLoad) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      Src pt;
      const int ptks = S == 3 && ks > 0 ? target(ks - 1, pt) : 0;
      substep(g, 1, ks, std::true_type{}, [&](int m) __attribute__((always_inline)) {
        if constexpr (S == 3) {
          if (ks > 0) {
#pragma unroll
            for (int i = kFirst + kPer * m; i < kFirst + kPer * m + kPer; ++i)
              if (i < kLoadOps) load_part(i, pt, ptks, g - 1 + S);
          }
        }
      });
      // this wave's part of stage g + 1 has landed (S = 3: stage g + 2 may be in flight)
      if constexpr (S == 2) wait_loads<0>();
      else wait_loads_le(ks > 0 ? ops_of(ptks) : latest);
      drain_barrier();    // every wave's has, and nobody reads slot g % S any more
      if constexpr (decltype(kLoad)::value) {
        Src t;
        const int tks = target(ks, t);
        substep(g + 1, 0, ks + 1, std::true_type{}, [&](int m) __attribute__((always_inline)) {
#pragma unroll
          for (int i = kPer * m; i < kPer * m + kPer; ++i)
            if (i < kFirst) load_part(i, t, tks, g + S);
        });
      } else {
        substep(g + 1, 0, 0, std::false_type{}, [&](int) {});
      }
      __builtin_amdgcn_sched_barrier(0);
      ++g;
    };
    // the tile's bias, a value per thread, goes to LDS before the last stage's
    // barrier; the epilogue reads it after that, and the tile's closing barrier
    // comes before the next tile's
    float bias = 0.0f;
    if (p.bias && tid < cur.rows_n) bias = bias_at(p, cur.n0 + tid);
    for (int ks = 0; ks + 1 < nk; ++ks) stage(ks, std::true_type{});
    static_assert(BN <= 64 * kWaves, "a thread per feature");
    if (tid < BN) s_bias[tid] = bias;
    stage(nk - 1, std::false_type{});

    // ---- epilogue ---------------------------------------------------------------------
    // The slot of the last stage is free until the barrier below.  A wave stages
    // 16 or 32 tokens x 64 features at a time as fp32 rows of 256 bytes, 16-byte
    // chunk c of row r at c ^ (r % 16): the writes (16 rows, one chunk) and the
    // reads (8 lanes of a row) hit distinct banks.  Read back, a lane holds 8 consecutive
    // features of a token, so the residual comes in and the output leaves 128
    // bytes of a row at a time, and a quad holds an MX block.  A wave's memory
    // operations complete in order and a wait behind a conditional store waits
    // for it: the residual comes 64 tokens x 64 features at a time, so that only
    // the first of their rows waits for memory.
    if (active) {
      const int li = opaque(lane & 31), lg = opaque(lane >> 5), lane_e = opaque(lane);
      constexpr int kTok = kWaves * 8192 <= kSlotData ? 32 : 16;   // tokens staged at a time
      static_assert(kWaves * kTok * 256 <= kSlotData && NA % 2 == 0 && NB == 2, "staging fits the slot");
      lds_u8* stg = (lds_u8*)(uintptr_t)(ring0 + (uint32_t)slot_of(g - 1) * (uint32_t)kSlot +
                                         (uint32_t)(wave * kTok * 256));
      const int rr = lane_e >> 3, rc = lane_e & 7;
      const int64_t t_w = cur.t0 + 32 * NB * wm, n_w = cur.n0 + 32 * NA * wn;   // the wave's first token and feature
      const int t_left = (int)std::min<int64_t>(p.T - t_w, 32 * NB);
      const uint32_t lane_el = (uint32_t)rr * (uint32_t)p.N + (uint32_t)(8 * rc);
      const uint32_t lane_s = (uint32_t)rr * (uint32_t)p.ys_stride + (uint32_t)(rc >> 2);
#pragma unroll
      for (int h = 0; h < NA / 2; ++h) {
        const int f = 32 * NA * wn + 64 * h + 8 * rc;   // the lane's features in the tile
        const int64_t n = cur.n0 + f;
        const int cnt = (int)std::min<int64_t>(p.N - n, 8);
        __builtin_amdgcn_sched_barrier(0);
        // the lane's tokens are rr + 8 i
        auto el_of = [&](int i) __attribute__((always_inline)) -> int64_t { return (t_w + 8 * i) * p.N + n_w + 64 * h; };
        uint4 res[8];
#pragma unroll
        for (int pass = 0; pass < 64 / kTok; ++pass) {   // tokens kTok pass ..
          const int fm = pass * kTok / 32;
          if (kTok == 32 || (li >> 4) == (pass & 1)) {
#pragma unroll
            for (int ff = 0; ff < 2; ++ff)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const v16f& c = acc[2 * h + ff][fm];
                const f32x4 o = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
                *reinterpret_cast<lds_f32x4*>(stg + (li % kTok) * 256 + (((8 * ff + 2 * q + lg) ^ (li & 15)) << 4)) = o;
              }
          }
          asm volatile("" ::: "memory");   // a wave's LDS accesses execute in issue order
          if (pass == 0) {
            // after the first accumulators left their registers
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) res[i] = make_uint4(0, 0, 0, 0);
            if (p.res && cnt > 0) {
              if (p.stream_res) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (rr + 8 * i < t_left) res[i] = load_res8<true>(at(p.res, el_of(i), lane_el), cnt);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (rr + 8 * i < t_left) res[i] = load_res8<false>(at(p.res, el_of(i), lane_el), cnt);
              }
            }
          }
          const f32x4 b0 = *reinterpret_cast<const f32x4*>(s_bias + f), b1 = *reinterpret_cast<const f32x4*>(s_bias + f + 4);
          const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int it = 0; it < kTok / 8; ++it) {
            const int r = 8 * it + rr, i = kTok / 8 * pass + it;
            const f32x4 z0 = *reinterpret_cast<const lds_f32x4*>(stg + r * 256 + (((2 * rc) ^ (r & 15)) << 4));
            const f32x4 z1 = *reinterpret_cast<const lds_f32x4*>(stg + r * 256 + (((2 * rc + 1) ^ (r & 15)) << 4));
            float z[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
            const Place pl{el_of(i), (t_w + 8 * i) * p.ys_stride + ((n_w + 64 * h) >> 5), lane_el, lane_s};
            epilogue8(p, pl, n, rr + 8 * i < t_left ? cnt : 0, b, res[i], z);
            __builtin_amdgcn_sched_barrier(0);   // one row at a time (reading the next one ahead gains nothing)
          }
          asm volatile("" ::: "memory");
        }
      }
    }
    // the staging slot is done with: the loads that the last stage left out
    drain_barrier();
    if constexpr (S == 3) {
      if (has_next) {
        load_stage(nsrc, S - 1, g + S - 1);
        latest = ops_of(S - 1);
      }
    } else if (nk > 1) {
      if (has_next) load_stage(nsrc, 1, g + 1);
    } else if (cj + 2 < my_tiles) {
      load_stage(src_of(tile_at(cj + 2)), 0, g + 1);
    }
  }
  wait_loads<0>();   // nothing may land in LDS that is no longer ours
}

template <int NA, int NB, int WN, int WM, int S>
int launch_tiles(const LinParams& p, int per_cu, hipStream_t stream) {
  constexpr int BN = 32 * NA * WN, BM = 32 * NB * WM;
  const int64_t m_tiles = (p.T + BM - 1) / BM, n_tiles = (p.N + BN - 1) / BN;
  const int64_t total = m_tiles * n_tiles;   // under 2^30 (the entry point)
  const int64_t full = std::max<int64_t>(8, (int64_t)num_cus() * per_cu / 8 * 8);
  const dim3 grid((unsigned)std::min(full, (total + 7) / 8 * 8)), block(64 * WN * WM);
  const bool groups = p.K % (4 * kStageK) == 0 && reinterpret_cast<uintptr_t>(p.xs) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(p.ws) % 16 == 0;
  const int mt = (int)m_tiles, nt = (int)n_tiles;
  if (p.K % kStageK) lin_tile_kernel<NA, NB, WN, WM, S, 1, true><<<grid, block, 0, stream>>>(p, mt, nt);
  else if (groups) lin_tile_kernel<NA, NB, WN, WM, S, 4, false><<<grid, block, 0, stream>>>(p, mt, nt);
  else lin_tile_kernel<NA, NB, WN, WM, S, 1, false><<<grid, block, 0, stream>>>(p, mt, nt);
  return check_launch("mx_linear_fused");
}

}  // namespace

int launch_lin_tile256(const LinParams& p, hipStream_t stream) { return launch_tiles<4, 2, 2, 4, 2>(p, 1, stream); }
int launch_lin_tile128(const LinParams& p, hipStream_t stream) { return launch_tiles<2, 2, 2, 2, 2>(p, 2, stream); }
int launch_lin_tile256x128(const LinParams& p, hipStream_t stream) { return launch_tiles<2, 2, 4, 2, 3>(p, 1, stream); }

}  // namespace mxmoe
