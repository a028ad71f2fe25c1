// The tile kernel of int8_linear and gmm_int8: batches whose arithmetic sets the
// time.
//
// A workgroup of WN x WM waves computes a BN (weight rows) x BM (tokens) tile, each
// wave NA x NB fragments of 32 x 32.  K advances 128 bytes per stage through a
// two-slot LDS ring filled by direct global->LDS loads; a stage is two 64-wide
// sub-steps; every operand fragment is reloaded for the next sub-step right after
// its last MFMA, so the LDS reads overlap the matrix work; one barrier per stage
// sits between the sub-steps, and the loads of the stage after next follow it into
// the slot it frees.  The kernel is persistent and the stage stream runs across
// tile boundaries: a tile's epilogue runs while the next tile's first stage is
// already in LDS.  V_MFMA_I32_32X32X32_I8: lane l holds 16 consecutive k of operand
// row l % 32, half l / 32 of the 32; of the result, row l % 32 of the second operand
// (a token) and rows 8 q + 4 (l / 32) + (0 .. 3) of the first (features) in elements
// 4 q ...
//
// With SwiGLU every 64 weight rows of a tile are 32 gate rows and the up rows of
// the same 32 features.
//
// Bounds: the main loop, which runs at the rate of the library's plain int8 product
// (about 2100 TOP/s: the matrix units busy half of the time at the 1.9 GHz that the
// card keeps under them), then the epilogue.  T = 16384, K = N = 4096 with residual
// 263 to 277 us (the library without scales or residual 254); 16384 tokens to 8 of
// 128 experts, K = 2048, N = 768, SwiGLU 456 to 490 us: 393 of main loop with 1024 rows
// each, 40 to 45 of stores, the rest the experts' last tiles.  Passes straight behind
// each other run at the clock that the card's power leaves them: the linear's first 30
// take 296 to 313 us, the next 30 281; codes that use more of their 8 bits (a normal's,
// without the few large channels) 278 to 297.
#include <algorithm>
#include <type_traits>

#include "int8.h"

namespace mxmoe {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const volatile u32x4 lds_u32x4_v;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i32x4 lds_i32x4;

// Workgroup barrier that first drains this wave's LDS accesses.
__device__ __forceinline__ void drain_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ int opaque(int v) {   // keeps address arithmetic where it is used
  asm("" : "+v"(v));
  return v;
}

// Tiles of one group are dealt in bands of this many n-tiles, m-tile after m-tile
// within a band, so the tiles that the CUs of one XCD hold at a time share both
// operands.
constexpr int kBand = 8;

template <int NA, int NB, int WN, int WM, bool kGrouped, bool kSwiglu>
__global__ __launch_bounds__(64 * WN * WM) void int8_tile_kernel(Int8Params p, int m_tiles, int n_tiles) {
  constexpr int kWaves = WN * WM;
  constexpr int BN = 32 * NA * WN, BM = 32 * NB * WM;
  constexpr int kOut = kSwiglu ? BN / 2 : BN;                 // features a tile computes
  constexpr int kRowsA = BN / kWaves, kRowsB = BM / kWaves;   // rows each wave fetches
  constexpr int kOpsA = kRowsA / 8, kOpsB = kRowsB / 8;
  constexpr int kSlot = (BN + BM) * kStageK;
  static_assert(NA % 2 == 0, "the epilogue's blocks of 64 weight rows");
  // SwiGLU's epilogue has LDS of its own (2 KB a wave), so that the next tile's second
  // stage is on its way before its stores (16K tokens to 8 of 128 experts, K = 2048, N =
  // 768: 496 -> 472 us); the other one uses the last stage's slot (with twice the
  // outputs of its own: K = 2048, N = 1536 447 -> 453).
  constexpr bool kEarly = kSwiglu;
  constexpr int kStage = 2048;
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * kSlot];
  __shared__ __attribute__((aligned(16))) float s_ws[BN];     // the tile's scales and bias
  __shared__ __attribute__((aligned(16))) float s_xs[BM];
  __shared__ __attribute__((aligned(16))) float s_bias[kGrouped ? 4 : BN];
  __shared__ __attribute__((aligned(16))) uint8_t s_out[kEarly ? kWaves * kStage : 16];
  extern __shared__ int s_tab[];   // kGrouped: tile0 and row0, E + 1 each

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const int li = lane & 31, lg = lane >> 5;
  const int nk = p.e.nk;
  const int64_t K = p.e.K, N = p.e.N;
  if constexpr (kGrouped) {
    if (wave == 0) group_tables<BM>(p, s_tab, s_tab + p.E + 1);
    __syncthreads();
    m_tiles = uniform(s_tab[p.E]);
  }
  const int total = m_tiles * n_tiles;
  const int G = gridDim.x, GX = G >> 3;   // G is a multiple of 8 (host)
  // XCD x holds workgroups x, x + 8, ...: round j gives it the GX consecutive
  // tiles from j G + x GX on
  const int first_tile = (blockIdx.x & 7) * GX + (blockIdx.x >> 3);
  if (first_tile >= total) return;
  const int my_tiles = (total - first_tile + G - 1) / G;

  struct Tile {
    int64_t n0, t0;       // first feature and token
    int64_t first_row;    // the expert's first weight row
    int rows_n, rows_t;   // features and tokens that exist
  };
  auto tile_at = [&](int j) __attribute__((always_inline)) -> Tile {
    const int t = first_tile + j * G;
    Tile ti;
    int64_t t_end = p.e.T;
    int nt;
    if constexpr (kGrouped) {
      const int mt = uniform(t / n_tiles);
      nt = uniform(t - mt * n_tiles);
      const int e = expert_of(s_tab, p.E, mt);
      const int* row0 = s_tab + p.E + 1;
      ti.t0 = uniform(row0[e] + (mt - s_tab[e]) * BM);
      t_end = uniform(row0[e + 1]);
      ti.first_row = e * p.rows;
    } else {
      const int band = t / (kBand * m_tiles);
      const int r = t - band * (kBand * m_tiles);
      const int w = std::min(kBand, n_tiles - band * kBand);
      ti.t0 = (int64_t)uniform(r / w) * BM;
      nt = uniform(band * kBand + r % w);
      ti.first_row = 0;
    }
    ti.n0 = (int64_t)nt * kOut;
    ti.rows_n = uniform((int)std::min<int64_t>(kOut, N - ti.n0));
    ti.rows_t = uniform((int)std::min<int64_t>(BM, t_end - ti.t0));
    return ti;
  };

  // ---- loads ------------------------------------------------------------------------
  // An instruction fills 8 rows of 128 bytes: lane l row l / 8, chunk position
  // l % 8, holding chunk (l % 8) ^ ((row / 2) % 8).
  const int drow = lane >> 3;
  const int ch_even = (lane & 7) ^ (lane >> 4), ch_odd = ch_even ^ 4;   // rows 8 j + .., j even and odd
  const uint32_t ring0 = lds_offset(ring);
  struct Src {
    const int8_t* w;      // weight row of feature n0
    const int8_t* x;      // token row t0
    int last_n, last_t;
  };
  auto src_of = [&](const Tile& ti) __attribute__((always_inline)) -> Src {
    Src s;
    s.w = uniform(p.w + (ti.first_row + ti.n0) * K);
    s.x = uniform(p.x + ti.t0 * K);
    s.last_n = ti.rows_n - 1;
    s.last_t = ti.rows_t - 1;
    return s;
  };
  constexpr int kLoadOps = kOpsA + kOpsB;
  // a stage's loads go out behind the first MFMAs of one sub-step
  constexpr int kPer = 2;
  auto load_part = [&](int i, const Src& s, int ks, int gs) __attribute__((always_inline)) {
    const uint32_t base = ring0 + (uint32_t)(gs & 1) * (uint32_t)kSlot;
    const int present = ks == nk - 1 ? p.present : 8;
    const bool is_w = i < kOpsA;
    const int j = is_w ? i : i - kOpsA;
    const int row0 = (is_w ? kRowsA : kRowsB) * wave + 8 * j;   // in the operand's part of the tile
    int c = (j & 1) ? ch_odd : ch_even;
    if (c >= present) c = 0;   // (chunks past the row's end repeat its first)
    // rows past the last repeat it
    int row = row0 + drow;
    const int8_t* src = s.x;
    if (is_w) {
      src = s.w;
      if constexpr (kSwiglu) {
        if (row0 & 32) src += N * K;   // up rows
        row = ((row0 >> 6) << 5) + (row0 & 31) + drow;
      }
    }
    row = std::min(row, is_w ? s.last_n : s.last_t);
    load_lds16((uint32_t)row * (uint32_t)K + (uint32_t)(ks * kStageK + c * 16), src,
               base + (uint32_t)((is_w ? 0 : BN * kStageK) + row0 * kStageK));
  };
  auto load_stage = [&](const Src& s, int ks, int gs) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoadOps; ++i) load_part(i, s, ks, gs);
  };

  // ---- fragments --------------------------------------------------------------------
  const int sw = (li >> 1) & 7;
  const uint32_t rd_a = (uint32_t)((32 * NA * wn + li) * kStageK);
  const uint32_t rd_b = (uint32_t)((BN + 32 * NB * wm + li) * kStageK);
  uint32_t chk[4];   // byte offset of chunk 2 c + lg within a row
#pragma unroll
  for (int c = 0; c < 4; ++c) chk[c] = (uint32_t)(((2 * c + lg) ^ sw) << 4);
  auto slot_ptr = [&](int gs) __attribute__((always_inline)) {
    uint32_t b = ring0 + (uint32_t)(gs & 1) * (uint32_t)kSlot;
    asm("" : "+s"(b));
    return (const lds_u8*)(uintptr_t)b;
  };
  auto frag_at = [&](int gs, int c, uint32_t rd) __attribute__((always_inline)) -> v4i {
    const u32x4 a = *reinterpret_cast<lds_u32x4_v*>(slot_ptr(gs) + rd + chk[c]);
    return v4i{(int)a.x, (int)a.y, (int)a.z, (int)a.w};
  };

  // prologue: the first two stages
  const Src first = src_of(tile_at(0));
  load_stage(first, 0, 0);
  if (nk > 1) load_stage(first, 1, 1);
  else if (my_tiles > 1) load_stage(src_of(tile_at(1)), 0, 1);
  wait_loads<0>();
  drain_barrier();

  int g = 0;   // stages so far: stage g is in slot g % 2
  constexpr int kStores = NA * NB;   // kEarly: store instructions of a wave's whole tile
  bool stored = false;   // the last tile was one
  for (int cj = 0; cj < my_tiles; ++cj) {
    const Tile cur = tile_at(cj);
    const Src csrc = src_of(cur);
    // the tile whose stages the last two stages' loads bring (one stage a tile: the one after next)
    const int ahead = nk > 1 ? cj + 1 : cj + 2;
    const bool has_next = ahead < my_tiles;
    const Src nsrc = has_next ? src_of(tile_at(ahead)) : csrc;
    // waves with no row that exists compute nothing, but load their share and meet the barriers
    const bool active = 32 * NA * wn < (kSwiglu ? 2 * cur.rows_n : cur.rows_n) && 32 * NB * wm < cur.rows_t;
    v4i fa[2][NA], fb[2][NB];   // chunk pairs 2 s and 2 s + 1 of sub-step s
    v16i acc[NA][NB];
    auto load_a = [&](int gs, int s, int f) __attribute__((always_inline)) {
      fa[0][f] = frag_at(gs, 2 * s, rd_a + f * 32 * kStageK);
      fa[1][f] = frag_at(gs, 2 * s + 1, rd_a + f * 32 * kStageK);
    };
    // last: the stage is the tile's last one, whose absent chunks hold other bytes
    auto load_b = [&](int gs, int s, int f, bool last) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fb[h][f] = frag_at(gs, 2 * s + h, rd_b + f * 32 * kStageK);
        if (last && p.present < 8) {
          if (2 * (2 * s + h) + lg >= p.present) fb[h][f] = v4i{0, 0, 0, 0};
        }
      }
    };
    auto substep = [&](int gs, int ns, bool last, auto kReload, auto extra) __attribute__((always_inline)) {
      if (!active) {
#pragma unroll
        for (int m = 0; m < NA * NB; ++m) extra(m);
        return;
      }
#pragma unroll
      for (int m = 0; m < NA * NB; ++m) {
        const int fm = m / NA, fn = m % NA;
        acc[fn][fm] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[0][fn], fb[0][fm], acc[fn][fm], 0, 0, 0);
        acc[fn][fm] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[1][fn], fb[1][fm], acc[fn][fm], 0, 0, 0);
        // keeps the MFMAs here, among the loads they overlap; with 512 registers a
        // wave (4 waves) the accumulators live in the upper half
        if constexpr (kWaves > 4) asm volatile("" : "+v"(acc[fn][fm]));
        else asm volatile("" : "+a"(acc[fn][fm]));
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(kReload)::value) {
          if (fm == NB - 1) load_a(gs, ns, fn);
          if (fn == NA - 1) load_b(gs, ns, fm, last);
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
        for (int v = 0; v < 16; ++v) acc[a][c][v] = 0;
    if (active) {
#pragma unroll
      for (int f = 0; f < NA; ++f) load_a(g, 0, f);
#pragma unroll
      for (int f = 0; f < NB; ++f) load_b(g, 0, f, nk == 1);
    }
    // wait: the memory instructions that may be outstanding at the stage's barrier
    auto stage = [&](int ks, auto kLast, auto wait) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      substep(g, 1, decltype(kLast)::value, std::true_type{}, [&](int) {});
      wait();             // this wave's part of stage g + 1 has landed
      drain_barrier();    // every wave's has, and nobody reads slot g % 2 any more
      // the stage after next: ks + 2 of the tile, else one of the next tile's first
      // two, else a repeat of the last that is never read
      const bool in_tile = ks + 2 < nk;
      Src t;
      t.w = in_tile ? csrc.w : nsrc.w;
      t.x = in_tile ? csrc.x : nsrc.x;
      t.last_n = in_tile ? csrc.last_n : nsrc.last_n;
      t.last_t = in_tile ? csrc.last_t : nsrc.last_t;
      const int tks = in_tile ? ks + 2 : has_next ? ks + 2 - (nk > 1 ? nk : 2) : nk - 1;
      auto loads = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int i = kPer * m; i < kPer * m + kPer; ++i)
          if (i < kLoadOps) load_part(i, t, tks, g + 2);
      };
      if constexpr (decltype(kLast)::value && kEarly) substep(g + 1, 0, false, std::false_type{}, loads);
      else if constexpr (decltype(kLast)::value) substep(g + 1, 0, false, std::false_type{}, [&](int) {});
      else substep(g + 1, 0, ks + 1 == nk - 1, std::true_type{}, loads);
      __builtin_amdgcn_sched_barrier(0);
      ++g;
    };
    // the tile's scales and bias, a value per thread, go to LDS before the last
    // stage's barrier; the epilogue reads them after that, and the tile's closing
    // barrier comes before the next tile's
    static_assert(BN <= 64 * kWaves && BM <= 64 * kWaves, "a thread per row");
    float my_ws = 0.0f, my_xs = 0.0f, my_bias = 0.0f;
    {
      const int f = kSwiglu ? ((tid >> 6) << 5) + (tid & 31) : tid;
      if (tid < BN && f < cur.rows_n) my_ws = p.ws[cur.first_row + cur.n0 + f + (kSwiglu && (tid & 32) ? N : 0)];
      if (tid < cur.rows_t) my_xs = p.xs[cur.t0 + tid];
      if constexpr (!kGrouped) {
        if (p.e.bias && tid < cur.rows_n) my_bias = bias_at(p.e, cur.n0 + tid);
      }
    }
    auto all = [] { wait_loads<0>(); };
    int ks = 0;
    if constexpr (kEarly) {
      // The last tile's outputs are on their way while this one's first stage runs:
      // the loads that it waits for were issued before them, and a wave's memory
      // operations complete in order.
      if (nk > 1) {
        stage(0, std::false_type{}, [&] {
          if (stored) wait_loads<kStores>();
          else wait_loads<0>();
        });
        ks = 1;
      }
    }
    for (; ks + 1 < nk; ++ks) stage(ks, std::false_type{}, all);
    if (tid < BN) s_ws[tid] = my_ws;
    if (tid < BM) s_xs[tid] = my_xs;
    if constexpr (!kGrouped) {
      if (tid < BN) s_bias[tid] = my_bias;
    }
    stage(nk - 1, std::true_type{}, all);

    // ---- epilogue ---------------------------------------------------------------------
    // A wave's fragments turn through LDS, so that 8 lanes hold 128 bytes of a
    // token's outputs.
    stored = false;
    if (active) {
      const int li = opaque(lane & 31), lg = opaque(lane >> 5), lane_e = opaque(lane);
      const int64_t t_w = cur.t0 + 32 * NB * wm;   // the wave's first token
      const int t_left = cur.rows_t - 32 * NB * wm;
      if constexpr (kEarly) {
        // A lane has 4 consecutive features of token li in each quarter q of a
        // fragment: scales and SwiGLU are applied there (gate fragment 2 f, up 2 f + 1),
        // and 16 tokens at a time go as bf16 through 2 KB per wave, 16-byte chunk c of
        // row r at c ^ (r % 8): writes and reads hit distinct banks.
        stored = cur.rows_t == BM && cur.rows_n == kOut;   // every store instruction is issued
        lds_u8* stg = (lds_u8*)(uintptr_t)(lds_offset(s_out) + (uint32_t)(wave * kStage));
        // 16 sums of a fragment (rows `row` .. of the tile) times their scales
        auto scaled = [&](const v16i& c, int row, float xs, float (&z)[16]) __attribute__((always_inline)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 w = *reinterpret_cast<const float4*>(s_ws + opaque(row + 4 * lg) + 8 * q);
            z[4 * q] = (float)c[4 * q] * xs * w.x;
            z[4 * q + 1] = (float)c[4 * q + 1] * xs * w.y;
            z[4 * q + 2] = (float)c[4 * q + 2] * xs * w.z;
            z[4 * q + 3] = (float)c[4 * q + 3] * xs * w.w;
          }
        };
        constexpr int kF = NA / 2;             // fragments of outputs
        constexpr int kLanes = 4 * kF;         // of a token's row
        constexpr int kStep = 64 / kLanes;     // tokens an instruction stores
        const int rr = lane_e / kLanes, rc = lane_e % kLanes;
        const int f0 = 32 * kF * wn, cnt = cur.rows_n - f0 - 8 * rc;   // the wave's first feature in the tile
        const uint32_t lane_el = (uint32_t)rr * (uint32_t)N + (uint32_t)(8 * rc);
#pragma unroll
        for (int fm = 0; fm < NB; ++fm) {
          __builtin_amdgcn_sched_barrier(0);
          const float xs = s_xs[32 * NB * wm + 32 * fm + li];
          uint32_t o[kF][8];
#pragma unroll
          for (int f = 0; f < kF; ++f) {
            float z[16], u[16];
            scaled(acc[2 * f][fm], 32 * NA * wn + 64 * f, xs, z);
            scaled(acc[2 * f + 1][fm], 32 * NA * wn + 64 * f + 32, xs, u);
#pragma unroll
            for (int v = 0; v < 16; ++v) z[v] = silu_mul(z[v], u[v]);
#pragma unroll
            for (int v = 0; v < 8; ++v) o[f][v] = bf16x2(z[2 * v], z[2 * v + 1]);
          }
#pragma unroll
          for (int pass = 0; pass < 2; ++pass) {
            if ((li >> 4) == pass) {
#pragma unroll
              for (int f = 0; f < kF; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  *reinterpret_cast<lds_u32x2*>(stg + (li & 15) * 128 + (((4 * f + q) ^ (li & 7)) << 4) + 8 * lg) =
                      u32x2{o[f][2 * q], o[f][2 * q + 1]};
            }
            asm volatile("" ::: "memory");   // a wave's LDS accesses execute in issue order
#pragma unroll
            for (int it = 0; it < 16 / kStep; ++it) {
              const int r = kStep * it + rr, tok = 32 * fm + 16 * pass + kStep * it;
              const u32x4 v = *reinterpret_cast<const lds_u32x4*>(stg + r * 128 + ((rc ^ (r & 7)) << 4));
              store8_bits(p.e.y, (t_w + tok) * N + cur.n0 + f0, lane_el, tok + rr < t_left ? cnt : 0,
                          u32x4_any{v.x, v.y, v.z, v.w});
            }
            asm volatile("" ::: "memory");
          }
        }
      } else {
        // Through the slot of the last stage, which is free until the barrier below: 32
        // tokens x 64 features at a time as int32 rows of 256 bytes, 16-byte chunk c of
        // row r at c ^ (r % 16).  Read back, a lane holds 8 consecutive features of a
        // token, where the residual is added before the rounding.
        constexpr int kTok = 32;
        static_assert(kWaves * kTok * 256 <= kSlot, "staging fits the slot");
        lds_u8* stg = (lds_u8*)(uintptr_t)(ring0 + (uint32_t)((g - 1) & 1) * (uint32_t)kSlot +
                                           (uint32_t)(wave * kTok * 256));
        const int rr = lane_e >> 3, rc = lane_e & 7;
#pragma unroll
        for (int h = 0; h < NA / 2; ++h) {
          const int row = 32 * NA * wn + 64 * h;        // first weight row of the 64 in the tile
          const int cnt = cur.rows_n - row - 8 * rc;
          const uint32_t lane_el = (uint32_t)rr * (uint32_t)N + (uint32_t)(8 * rc);
          __builtin_amdgcn_sched_barrier(0);
          // the lane's tokens are rr + 8 i
          auto el_of = [&](int i) __attribute__((always_inline)) -> int64_t {
            return (t_w + 8 * i) * N + cur.n0 + row;
          };
          uint4 res[8];
          auto get8 = [&](const float* src, float (&v)[8]) __attribute__((always_inline)) {
            const float4 a = reinterpret_cast<const float4*>(src)[0], c = reinterpret_cast<const float4*>(src)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = c.x; v[5] = c.y; v[6] = c.z; v[7] = c.w;
          };
          // of its features, in registers where there are some left (T = 2048, K = 1024, N =
          // 2048: 14.2 us, read for every token 14.5; with 256 rows they would spill)
          float b[8] = {}, ws[8];
          if constexpr (kWaves == 4) {
            get8(s_ws + row + 8 * rc, ws);
            if constexpr (!kGrouped) get8(s_bias + row + 8 * rc, b);
          }
#pragma unroll
          for (int fm = 0; fm < NB; ++fm) {
#pragma unroll
            for (int ff = 0; ff < 2; ++ff)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const v16i& c = acc[2 * h + ff][fm];
                const i32x4 o = {c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
                *reinterpret_cast<lds_i32x4*>(stg + li * 256 + (((8 * ff + 2 * q + lg) ^ (li & 15)) << 4)) = o;
              }
            asm volatile("" ::: "memory");   // a wave's LDS accesses execute in issue order
            if constexpr (!kGrouped) {
              if (fm == 0) {
                // after the first accumulators left their registers
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 8; ++i) res[i] = make_uint4(0, 0, 0, 0);
                if (p.e.res && cnt > 0) {
                  if (p.e.stream_res) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                      if (rr + 8 * i < t_left) res[i] = load_res8<true>(at(p.e.res, el_of(i), lane_el), cnt);
                  } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                      if (rr + 8 * i < t_left) res[i] = load_res8<false>(at(p.e.res, el_of(i), lane_el), cnt);
                  }
                }
              }
            }
#pragma unroll
            for (int it = 0; it < kTok / 8; ++it) {
              const int r = 8 * it + rr, i = kTok / 8 * fm + it;
              const float xs = s_xs[32 * NB * wm + 32 * fm + r];
              float z[8];
              if constexpr (kWaves > 4) {
                const int at_row = opaque(row + 8 * rc);
                get8(s_ws + at_row, ws);
                if constexpr (!kGrouped) get8(s_bias + at_row, b);
              }
              const i32x4 z0 = *reinterpret_cast<const lds_i32x4*>(stg + r * 256 + (((2 * rc) ^ (r & 15)) << 4));
              const i32x4 z1 = *reinterpret_cast<const lds_i32x4*>(stg + r * 256 + (((2 * rc + 1) ^ (r & 15)) << 4));
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                z[v] = (float)z0[v] * xs * ws[v];
                z[4 + v] = (float)z1[v] * xs * ws[4 + v];
              }
              const int have = rr + 8 * i < t_left ? cnt : 0;
              if constexpr (kGrouped) store8(p.e.y, el_of(i), lane_el, have, z, p.cached);
              else finish8(p.e, el_of(i), lane_el, have, b, res[i], z);
              __builtin_amdgcn_sched_barrier(0);   // one row at a time
            }
            asm volatile("" ::: "memory");
          }
        }
      }
    }
    if constexpr (kEarly) {
      // (the next tile's scales are written behind its first stage's barrier, if there is one)
      if (nk == 1) drain_barrier();
    } else {
      // the staging slot is done with: the loads that the last stage left out
      drain_barrier();
      if (has_next) load_stage(nsrc, nk > 1 ? 1 : 0, g + 1);
    }
  }
  wait_loads<0>();   // nothing may land in LDS that is no longer ours
}

template <int NA, int NB, int WN, int WM, bool kGrouped, bool kSwiglu>
int launch_tiles(const Int8Params& p, int per_cu, hipStream_t stream, const char* name) {
  constexpr int BN = 32 * NA * WN, BM = 32 * NB * WM, kOut = kSwiglu ? BN / 2 : BN;
  const int64_t m_tiles = (p.e.T + BM - 1) / BM, n_tiles = (p.e.N + kOut - 1) / kOut;
  const int64_t total = (m_tiles + (kGrouped ? p.E : 0)) * n_tiles;   // under 2^30 (the entry points)
  const int64_t full = std::max<int64_t>(8, (int64_t)num_cus() * per_cu / 8 * 8);
  const dim3 grid((unsigned)std::min(full, (total + 7) / 8 * 8));
  const size_t tab = kGrouped ? (size_t)(p.E + 1) * 8 : 0;
  int8_tile_kernel<NA, NB, WN, WM, kGrouped, kSwiglu><<<grid, dim3(64 * WN * WM), tab, stream>>>(p, (int)m_tiles, (int)n_tiles);
  return check_launch(name);
}

}  // namespace

int launch_int8_tile256(const Int8Params& p, hipStream_t stream, const char* name) {
  if (!p.gl) return launch_tiles<4, 2, 2, 4, false, false>(p, 1, stream, name);
  if (p.swiglu) return launch_tiles<4, 2, 2, 4, true, true>(p, 1, stream, name);
  return launch_tiles<4, 2, 2, 4, true, false>(p, 1, stream, name);
}
int launch_int8_tile128(const Int8Params& p, hipStream_t stream, const char* name) {
  if (!p.gl) return launch_tiles<2, 2, 2, 2, false, false>(p, 2, stream, name);
  if (p.swiglu) return launch_tiles<2, 2, 2, 2, true, true>(p, 2, stream, name);
  return launch_tiles<2, 2, 2, 2, true, false>(p, 2, stream, name);
}

}  // namespace mxmoe
