// The streaming kernel of int8_linear and gmm_int8: few tokens per weight row, so
// that the weights' way through the chip sets the time.
//
// A workgroup of WV waves computes 16 NR weight rows x 16 MT tokens (with SwiGLU
// the first half of the weight rows are gates, the second half the same features'
// up rows); the waves share the tile and split K: wave w takes the 128-element
// stages w, w + WV, ....  Each wave streams its stages through an LDS ring of its
// own by direct global->LDS loads, S stages ahead, with no barrier in the loop;
// the int32 sums meet in LDS at the end of a tile, where an integer sum's order
// does not matter.  V_MFMA_I32_16X16X64_I8: lane l holds 16 consecutive k of
// operand row l % 16, chunk l / 16 of the 64; of the result, row l % 16 of the
// second operand (a token) and rows 4 (l / 16) .. + 3 of the first (features).
//
// The workgroups are persistent.  A wave's stream of stages runs on into its next
// tile while the sums of the last one are stored, or, with kOnce, the sums take the
// ring's place and a tile's loads begin when the last one is stored.  (The ring
// beside the partial sums would leave one workgroup a CU room from 32 x 32 on.)
//
// Bounds: the weights' way from HBM where they are read once (32 tokens to 8 of 128
// experts, K = 2048, N = 768, SwiGLU: 63 us, 5.5 TB/s); operand delivery to the CUs that
// a round of tiles fills where they fit the caches (T = 203, K = 2096, N = 4099: 430 tiles
// of 48 x 48, 12 us; the other shapes 13 at best); one token launch, first loads and
// one round (K = 2048, N = 4096, bf16: 5.4 us).
//
// kBf16: p.x is bf16 [T, K], T <= 16 and T K <= kMaxResident (host): every
// workgroup quantises the tokens itself, as int8_quantize does, into rows that stay
// in LDS, swizzled like a slot's; only the weights go through the rings.
#include <algorithm>

#include "int8.h"

namespace mxmoe {

namespace {

constexpr int kMaxResident = 16384;
constexpr int S = 2;   // stages a wave's ring holds

template <int NR, int MT, int WV, bool kGrouped, bool kSwiglu, bool kOnce, bool kBf16>
__global__ __launch_bounds__(64 * WV) void int8_stream_kernel(Int8Params p, uint32_t n_tiles, uint32_t t_tiles) {
  constexpr int kRowsW = 16 * NR, kRowsX = 16 * MT, kRows = kRowsW + (kBf16 ? 0 : kRowsX);   // LDS rows per slot
  constexpr int kOut = kSwiglu ? kRowsW / 2 : kRowsW;   // features a tile computes
  constexpr int kScaleOps = (kRows + 63) / 64;
  constexpr int kSlot = kRows * kStageK + kScaleOps * 256;
  constexpr int kOps = kRows / 8 + kScaleOps;
  constexpr int kRing = WV * S * kSlot;
  constexpr int kPitch = kRowsW + 4;                    // ints per token of a partial tile
  constexpr int kPart = WV * kRowsX * kPitch * 4 + kScaleOps * 256;
  static_assert(kOps < 64, "vmcnt range");
  static_assert(!kOnce || kPart <= kRing, "the partial tiles reuse the ring");
  static_assert(!kSwiglu || NR % 2 == 0, "gate and up fragments");
  static_assert(!kBf16 || (kOnce && !kGrouped && MT == 1), "resident tokens");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRing];
  __shared__ __attribute__((aligned(16))) uint8_t parts[kOnce ? 16 : 2 * kPart];
  // kBf16: a row has an odd number of stages, so that 16 rows' chunks hit distinct banks: at most T (K + 256) bytes
  __shared__ __attribute__((aligned(16))) uint8_t xres[kBf16 ? kMaxResident + 16 * 256 : 16];
  __shared__ uint32_t s_amax[kBf16 ? 16 : 1];
  __shared__ float s_xs[kBf16 ? 16 : 1];
  extern __shared__ int s_tab[];   // kGrouped: tile0 and row0, E + 1 each

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if constexpr (kGrouped) {
    if (wave == 0) group_tables<kRowsX>(p, s_tab, s_tab + p.E + 1);
    __syncthreads();
    t_tiles = (uint32_t)s_tab[p.E];
  }
  const uint32_t total = n_tiles * t_tiles;   // under 2^30 (the entry points)
  const uint32_t G = gridDim.x;
  if (blockIdx.x >= total) return;
  const int my_tiles = (int)((total - blockIdx.x + G - 1) / G);
  const int nk = p.e.nk;
  const int64_t K = p.e.K, N = p.e.N;

  struct Tile {
    const int8_t* w;    // first weight row (gate)
    const int8_t* x;    // first token row
    const float* ws;    // their scales
    const float* xs;
    int n_last, t_last; // last feature and token that exist, from the first
    int64_t n0, t0;
  };
  auto tile_at = [&](int j) __attribute__((always_inline)) -> Tile {
    uint32_t id = blockIdx.x + (uint32_t)j * G;
    Tile t;
    int64_t t_end = p.e.T, first_row = 0;
    uint32_t nt;
    if constexpr (kGrouped) {
      const uint32_t mt = id / n_tiles;
      nt = id - mt * n_tiles;
      const int e = expert_of(s_tab, p.E, (int)mt);
      const int* row0 = s_tab + p.E + 1;
      t.t0 = uniform(row0[e] + ((int)mt - s_tab[e]) * kRowsX);
      t_end = uniform(row0[e + 1]);
      first_row = e * p.rows;
    } else {
      // Workgroups go over the XCDs in turn: XCD b % 8 takes a contiguous share of
      // a round's tiles, cut along the longer side, so that one L2 sees an operand row.
      const uint32_t round = id / G, in_round = std::min(G, total - round * G), b = id - round * G;
      const uint32_t share = in_round >> 3, spare = in_round & 7, xcd = b & 7;
      id = round * G + xcd * share + std::min(xcd, spare) + (b >> 3);
      const bool by_rows = N >= p.e.T;
      const uint32_t inner = by_rows ? t_tiles : n_tiles;
      const uint32_t outer_i = id / inner, inner_i = id - outer_i * inner;
      nt = by_rows ? outer_i : inner_i;
      t.t0 = (int64_t)(by_rows ? inner_i : outer_i) * kRowsX;
    }
    t.n0 = (int64_t)nt * kOut;
    t.n_last = uniform((int)std::min<int64_t>(N - 1 - t.n0, kOut - 1));
    t.t_last = uniform((int)std::min<int64_t>(t_end - 1 - t.t0, kRowsX - 1));
    t.w = uniform(p.w + (first_row + t.n0) * K);
    t.ws = uniform(p.ws + first_row + t.n0);
    t.x = uniform(p.x + t.t0 * K);
    t.xs = uniform(p.xs + t.t0);
    return t;
  };

  // ---- loads of one stage: instruction j fills LDS rows [8 j, 8 j + 8) ------------------
  const int drow = lane >> 3;
  const uint32_t ring0 = lds_offset(ring) + (uint32_t)(wave * S * kSlot);
  auto issue = [&](const Tile& t, int ks, int slot) __attribute__((always_inline)) {
    const uint32_t dst = ring0 + (uint32_t)(slot * kSlot);
    const int present = ks == nk - 1 ? p.present : 8;
#pragma unroll
    for (int j = 0; j < kRows / 8; ++j) {
      const int r = 8 * j + drow;
      int c = (lane & 7) ^ ((r >> 1) & 7);
      if (c >= present) c = 0;   // (chunks past the row's end repeat its first)
      const bool is_w = 8 * j < kRowsW, is_up = kSwiglu && is_w && 8 * j >= kOut;
      // rows past the last repeat it
      const int row = is_w ? std::min(is_up ? r - kOut : r, t.n_last) : std::min(r - kRowsW, t.t_last);
      const int8_t* base = is_w ? (is_up ? t.w + N * K : t.w) : t.x;
      load_lds16((uint32_t)row * (uint32_t)K + (uint32_t)(ks * kStageK + c * 16), base, dst + (uint32_t)(j * 1024));
    }
#pragma unroll
    for (int j = 0; j < kScaleOps; ++j) {
      const int r = (64 * j + lane) % kRows;   // (lanes past the last row repeat others)
      const float* s = r >= kRowsW ? t.xs + std::min(r - kRowsW, t.t_last)
                       : kSwiglu && r >= kOut ? t.ws + N + std::min(r - kOut, t.n_last)
                                              : t.ws + std::min(r, t.n_last);
      load_lds4(reinterpret_cast<const uint8_t*>(s), dst + (uint32_t)(kRows * kStageK + j * 256));
    }
  };

  const int li = lane & 15, lc = lane >> 4;
  const int cnt = wave < nk ? (nk - wave + WV - 1) / WV : 0;   // this wave's stages of a tile
  // the stream of this wave's stages: issued ahead of the consumed ones
  Tile ahead = tile_at(0);
  int ahead_j = 0, ahead_i = 0, in_flight = 0, fill = 0, slot = 0;
  auto issue_next = [&](int tj) __attribute__((always_inline)) {
    if (ahead_j >= my_tiles || cnt == 0 || (kOnce && ahead_j > tj)) return;
    issue(ahead, wave + ahead_i * WV, fill);
    fill = fill + 1 == S ? 0 : fill + 1;
    ++in_flight;
    if (++ahead_i == cnt) {
      ahead_i = 0;
      if (++ahead_j < my_tiles) ahead = tile_at(ahead_j);
    }
  };
  if constexpr (!kOnce) {
#pragma unroll
    for (int i = 0; i < S; ++i) issue_next(0);
  }

  const int xstages = nk | 1;   // kBf16: stages of 128 bytes per token row
  if constexpr (kBf16) {
    constexpr int kThreads = 64 * WV, kIn = kMaxResident / 8 / kThreads;   // 8 elements at a time, all in flight
    const int per_row = (int)K / 8, total8 = (int)p.e.T * per_row;
    const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x);
    u32x4_any in[kIn];
    if (tid < 16) s_amax[tid] = 0;
#pragma unroll
    for (int i = 0; i < kIn; ++i)
      if (tid + i * kThreads < total8) in[i] = *reinterpret_cast<const u32x4_any*>(x + 8 * (int64_t)(tid + i * kThreads));
#pragma unroll
    for (int i = 0; i < S; ++i) issue_next(0);   // the first weights, behind the tokens
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const int u = tid + i * kThreads, r = u / per_row;
      if (i * kThreads >= total8) break;   // uniform
      const uint32_t m = u < total8 ? amax8(in[i]) : 0;
      if (__ballot(r != uniform(r)) == 0) {   // a wave within one row
        const uint32_t most = wave_max(m);
        if (lane == 0 && u < total8) atomicMax(&s_amax[r], most);
      } else if (u < total8) {
        atomicMax(&s_amax[r], m);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const int u = tid + i * kThreads;
      if (u >= total8) break;
      const int r = u / per_row, c8 = u - r * per_row;
      const float sx = int8_scale(s_amax[r]);
      if (c8 == 0) s_xs[r] = sx;
      const u32x2_any q = int8_codes8(in[i], 1.0f / sx);
      uint8_t* row = xres + (r * xstages + (c8 >> 4)) * kStageK;
      *reinterpret_cast<uint2*>(row + ((((c8 >> 1) & 7) ^ ((r >> 1) & 7)) << 4) + 8 * (c8 & 1)) = make_uint2(q.x, q.y);
    }
    // zeros behind the rows' ends
    if (tid < 8 * (int)p.e.T && (tid & 7) >= p.present) {
      const int r = tid >> 3;
      *reinterpret_cast<uint4*>(xres + (r * xstages + nk - 1) * kStageK + (((tid & 7) ^ ((r >> 1) & 7)) << 4)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  }

  for (int tj = 0; tj < my_tiles; ++tj) {
    if constexpr (kOnce) {
      if (tj > 0) __syncthreads();   // the last tile's sums are read
      if (!kBf16 || tj > 0) {
#pragma unroll
        for (int i = 0; i < S; ++i) issue_next(tj);
      }
    }
    // 8 features of a token per lane and unit of the epilogue, the same features in each.
    // The linear's residual is requested here, behind the first stages' loads, its bias
    // before the sums meet (T = 203, K = 2096, N = 4099 with both and gelu: 13.7 us with
    // both requested in the epilogue, 12.6; T = 400, K = 1024, N = 4096: 11.9, 10.5).
    constexpr int kUnits = kRowsX * (kOut / 8), kThreads = 64 * WV, kPer = (kUnits + kThreads - 1) / kThreads;
    static_assert(kThreads % (kOut / 8) == 0, "a lane's units share their features");
    const Tile cur = tile_at(tj);
    const int f8 = tid % (kOut / 8) * 8, tl0 = tid / (kOut / 8);
    auto cnt_of = [&](int i) __attribute__((always_inline)) {   // features that exist of unit i
      const int tl = tl0 + i * (kThreads / (kOut / 8));
      return tl <= cur.t_last ? std::min(cur.n_last + 1 - f8, 8) : 0;
    };
    float bias[8] = {};
    uint4 res[kPer];
    if constexpr (!kGrouped) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        res[i] = make_uint4(0, 0, 0, 0);
        if (p.e.res && cnt_of(i) > 0)
          res[i] = load_res8<false>(p.e.res + (cur.t0 + tl0 + i * (kThreads / (kOut / 8))) * N + cur.n0 + f8, cnt_of(i));
      }
    }
    v4i acc[NR][MT];
#pragma unroll
    for (int f = 0; f < NR; ++f)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[f][m] = v4i{0, 0, 0, 0};
    uint32_t sc[kScaleOps] = {};
    for (int i = 0; i < cnt; ++i) {
      // the stage has landed once only the later one's loads are outstanding
      if (in_flight == 1) wait_loads<0>();
      else wait_loads<kOps>();
      const uint8_t* sl = ring + wave * S * kSlot + slot * kSlot;
      v4i fa[2][NR], fb[2][MT];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int f = 0; f < NR; ++f)
          fa[s][f] = *reinterpret_cast<const v4i*>(sl + chunk_offset(16 * f + li, 4 * s + lc));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (kBf16) {
            const int r = std::min(li, (int)p.e.T - 1);
            fb[s][m] = *reinterpret_cast<const v4i*>(xres + (r * xstages + wave + i * WV) * kStageK +
                                                     (((4 * s + lc) ^ ((r >> 1) & 7)) << 4));
          } else {
            fb[s][m] = *reinterpret_cast<const v4i*>(sl + chunk_offset(kRowsW + 16 * m + li, 4 * s + lc));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kScaleOps; ++j)
        sc[j] = *reinterpret_cast<const uint32_t*>(sl + kRows * kStageK + j * 256 + lane * 4);
      wait_lds();   // the slot is read: refill it
      --in_flight;
      issue_next(tj);
      if (!kBf16 && p.present < 8 && wave + i * WV == nk - 1) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            if (4 * s + lc >= p.present) fb[s][m] = v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int f = 0; f < NR; ++f)
            acc[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[s][f], fb[s][m], acc[f][m], 0, 0, 0);
      slot = slot + 1 == S ? 0 : slot + 1;
    }

    // ---- the waves' sums meet in LDS ----------------------------------------------------
    // kOnce: every wave has read its last stage and no load is outstanding; else
    // the buffers alternate, and the barrier of the tile before says that the one of
    // two tiles ago is read
    if constexpr (kOnce) __syncthreads();
    uint8_t* buf = kOnce ? ring : parts + (tj & 1) * kPart;
    int* part = reinterpret_cast<int*>(buf);
    uint32_t* scales = reinterpret_cast<uint32_t*>(buf + WV * kRowsX * kPitch * 4);
#pragma unroll
    for (int f = 0; f < NR; ++f)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<v4i*>(part + (wave * kRowsX + 16 * m + li) * kPitch + 16 * f + 4 * lc) = acc[f][m];
    if (wave == 0) {   // (which has a stage of every tile)
#pragma unroll
      for (int j = 0; j < kScaleOps; ++j) scales[64 * j + lane] = sc[j];
    }
    if constexpr (!kGrouped) epilogue_bias(p.e, cur.n0 + f8, cnt_of(0), bias);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int tl = tl0 + i * (kThreads / (kOut / 8));
      if (kUnits % kThreads != 0 && tl >= kRowsX) break;
      auto sum8 = [&](int f, float (&z)[8]) __attribute__((always_inline)) {
        int s[8] = {};
#pragma unroll
        for (int w = 0; w < WV; ++w) {
          const int* src = part + (w * kRowsX + tl) * kPitch + f;
          const v4i a = reinterpret_cast<const v4i*>(src)[0], b = reinterpret_cast<const v4i*>(src)[1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[i] += a[i];
            s[4 + i] += b[i];
          }
        }
        const float xs = kBf16 ? s_xs[tl] : __uint_as_float(scales[kRowsW + tl]);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = (float)s[i] * xs * __uint_as_float(scales[f + i]);
      };
      float z[8];
      const int64_t t = cur.t0 + tl, n = cur.n0 + f8;
      sum8(f8, z);
      if constexpr (kSwiglu) {
        float up[8];
        sum8(kOut + f8, up);
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] = silu_mul(z[v], up[v]);
      }
      if constexpr (kGrouped) store8(p.e.y, t * N + n, 0, cnt_of(i), z, p.cached);
      else finish8(p.e, t * N + n, 0, cnt_of(i), bias, res[i], z);
    }
  }
}

template <int NR, int MT, int WV, bool kGrouped, bool kSwiglu, bool kOnce, bool kBf16 = false>
int launch_stream(const Int8Params& p, int per_cu, hipStream_t stream, const char* name) {
  constexpr int kOut = kSwiglu ? 8 * NR : 16 * NR;
  const int64_t n_tiles = (p.e.N + kOut - 1) / kOut;
  const int64_t t_tiles = (p.e.T + 16 * MT - 1) / (16 * MT) + (kGrouped ? p.E : 0);
  const int64_t grid = std::min<int64_t>(n_tiles * t_tiles, (int64_t)num_cus() * per_cu);
  const size_t tab = kGrouped ? (size_t)(p.E + 1) * 8 : 0;
  int8_stream_kernel<NR, MT, WV, kGrouped, kSwiglu, kOnce, kBf16>
      <<<dim3((unsigned)grid), dim3(64 * WV), tab, stream>>>(p, (uint32_t)n_tiles, (uint32_t)t_tiles);
  return check_launch(name);
}

template <int NR, int MT, int WV, bool kOnce>
int launch_any(const Int8Params& p, int per_cu, hipStream_t stream, const char* name) {
  if (!p.gl) return launch_stream<NR, MT, WV, false, false, kOnce>(p, per_cu, stream, name);
  if (p.swiglu) return launch_stream<NR, MT, WV, true, true, kOnce>(p, per_cu, stream, name);
  return launch_stream<NR, MT, WV, true, false, kOnce>(p, per_cu, stream, name);
}

}  // namespace

int launch_int8_32x16(const Int8Params& p, hipStream_t stream, const char* name) {
  return launch_any<2, 1, 4, false>(p, 2, stream, name);
}
int launch_int8_32x16_wide(const Int8Params& p, hipStream_t stream, const char* name) {
  return launch_any<2, 1, 8, false>(p, 1, stream, name);
}
int launch_int8_32x32(const Int8Params& p, hipStream_t stream, const char* name) {
  return launch_any<2, 2, 4, true>(p, 2, stream, name);
}
int launch_int8_48x48(const Int8Params& p, hipStream_t stream, const char* name) {   // (int8_linear only)
  return launch_stream<3, 3, 3, false, false, true>(p, 2, stream, name);
}
int launch_int8_64x64(const Int8Params& p, hipStream_t stream, const char* name) {
  return launch_any<4, 4, 2, true>(p, 2, stream, name);
}

// bf16 tokens quantised by every workgroup itself, where that takes no longer than a
// kernel of its own before the product: of up to 16384 elements (1 x 2048, N = 4096: 5.4
// us, two kernels 6.6; 5 x 2096, N = 4099: 7.0, 7.5; 16 x 1024, N = 8192: 6.9, 6.8; with
// room for 65536: 16 x 4096, N = 4096 14.7, 8.5) for one workgroup a CU (16 x 1024, N =
// 32768: 13.8, 11.2).  A call saves a launch and the workspace besides.  The bound on
// N is one workgroup for each of 256 CUs whatever the device has: it says which calls
// need a workspace, which callers read in the header and ask for without a device.
constexpr int64_t kMaxResidentN = 32 * 256;
bool int8_resident(int64_t T, int64_t K, int64_t N) { return T <= 16 && T * K <= kMaxResident && N <= kMaxResidentN; }
int launch_int8_resident(const Int8Params& p, hipStream_t stream, const char* name) {
  return launch_stream<2, 1, 8, false, false, true, true>(p, 1, stream, name);
}

}  // namespace mxmoe
