// mx_linear_fused: a dense MXFP8 linear layer with its epilogue fused:
//
//   z[t, n] = sum over 32-blocks b of 2^(sx[t,b] + sw[n,b]) (xq[t,b] . wq[n,b])
//   out     = act(z + bias) + residual      fp32, rounded once: to bf16, or
//             per 32 outputs to MXFP8
//
// The MFMA orientation and operand layout are the grouped GEMMs': weight rows
// are the A operand, tokens the B operand of V_MFMA_SCALE_F32_32X32X64 (lane l
// holds operand row l % 32; of its 32 bytes, 0-15 and 16-31 belong to scale
// blocks 0 and 1 of the 64-wide step, lane group l / 32 supplying 16 elements
// of each; output lane l holds token l % 32 and features 8 q + 4 (l / 32) +
// (0..3) in accumulator elements 4 q ..).
//
// What the instruction rounds: within each aligned group of 8 consecutive k it
// truncates a product to a multiple of 2^(e - 13), e the largest of the group's
// sums of operand exponents; the groups and steps then add in fp32 (probed with
// one large product beside a small one at every position).  It is the only
// instruction that applies the block scales, so z carries about 13 bits of a
// group's largest product, which is more than e4m3 operands hold; bf16 products
// of scaled operands would be exact at half its rate.
//
// lin_stream_kernel.  A workgroup of WV waves computes 32 NF weight rows x
// 32 MF tokens; the waves share the tile and split K (wave w takes the
// 128-element stages w, w + WV, ...), so the waves of a workgroup read whole
// kilobytes of a weight row together.  Each wave streams its stages through an
// LDS ring of its own by direct global->LDS loads, S stages ahead, with no
// barrier in the loop; the accumulators meet in LDS at the end.  Few bf16 tokens
// (a decode step) skip the quantiser's launch: every workgroup quantises them
// into LDS itself while its first weights are on their way.
//
// Bounded by what a CU can take in, about 60 GB/s (26 bytes a cycle) of weights
// and tokens together, on as many CUs as there are tiles (N / 32 for few tokens),
// behind 3 us of launch and first loads: T = 32, K = N = 4096 takes 7.0 us on 128 CUs
// (17 MB of weights at 2.4 TB/s), T = 1 5.7 us; K = N = 8192 at T = 1 12.2 us (67
// MB, 5.5 TB/s); T = 1, K = N = 2048 from bf16 4.6 us on 64.  The tile is a choice
// between re-reading the tokens (few rows) and few workgroups (many rows).
#include <algorithm>

#include "linear_fused.h"

namespace mxmoe {

int launch_mx_quantize(const uint16_t* x, int64_t rows, int64_t kd, int64_t ld, uint8_t* q, uint8_t* s,
                       hipStream_t stream);

int launch_lin_tile256(const LinParams& p, hipStream_t stream);
int launch_lin_tile128(const LinParams& p, hipStream_t stream);
int launch_lin_tile256x128(const LinParams& p, hipStream_t stream);

namespace {

constexpr int64_t kMaxK = (int64_t)1 << 20;   // 32-bit offsets within a tile's rows

// byte offset of 16-byte chunk c of row r in a tile of 128-byte rows: the 16
// lanes of one LDS access (consecutive rows, one chunk) hit distinct banks
__device__ __forceinline__ int swz(int r, int c) { return r * kStageK + ((c ^ ((r >> 1) & 7)) << 4); }

// kTail: K is not a multiple of 128.  The last stage's absent blocks repeat
// bytes of the row's first present ones (nothing past a row is read), and the
// token operand's are zeroed, so they add nothing; scale rows are then only
// 2-byte aligned and come two bytes at a time.
//
// XR: token rows a slot holds.  8 or 16 where no more tokens exist (T <= XR,
// host): the lanes of the tokens beyond repeat them, and the ring is deeper (T =
// 1, K = N = 4096: 6.1 -> 5.7 us; K = 8192, N = 512: 7.6 -> 7.1).
//
// XR = 0 (kX16): p.x is bf16 [T, K], T <= 32, T K <= kMaxResident, one launch (host).  The tokens
// stay in LDS as MXFP8 rows of nk stages, swizzled like a slot's, each row an
// odd number of 128-byte stages long so that 16 rows' chunks hit distinct banks;
// only the weights go through the rings.
constexpr int kMaxResident = 65536;

// Workgroups per launch (a grid holds fewer than 2^32 threads).
constexpr uint32_t kGridMax = 1u << 22;

template <int NF, int MF, int WV, int S, bool kTail, int XR>
__global__ __launch_bounds__(64 * WV) void lin_stream_kernel(LinParams p) {
  constexpr bool kX16 = XR == 0;
  static_assert(XR == 32 * MF || (MF == 1 && (XR == 0 || XR == 8 || XR == 16)), "token rows per slot");
  constexpr int kRows = 32 * NF + XR;   // LDS rows per slot: weights, then tokens
  constexpr int kScaleOps = (kRows + 63) / 64;       // 64 rows per scale load
  constexpr int kScaleBytes = kScaleOps * 256 * (kTail ? 2 : 1);
  constexpr int kSlot = kRows * kStageK + kScaleBytes;
  constexpr int kOps = kRows / 8 + kScaleOps * (kTail ? 2 : 1);
  constexpr int kRing = WV * S * kSlot;
  constexpr int kPitch = 36;                         // floats per token row of a partial tile
  static_assert(S >= 2 && S <= 3 && (S - 1) * kOps < 64, "vmcnt range");
  static_assert(WV * NF * MF * 32 * kPitch * 4 <= kRing, "the partial tiles reuse the ring");
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRing];
  // kX16: at most T (nk + 1) stages of 128 bytes and T nk scale words; T (K + 256) and T (K + 128) / 32 bound them
  __shared__ __attribute__((aligned(16))) uint8_t xres[kX16 ? kMaxResident + 32 * 256 : 16];
  __shared__ uint32_t xsc[kX16 ? (kMaxResident + 32 * 128) / 128 : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroups go over the XCDs in turn: XCD b % 8 takes a contiguous share of
  // the tiles, cut along the longer side, so that one L2 sees an operand row.
  const uint32_t share = (p.n_tiles * p.t_tiles) >> 3, spare = (p.n_tiles * p.t_tiles) & 7;
  const uint32_t xcd = blockIdx.x & 7;
  const uint32_t id = xcd * share + std::min(xcd, spare) + (blockIdx.x >> 3) + (kX16 ? 0 : p.first8);
  const bool by_rows = p.N >= p.T;
  const uint32_t inner = by_rows ? p.t_tiles : p.n_tiles;
  const uint32_t outer_i = id / inner, inner_i = id - outer_i * inner;
  const int64_t n0 = (int64_t)(by_rows ? outer_i : inner_i) * (32 * NF);
  const int64_t t0 = (int64_t)(by_rows ? inner_i : outer_i) * (32 * MF);
  const int n_last = (int)std::min<int64_t>(p.N - 1 - n0, 32 * NF - 1);   // last row that exists
  const int t_last = (int)std::min<int64_t>(p.T - 1 - t0, 32 * MF - 1);

  // ---- loads of one stage ------------------------------------------------------------
  // instruction j fills LDS rows [8 j, 8 j + 8): lane l row 8 j + l / 8, chunk
  // position l % 8, which holds chunk (l % 8) ^ ((row / 2) % 8)
  const int drow = lane >> 3;
  const uint8_t* wbase = p.w + n0 * p.K;
  const uint8_t* xbase = p.x + t0 * p.K;
  const uint32_t ring0 = lds_offset(ring) + (uint32_t)(wave * S * kSlot);
  const uint8_t* sptr[kScaleOps];
#pragma unroll
  for (int j = 0; j < kScaleOps; ++j) {
    // (lanes past the last row repeat others)
    const int r = kX16 ? (64 * j + lane) & (32 * NF - 1) : 64 * j + lane;
    sptr[j] = r < 32 * NF ? p.ws + (n0 + std::min(r, n_last)) * p.s_stride
                          : p.xs + (t0 + std::min(r - 32 * NF, t_last)) * p.s_stride;
  }
  auto issue = [&](int ks, int slot) __attribute__((always_inline)) {
    const uint32_t dst = ring0 + (uint32_t)(slot * kSlot);
    const int present = kTail && ks == p.nk - 1 ? 2 * p.tail_blocks : 8;   // 16-byte chunks
#pragma unroll
    for (int j = 0; j < kRows / 8; ++j) {
      const int r = 8 * j + drow;
      int c = (lane & 7) ^ ((r >> 1) & 7);
      if (kTail && c >= present) c &= 1;
      const bool is_w = 8 * j < 32 * NF;
      const int row = is_w ? std::min(r, n_last) : std::min(r - 32 * NF, t_last);
      const uint32_t voff = (uint32_t)row * (uint32_t)p.K + (uint32_t)(ks * kStageK + c * 16);
      load_lds16(voff, is_w ? wbase : xbase, dst + (uint32_t)(j * 1024));
    }
#pragma unroll
    for (int j = 0; j < kScaleOps; ++j) {
      if constexpr (kTail) {
        // two pairs of scale bytes; a pair that does not exist repeats the first
        const uint8_t* s = sptr[j] + 4 * ks;
        load_lds2(s, dst + (uint32_t)(kRows * kStageK + j * 512));
        load_lds2(present > 4 ? s + 2 : s, dst + (uint32_t)(kRows * kStageK + j * 512 + 256));
      } else {
        load_lds4(sptr[j] + 4 * ks, dst + (uint32_t)(kRows * kStageK + j * 256));
      }
    }
  };

  v16f acc[NF][MF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[f][m][v] = 0.0f;

  // ---- kX16: the tokens, quantised by the workgroup ----------------------------------
  const int xstages = p.nk | 1;   // per row
  constexpr int kBlk = 2;         // blocks whose loads a thread has in flight
  const int nblk = (int)p.T * p.nk * 4;   // blocks past K are zeros
  u32x4_any xin[kX16 ? kBlk : 1][4];
  auto load_blocks = [&](int u0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      const int u = u0 + i * 64 * WV;
      const int r = u / (p.nk * 4), b = u - r * (p.nk * 4);
#pragma unroll
      for (int v = 0; v < 4; ++v) xin[i][v] = u32x4_any{0, 0, 0, 0};
      if (u < nblk && 32 * b < p.K) {
        const u32x4_any* src = reinterpret_cast<const u32x4_any*>(reinterpret_cast<const uint16_t*>(p.x) + r * p.K + 32 * b);
#pragma unroll
        for (int v = 0; v < 4; ++v) xin[i][v] = src[v];
      }
    }
  };
  auto store_blocks = [&](int u0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBlk; ++i) {
      const int u = u0 + i * 64 * WV;
      if (u >= nblk) continue;
      const int r = u / (p.nk * 4), b = u - r * (p.nk * 4);
      float v[32];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        unpack_bf16x8(make_uint4(xin[i][j].x, xin[i][j].y, xin[i][j].z, xin[i][j].w), v + 8 * j);
      uint32_t q[8];
      reinterpret_cast<uint8_t*>(xsc)[r * p.nk * 4 + b] = static_cast<uint8_t>(mx_block32(v, q));
      uint8_t* dst = xres + (r * xstages + (b >> 2)) * kStageK;
      const int c = 2 * (b & 3), sw = (r >> 1) & 7;
      *reinterpret_cast<uint4*>(dst + ((c ^ sw) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
      *reinterpret_cast<uint4*>(dst + (((c + 1) ^ sw) << 4)) = make_uint4(q[4], q[5], q[6], q[7]);
    }
  };
  if constexpr (kX16) load_blocks(tid);

  const int li = lane & 31, lg = lane >> 5;
  const int cnt = wave < p.nk ? (p.nk - wave + WV - 1) / WV : 0;   // this wave's stages
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (i < cnt) issue(wave + i * WV, i);
  if constexpr (kX16) {
    store_blocks(tid);
    for (int u = tid + kBlk * 64 * WV; u < nblk; u += kBlk * 64 * WV) {
      load_blocks(u);
      store_blocks(u);
    }
    __syncthreads();
  }
  const int xrow = std::min(li, t_last);
  int slot = 0;
  for (int i = 0; i < cnt; ++i) {
    const int ks = wave + i * WV;
    // stage i has landed once only the later stages' loads are outstanding
    const int later = std::min(cnt, i + S) - (i + 1);
    if (later == 0) wait_loads<0>();
    else if (S == 2 || later == 1) wait_loads<kOps>();
    else wait_loads<(S - 1) * kOps>();
    const uint8_t* sl = ring + wave * S * kSlot + slot * kSlot;
    const uint8_t* sc = sl + kRows * kStageK;
    v8i fa[2][NF], fb[2][MF];
    int sa[2][NF], sb[2][MF];
    auto frag = [&](int r, int s) __attribute__((always_inline)) -> v8i {
      const uint4 u0 = *reinterpret_cast<const uint4*>(sl + swz(r, 4 * s + lg));
      const uint4 u1 = *reinterpret_cast<const uint4*>(sl + swz(r, 4 * s + 2 + lg));
      return v8i{(int)u0.x, (int)u0.y, (int)u0.z, (int)u0.w, (int)u1.x, (int)u1.y, (int)u1.z, (int)u1.w};
    };
    auto scale = [&](int r, int s) __attribute__((always_inline)) -> int {
      if constexpr (kTail)   // pair s of row r: word r % 64 of its half of the row group's 512 bytes
        return sc[(r >> 6) * 512 + s * 256 + (r & 63) * 4 + lg];
      else
        return sc[r * 4 + 2 * s + lg];
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        fa[s][f] = frag(32 * f + li, s);
        sa[s][f] = scale(32 * f + li, s);
      }
#pragma unroll
      for (int m = 0; m < MF; ++m) {
        if constexpr (kX16) {
          const uint8_t* xr = xres + (xrow * xstages + ks) * kStageK;
          const int sw = (xrow >> 1) & 7;
          const uint4 u0 = *reinterpret_cast<const uint4*>(xr + (((4 * s + lg) ^ sw) << 4));
          const uint4 u1 = *reinterpret_cast<const uint4*>(xr + (((4 * s + 2 + lg) ^ sw) << 4));
          fb[s][m] = v8i{(int)u0.x, (int)u0.y, (int)u0.z, (int)u0.w, (int)u1.x, (int)u1.y, (int)u1.z, (int)u1.w};
          sb[s][m] = reinterpret_cast<const uint8_t*>(xsc)[(xrow * p.nk + ks) * 4 + 2 * s + lg];
        } else {
          const int r = 32 * (NF + m) + (XR < 32 ? li & (XR - 1) : li);
          fb[s][m] = frag(r, s);
          sb[s][m] = scale(r, s);
        }
      }
    }
    wait_lds();   // the slot is read: refill it
    if (i + S < cnt) issue(ks + S * WV, slot);
    if (kTail && !kX16 && ks == p.nk - 1) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
          for (int v = 0; v < 8; ++v)
            if (2 * s + (v >> 2) >= p.tail_blocks) fb[s][m][v] = 0;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[s][f], fb[s][m], acc[f][m], 0, 0, 0,
                                                                      sa[s][f], 0, sb[s][m]);
    slot = slot + 1 == S ? 0 : slot + 1;
  }

  // ---- the waves' partial tiles meet in LDS ----------------------------------------
  __syncthreads();   // every wave has read its last stage, and no load is outstanding
  float* part = reinterpret_cast<float*>(ring);
  constexpr int kTile = 32 * kPitch;   // one 32 x 32 fragment, token-major
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(part + (wave * NF * MF + f * MF + m) * kTile + li * kPitch + 8 * q + 4 * lg) =
            make_float4(acc[f][m][4 * q], acc[f][m][4 * q + 1], acc[f][m][4 * q + 2], acc[f][m][4 * q + 3]);
  __syncthreads();

  // four lanes per (fragment, token), 8 features each
  for (int u0 = wave * 16; u0 < NF * MF * 32; u0 += WV * 16) {   // NF MF 32 is a multiple of 16: whole quads
    const int u = u0 + (lane >> 2);
    const int f = u / (MF * 32), m = (u / 32) % MF, tl = u & 31;
    const int64_t t = t0 + 32 * m + tl;
    const int64_t n = n0 + 32 * f + 8 * (lane & 3);
    const int cnt = t < p.T ? (int)std::min<int64_t>(p.N - n, 8) : 0;
    float z[8] = {}, b[8];
    uint4 res = make_uint4(0, 0, 0, 0);
    epilogue_bias(p, n, cnt, b);
    if (p.res && cnt > 0) res = load_res8<false>(p.res + t * p.N + n, cnt);
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      const float* src = part + (w * NF * MF + f * MF + m) * kTile + tl * kPitch + 8 * (lane & 3);
      const float4 v0 = reinterpret_cast<const float4*>(src)[0], v1 = reinterpret_cast<const float4*>(src)[1];
      z[0] += v0.x; z[1] += v0.y; z[2] += v0.z; z[3] += v0.w;
      z[4] += v1.x; z[5] += v1.y; z[6] += v1.z; z[7] += v1.w;
    }
    const Place pl{t * p.N + n, t * p.ys_stride + (n >> 5), 0, 0};
    epilogue8(p, pl, n, cnt, b, res, z);
  }
}

template <int NF, int MF, int WV, int S, int XR = 32 * MF>
int launch_stream(LinParams p, hipStream_t stream) {
  p.n_tiles = (uint32_t)((p.N + 32 * NF - 1) / (32 * NF));
  p.t_tiles = (uint32_t)((p.T + 32 * MF - 1) / (32 * MF));
  const uint32_t total = p.n_tiles * p.t_tiles;   // under 2^30 (the entry point)
  for (uint32_t first = 0; first < total; first += kGridMax) {
    p.first8 = first / 8;
    const dim3 grid(std::min(total - first, kGridMax));
    if (p.K % kStageK) lin_stream_kernel<NF, MF, WV, S, true, XR><<<grid, dim3(64 * WV), 0, stream>>>(p);
    else lin_stream_kernel<NF, MF, WV, S, false, XR><<<grid, dim3(64 * WV), 0, stream>>>(p);
  }
  return check_launch("mx_linear_fused");
}

// Which kernel: the one whose time, in units of 0.1 us, a line through its
// measured times says is shortest.  Its tiles go over the CUs in rounds; a round
// costs a part per tile and a part per k stage of a wave.  Fitted to all kernels
// on 220 shapes (T to 16384, K and N to 8192, drawn over their logarithms), the
// rule's choice takes 0.3 % longer than the fastest on average, 13 % at worst.
// The smaller kernels differ only in how the tiles fill the rounds: T = 203, K =
// 2080, N = 4099 takes 19.3 us in 260 tiles of 64 x 64, 13.7 us in 903 of 32 x
// 32.  (Also measured: 32 x 32 over 8 waves, one per CU, and 64 x 32 over 6 or
// 3; they win by 0.5 % on average.  32 x 32 over 8 where one round holds the tiles:
// T = 1, K = 8192, N = 512 7.0 us instead of 7.2, rows of 2080 up to 7 % less, nearly
// all others 2 - 9 % more.)
mx_linear_kernel choose(int64_t T, int64_t K, int64_t N) {
  const int64_t cus = num_cus(), nk = (K + kStageK - 1) / kStageK;
  auto tiles = [&](int64_t bn, int64_t bm) { return ((N + bn - 1) / bn) * ((T + bm - 1) / bm); };
  auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const int64_t t32 = tiles(32, 32), t128 = tiles(128, 128);
  const bool big = N >= (int64_t)1 << 27;   // the tile kernels' 32-bit offsets within 8 rows
  const int64_t us[7] = {   // in mx_linear_kernel's order
      // K over 4 waves, two workgroups per CU
      t32 <= cus ? 35 + 5 * up(nk, 4) : up(t32, 2 * cus) * (33 + 7 * up(nk, 4)),
      up(tiles(64, 64), cus) * (44 + 11 * up(nk, 4)),           // over 4
      up(tiles(64, 96), cus) * (64 + 25 * up(nk, 3) / 2),       // over 3
      up(tiles(64, 64), 2 * cus) * (64 + 10 * up(nk, 2)),       // over 2, two workgroups per CU
      big ? INT64_MAX : t128 <= cus ? 82 + 17 * nk / 2 : up(t128, 2 * cus) * (82 + 11 * nk),   // two per CU
      big || nk < 3 ? INT64_MAX : up(tiles(256, 128), cus) * (100 + 9 * nk),
      big ? INT64_MAX : up(tiles(256, 256), cus) * (174 + 14 * nk)};
  return static_cast<mx_linear_kernel>(std::min_element(us, us + 7) - us);
}

int launch_linear(const LinParams& p, hipStream_t stream) {
  switch (choose(p.T, p.K, p.N)) {
    case MX_LINEAR_32X32:
      if (p.T <= 8) return launch_stream<1, 1, 4, 3, 8>(p, stream);
      if (p.T <= 16) return launch_stream<1, 1, 4, 3, 16>(p, stream);
      return launch_stream<1, 1, 4, 2>(p, stream);
    case MX_LINEAR_64X64: return launch_stream<2, 2, 4, 2>(p, stream);
    case MX_LINEAR_64X96: return launch_stream<2, 3, 3, 2>(p, stream);
    case MX_LINEAR_64X64_TWICE: return launch_stream<2, 2, 2, 2>(p, stream);
    case MX_LINEAR_128X128: return launch_lin_tile128(p, stream);
    case MX_LINEAR_256X128: return launch_lin_tile256x128(p, stream);
    default: return launch_lin_tile256(p, stream);
  }
}

// bf16 tokens that every workgroup quantises for itself (no workspace): few of
// them, and no more workgroups than CUs.  It is one launch in the place of two, 4 us
// of host work less, and one copy of the tokens per workgroup.  On the GPU alone
// (in place against quantiser + product, K = 2048): N = 2048 4.9 / 6.1 us at T = 1,
// 6.4 / 6.7 at T = 16, 8.5 / 7.1 at T = 32, where the workgroup's arithmetic
// shows; N = 8192 6.4 / 7.4, 7.6 / 7.8, 9.7 / 7.9.  Its LDS leaves one workgroup to a
// CU, and every round of them quantises again: N = 8224 9.0 / 8.0, 11.8 / 8.9, 15.7 /
// 9.2; N = 131072 75 / 51, 99 / 56, 129 / 63.
constexpr int64_t kMaxResidentN = 32 * 256;   // (a constant: the workspace query has no device)
bool resident(int64_t T, int64_t K, int64_t N) { return T <= 32 && T * K <= kMaxResident && N <= kMaxResidentN; }

// Workspace: the MXFP8 form of bf16 tokens.
struct FusedLayout {
  size_t xq, xs, total;
};
FusedLayout fused_layout(int64_t T, int64_t K, int64_t N, int x_is_mx) {
  FusedLayout L{0, 0, 0};
  if (x_is_mx || resident(T, K, N)) return L;
  L.xs = align_up((size_t)(T * K), 256);
  L.total = L.xs + align_up((size_t)(T * 2 * ((K + 63) / 64)), 256);
  return L;
}

// Tile indices are 32-bit in every kernel, also a round past the last: an output of a TB.
bool too_many_tiles(int64_t T, int64_t N) { return ((T + 31) / 32) * ((N + 31) / 32) >= (int64_t)1 << 30; }
int fail_tiles() { return fail(MX_ERR_UNSUPPORTED, "mx_linear_fused: 2^30 or more tiles of 32 x 32 outputs"); }

int check_sizes(int64_t T, int64_t K, int64_t N) {
  if (T < 0 || K <= 0 || N <= 0)
    return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: bad sizes T=%lld K=%lld N=%lld", (long long)T, (long long)K,
                (long long)N);
  if (!dims_in_range({T, N})) return fail(MX_ERR_UNSUPPORTED, "mx_linear_fused: T or N above 2^31 - 1");
  if (K % 32 != 0) return fail(MX_ERR_UNSUPPORTED, "mx_linear_fused: K=%lld is not a multiple of 32", (long long)K);
  if (K > kMaxK) return fail(MX_ERR_UNSUPPORTED, "mx_linear_fused: K=%lld > 2^20", (long long)K);
  return MX_OK;
}

}  // namespace

}  // namespace mxmoe

extern "C" size_t mx_linear_fused_workspace_size(int64_t T, int64_t K, int64_t N, int x_is_mx) {
  // 0 for sizes mx_linear_fused rejects
  if (mxmoe::check_sizes(T, K, N) != MX_OK || mxmoe::too_many_tiles(T, N)) return 0;
  return mxmoe::fused_layout(T, K, N, x_is_mx).total;
}

extern "C" int mx_linear_fused_kernel(int64_t T, int64_t K, int64_t N, int x_is_mx) {
  using namespace mxmoe;
  const int rc = check_sizes(T, K, N);
  if (rc) return rc;
  if (T == 0) return fail(MX_ERR_INVALID_ARG, "mx_linear_fused_kernel: no tokens");
  if (too_many_tiles(T, N)) return fail_tiles();
  return !x_is_mx && resident(T, K, N) ? MX_LINEAR_32X32_BF16 : choose(T, K, N);
}

extern "C" int mx_linear_fused(const void* x, const void* x_s, const void* w_u8, const void* w_s, const void* bias,
                               int bias_type, int activation, const void* residual_bf16, int64_t T, int64_t K,
                               int64_t N, void* y_bf16, void* yq_u8, void* ys_u8, void* workspace, size_t ws_bytes,
                               void* stream) {
  using namespace mxmoe;
  int rc = check_sizes(T, K, N);
  if (rc) return rc;
  if (bias && bias_type != MX_TYPE_BF16 && bias_type != MX_TYPE_F32)
    return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: bias_type must be MX_TYPE_BF16 or MX_TYPE_F32, got %d",
                bias_type);
  if (activation < MX_ACT_NONE || activation > MX_ACT_GELU_TANH)
    return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: unknown activation %d", activation);
  if (!yq_u8 != !ys_u8) return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: yq and ys go together");
  if (y_bf16 && yq_u8) return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: y or (yq, ys), not both");
  const FusedLayout L = fused_layout(T, K, N, x_s != nullptr);
  if (T > 0 && (!x || !w_u8 || !w_s || (!y_bf16 && !yq_u8) || (L.total > 0 && !workspace)))
    return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: null pointer");
  if (ws_bytes < L.total)
    return fail(MX_ERR_WORKSPACE, "mx_linear_fused: workspace %zu bytes < %zu", ws_bytes, L.total);
  const bool mx_in = x_s != nullptr;
  if (reinterpret_cast<uintptr_t>(x) % (mx_in ? 16 : 2) || reinterpret_cast<uintptr_t>(w_u8) % 16 ||
      reinterpret_cast<uintptr_t>(x_s) % 4 || reinterpret_cast<uintptr_t>(w_s) % 4 ||
      reinterpret_cast<uintptr_t>(bias) % (bias_type == MX_TYPE_F32 ? 4 : 2) ||
      reinterpret_cast<uintptr_t>(residual_bf16) % 2 || reinterpret_cast<uintptr_t>(y_bf16) % 2 ||
      (L.total > 0 && reinterpret_cast<uintptr_t>(workspace) % 256))
    return fail(MX_ERR_UNSUPPORTED, "mx_linear_fused: misaligned pointer");
  if (T == 0) return MX_OK;
  LinParams p{};
  p.T = T;
  p.K = K;
  p.N = N;
  p.s_stride = 2 * ((K + 63) / 64);
  p.ys_stride = 2 * ((N + 63) / 64);
  p.nk = (int)((K + kStageK - 1) / kStageK);
  p.tail_blocks = (int)((K - (int64_t)(p.nk - 1) * kStageK) / 32);
  p.w = static_cast<const uint8_t*>(w_u8);
  p.ws = static_cast<const uint8_t*>(w_s);
  p.bias = bias;
  p.bias_f32 = bias_type == MX_TYPE_F32;
  p.act = activation;
  p.res = static_cast<const uint16_t*>(residual_bf16);
  p.y = static_cast<uint16_t*>(y_bf16);
  p.yq = static_cast<uint8_t*>(yq_u8);
  p.ys = static_cast<uint8_t*>(ys_u8);
  // measured at N = 4096: non-temporal residual loads 282 -> 267 us at T = 16384
  // (134 MB), 46 -> 49 us at T = 4096 (34 MB)
  p.stream_res = T * N > (int64_t)48 << 20;
  // Outputs overlap nothing, except that y may take the residual's place.
  const uint64_t s_bytes = (uint64_t)p.s_stride, dense = (uint64_t)T * (uint64_t)N;
  const Span in[7] = {{x, (uint64_t)T * (uint64_t)K * (mx_in ? 1 : 2)},
                      {x_s, (uint64_t)T * s_bytes},
                      {w_u8, (uint64_t)N * (uint64_t)K},
                      {w_s, (uint64_t)N * s_bytes},
                      {bias, (uint64_t)N * (p.bias_f32 ? 4 : 2)},
                      {workspace, L.total},
                      {residual_bf16, dense * 2}};
  const Span out[3] = {{y_bf16, dense * 2}, {yq_u8, dense}, {ys_u8, (uint64_t)T * (uint64_t)p.ys_stride}};
  for (int o = 0; o < 3; ++o)
    for (int i = 0; i < 7; ++i)
      if (overlaps(out[o], in[i]) && !(o == 0 && i == 6 && y_bf16 == residual_bf16))
        return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: an output overlaps an input or the workspace");
  if (overlaps(out[1], out[2])) return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: two outputs overlap");
  for (int i = 0; i < 7; ++i)
    if (i != 5 && overlaps(in[5], in[i]))
      return fail(MX_ERR_INVALID_ARG, "mx_linear_fused: the workspace overlaps an input");
  if (too_many_tiles(T, N)) return fail_tiles();
  hipStream_t s = as_stream(stream);
  if (mx_in) {
    p.x = static_cast<const uint8_t*>(x);
    p.xs = static_cast<const uint8_t*>(x_s);
  } else if (resident(T, K, N)) {
    p.x = static_cast<const uint8_t*>(x);
    return launch_stream<1, 1, 8, 2, 0>(p, s);
  } else {
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + L.xs;
    rc = launch_mx_quantize(static_cast<const uint16_t*>(x), T, K, K, xq, xs, s);
    if (rc) return rc;
    p.x = xq;
    p.xs = xs;
  }
  return launch_linear(p, s);
}
