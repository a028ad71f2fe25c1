// moe_unpermute and moe_unpermute_backward: expert rows back to their tokens,
// and the gradients of that.  With p(i) = expanded_row_idx[i], i = t k + j, over
// the i whose p(i) is a row:
//
//   forward   out[t] = sum_j w[t, j] y[p(i)]
//   backward  dy[p(i)] = w[t, j] dout[t],   dw[t, j] = sum_c dout[t, c] y[p(i), c]
//
// in fp32, each output rounded once; without weights w = 1, and the forward is
// then the gradient of moe_permute.
//
// Rows of any width and alignment move 16 bytes a lane (gfx950 does them in one
// instruction on any boundary of elements): piece i of a row starts at byte 16 i,
// its last piece 16 bytes before its end, so that some elements may come twice,
// with the same result.  All of it is bound by HBM, or for few tokens by the launch:
// 16384 tokens of 2048 bf16 with 8 rows each take 112 us (5.4 TB/s) forward, 224 us
// (5.1) backward, 106 us (5.7) without dw; 2049 of 1001 fp16 8.9 us; 64 of 4096 with 2
// rows each 3.2 us backward.  (A binding that clears dy first, for the rows that no
// entry names, adds a pass over it: 330 us.)
#include <algorithm>
#include <type_traits>

#include "fused.h"

namespace mxmoe {

namespace {

struct UnpermuteParams {
  const uint8_t* y;      // [M, K]
  const uint8_t* dout;   // [T, K] (backward)
  const float* w;        // [T, k], or null
  const int32_t* eri;    // [T k]
  uint8_t* out;          // [T, K]; backward: dy [M, K]
  float* dw;             // [T, k], or null (backward)
  int64_t T, K, M;
  int64_t row_bytes;
  int k;
};

template <int kType>
struct Elem {
  static constexpr int kBytes = kType == MX_TYPE_F32 ? 4 : 2;
  static constexpr int kPer = 16 / kBytes;   // elements of a piece
};

template <int kType>
__device__ __forceinline__ void unpack(const u32x4_any& u, float (&v)[Elem<kType>::kPer]) {
  if constexpr (kType == MX_TYPE_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(u[i]);
  } else if constexpr (kType == MX_TYPE_BF16) {
    unpack_bf16x8(make_uint4(u.x, u.y, u.z, u.w), v);
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)u[i]);
      v[2 * i] = (float)h.x;
      v[2 * i + 1] = (float)h.y;
    }
  }
}

template <int kType>
__device__ __forceinline__ u32x4_any pack(const float (&v)[Elem<kType>::kPer]) {
  if constexpr (kType == MX_TYPE_F32) {
    return u32x4_any{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else if constexpr (kType == MX_TYPE_BF16) {
    return u32x4_any{bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7])};
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    u32x4_any u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
    return u;
  }
}

template <int kType>
__device__ __forceinline__ float load1(const uint8_t* p) {
  if constexpr (kType == MX_TYPE_F32) return *reinterpret_cast<const float*>(p);
  else if constexpr (kType == MX_TYPE_BF16) return bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
  else return (float)*reinterpret_cast<const _Float16*>(p);
}
template <int kType>
__device__ __forceinline__ void store1(uint8_t* p, float v) {
  if constexpr (kType == MX_TYPE_F32) *reinterpret_cast<float*>(p) = v;
  else if constexpr (kType == MX_TYPE_BF16) *reinterpret_cast<uint16_t*>(p) = (uint16_t)bf16x2(v, v);
  else *reinterpret_cast<_Float16*>(p) = (_Float16)v;
}

__device__ __forceinline__ u32x4_any load_piece(const uint8_t* p) {
  return *reinterpret_cast<const u32x4_any*>(p);
}
__device__ __forceinline__ void store_piece(uint8_t* p, const u32x4_any& u) {
  __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any*>(p));
}

constexpr int kThreads = 256;

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// kLanes = 64: a wave takes 64 pieces of a token at a time, whose k indices and
// weights come through the scalar unit.  16: rows of 16 pieces at most, four tokens
// a wave.  The rows of kBatch assignments are requested before they are added.
template <int kType, int kLanes>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(UnpermuteParams p) {
  constexpr int kPer = Elem<kType>::kPer, kBatch = 8;
  const int lane = threadIdx.x & 63;
  const int64_t pieces = (p.row_bytes + 15) / 16;
  const int64_t blocks = (pieces + 63) / 64;   // of a row; 1 when kLanes = 16
  const int64_t units = kLanes == 64 ? p.T * blocks : (p.T + 3) / 4;
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t u = first; u < units; u += (int64_t)gridDim.x * (kThreads / 64)) {
    const int64_t t = kLanes == 64 ? uniform(u / blocks) : 4 * u + lane / kLanes;
    const int64_t piece = kLanes == 64 ? (u - t * blocks) * 64 + lane : lane % kLanes;
    if (piece >= pieces || t >= p.T) continue;
    const int64_t at = std::min<int64_t>(16 * piece, p.row_bytes - 16);
    float acc[kPer] = {};
    for (int j0 = 0; j0 < p.k; j0 += kBatch) {
      u32x4_any row[kBatch];
      int32_t r[kBatch];
      float w[kBatch];
      bool ok[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {   // (assignments past the last repeat it)
        const int64_t i = t * p.k + std::min(j0 + b, p.k - 1);
        r[b] = p.eri[i];
        w[b] = p.w ? p.w[i] : 1.0f;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        ok[b] = j0 + b < p.k && r[b] >= 0 && r[b] < p.M;
        if (ok[b]) row[b] = load_piece(p.y + r[b] * p.row_bytes + at);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!ok[b]) continue;
        float v[kPer];
        unpack<kType>(row[b], v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += w[b] * v[i];
      }
    }
    store_piece(p.out + t * p.row_bytes + at, pack<kType>(acc));
  }
}

// Rows of fewer than 16 bytes: an element a thread.
template <int kType>
__global__ __launch_bounds__(kThreads) void unpermute_tiny(UnpermuteParams p) {
  const int64_t total = p.T * p.K;
  for (int64_t it = blockIdx.x * (int64_t)kThreads + threadIdx.x; it < total; it += (int64_t)gridDim.x * kThreads) {
    const int64_t t = it / p.K, at = (it - t * p.K) * Elem<kType>::kBytes;
    float acc = 0.0f;
    for (int j = 0; j < p.k; ++j) {
      const int32_t r = p.eri[t * p.k + j];
      if (r < 0 || r >= p.M) continue;
      acc += (p.w ? p.w[t * p.k + j] : 1.0f) * load1<kType>(p.y + r * p.row_bytes + at);
    }
    store1<kType>(p.out + t * p.row_bytes + at, acc);
  }
}

// The sum over 16 lanes (a DPP row), in its last lane.
__device__ __forceinline__ float row_sum16(float x) {
  x += dpp_f32<0x111>(0.0f, x);   // row_shr:1
  x += dpp_f32<0x112>(0.0f, x);   // row_shr:2
  x += dpp_f32<0x114>(0.0f, x);   // row_shr:4
  x += dpp_f32<0x118>(0.0f, x);   // row_shr:8
  return x;
}

// W waves share a token (four tokens of one wave each in a workgroup, or with
// kLanes = 16 four tokens a wave), whose row of dout stays in registers, C pieces a
// lane, while its rows of y are read and those of dy written, kBatch assignments at
// a time.  With few tokens `splits` workgroups (waves) share a token's assignments,
// `per` each.
template <int kType, int W, int C, int kLanes>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void unpermute_backward_kernel(UnpermuteParams p, int splits, int per) {
  constexpr int kPer = Elem<kType>::kPer, kBytes = Elem<kType>::kBytes, kBatch = 2;
  constexpr int kUnits = W < 4 ? 4 : 1;   // per workgroup
  static_assert(W == 1 || (W >= 4 && kLanes == 64), "a wave per token, or the workgroup's waves share one");
  __shared__ float part[kBatch][W];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t pieces = (p.row_bytes + 15) / 16;
  const int64_t units = (kLanes == 64 ? p.T : (p.T + 3) / 4) * splits;
  const int64_t first = (int64_t)blockIdx.x * kUnits + (W == 1 ? __builtin_amdgcn_readfirstlane(tid >> 6) : 0);
  for (int64_t u = first; u < units; u += (int64_t)gridDim.x * kUnits) {
    const int64_t tb = uniform(u / splits);
    const int j0 = (int)(u - tb * splits) * per, j1 = std::min(j0 + per, p.k);
    const int64_t t = kLanes == 64 ? tb : 4 * tb + lane / kLanes;
    const bool real = kLanes == 64 || t < p.T;
    u32x4_any d[C];
    int64_t at[C];
    bool has[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t piece = W == 1 ? c * kLanes + lane % kLanes : c * 64 * W + tid;
      has[c] = real && piece < pieces;
      at[c] = std::min<int64_t>(16 * piece, p.row_bytes - 16);
      if (has[c]) d[c] = load_piece(p.dout + t * p.row_bytes + at[c]);
    }
    for (int j = j0; j < j1; j += kBatch) {
      int32_t r[kBatch];
      float w[kBatch], sum[kBatch];
      bool ok[kBatch];
      u32x4_any y[kBatch][C];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        // (assignments past the last repeat it)
        const int64_t i = (real ? t : 0) * p.k + std::min(j + b, j1 - 1);
        r[b] = p.eri[i];
        w[b] = p.w ? p.w[i] : 1.0f;
        sum[b] = 0.0f;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        ok[b] = real && j + b < j1 && r[b] >= 0 && r[b] < p.M;
        if (p.dw && ok[b]) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (has[c]) y[b][c] = load_piece(p.y + r[b] * p.row_bytes + at[c]);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!ok[b]) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (!has[c]) continue;
          float v[kPer];
          unpack<kType>(d[c], v);
          if (p.dw) {
            float z[kPer];
            unpack<kType>(y[b][c], z);
            const int64_t piece = W == 1 ? c * kLanes + lane % kLanes : c * 64 * W + tid;
            const int skip = (int)(16 * piece - at[c]) / kBytes;   // elements that the piece before holds too
#pragma unroll
            for (int e = 0; e < kPer; ++e) sum[b] += e >= skip ? v[e] * z[e] : 0.0f;
          }
#pragma unroll
          for (int e = 0; e < kPer; ++e) v[e] *= w[b];
          store_piece(p.out + r[b] * p.row_bytes + at[c], pack<kType>(v));
        }
      }
      if (!p.dw) continue;
      if constexpr (kLanes == 16) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          sum[b] = row_sum16(sum[b]);
          if (lane % 16 == 15 && real && j + b < j1) p.dw[t * p.k + j + b] = sum[b];
        }
      } else {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) sum[b] = wave_sum(sum[b]);
        if constexpr (W > 1) {
          __syncthreads();   // the last partials are read
          if (lane == 0) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) part[b][tid >> 6] = sum[b];
          }
          __syncthreads();
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            sum[b] = 0.0f;
#pragma unroll
            for (int i = 0; i < W; ++i) sum[b] += part[b][i];
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (j + b < j1 && (W == 1 ? lane : tid) == b) p.dw[t * p.k + j + b] = sum[b];
      }
    }
  }
}

// Rows of more than 64 KB: a workgroup per assignment, dout read for each.
constexpr int kLongWaves = 16;
template <int kType>
__global__ __launch_bounds__(64 * kLongWaves) void unpermute_backward_long(UnpermuteParams p) {
  constexpr int kPer = Elem<kType>::kPer, kBytes = Elem<kType>::kBytes;
  __shared__ float part[kLongWaves];
  const int64_t total = p.T * p.k;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int64_t t = i / p.k;
    const int32_t r = p.eri[i];
    float sum = 0.0f;
    if (r >= 0 && r < p.M) {
      const float w = p.w ? p.w[i] : 1.0f;
      for (int64_t b = 16 * (int64_t)threadIdx.x; b < p.row_bytes; b += 16 * 64 * kLongWaves) {
        const int64_t at = std::min<int64_t>(b, p.row_bytes - 16);
        const int skip = (int)(b - at) / kBytes;   // elements that the piece before holds too
        float d[kPer];
        unpack<kType>(load_piece(p.dout + t * p.row_bytes + at), d);
        if (p.dw) {
          float v[kPer];
          unpack<kType>(load_piece(p.y + r * p.row_bytes + at), v);
#pragma unroll
          for (int e = 0; e < kPer; ++e) sum += e >= skip ? d[e] * v[e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) d[e] *= w;
        store_piece(p.out + r * p.row_bytes + at, pack<kType>(d));
      }
    }
    if (!p.dw) continue;
    sum = wave_sum(sum);
    __syncthreads();   // the last assignment's partials are read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kLongWaves; ++w) sum += part[w];
      p.dw[i] = sum;
    }
  }
}

// Rows of fewer than 16 bytes: an assignment a thread.
template <int kType>
__global__ __launch_bounds__(kThreads) void unpermute_backward_tiny(UnpermuteParams p) {
  constexpr int kBytes = Elem<kType>::kBytes;
  const int64_t total = p.T * p.k;
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t t = i / p.k;
    const int32_t r = p.eri[i];
    float sum = 0.0f;
    if (r >= 0 && r < p.M) {
      const float w = p.w ? p.w[i] : 1.0f;
      for (int c = 0; c < (int)p.K; ++c) {
        const float d = load1<kType>(p.dout + t * p.row_bytes + c * kBytes);
        if (p.dw) sum += d * load1<kType>(p.y + r * p.row_bytes + c * kBytes);
        store1<kType>(p.out + r * p.row_bytes + c * kBytes, d * w);
      }
    }
    if (p.dw) p.dw[i] = sum;
  }
}

// Entries a token may have: one wave or thread takes a token's in turn, and their
// indices, a batch or a share past the last included, are ints.
constexpr int64_t kMaxEntries = (int64_t)1 << 20;

int64_t elem_bytes(int type) { return type == MX_TYPE_F32 ? 4 : 2; }

int check_unpermute(const char* name, int type, int64_t T, int64_t K, int64_t k, int64_t M) {
  if (T < 0 || K <= 0 || k <= 0 || M < 0)
    return fail(MX_ERR_INVALID_ARG, "%s: bad sizes T=%lld K=%lld k=%lld M=%lld", name, (long long)T, (long long)K,
                (long long)k, (long long)M);
  if (type != MX_TYPE_BF16 && type != MX_TYPE_F32 && type != MX_TYPE_F16)
    return fail(MX_ERR_INVALID_ARG, "%s: type must be MX_TYPE_BF16, MX_TYPE_F32 or MX_TYPE_F16, got %d", name, type);
  if (!dims_in_range({T, k, M})) return fail(MX_ERR_UNSUPPORTED, "%s: T, k or M above 2^31 - 1", name);
  if (K > (int64_t)1 << 24) return fail(MX_ERR_UNSUPPORTED, "%s: K=%lld > 2^24", name, (long long)K);
  if (k > kMaxEntries) return fail(MX_ERR_UNSUPPORTED, "%s: k=%lld > 2^20", name, (long long)k);
  if (T * k >= (int64_t)1 << 31) return fail(MX_ERR_UNSUPPORTED, "%s: T*k >= 2^31", name);
  return MX_OK;
}

template <class F>
int by_type(int type, F f) {
  if (type == MX_TYPE_F32) return f(std::integral_constant<int, MX_TYPE_F32>{});
  if (type == MX_TYPE_F16) return f(std::integral_constant<int, MX_TYPE_F16>{});
  return f(std::integral_constant<int, MX_TYPE_BF16>{});
}

int launch_unpermute(const UnpermuteParams& p, int type, hipStream_t stream) {
  const int64_t pieces = (p.row_bytes + 15) / 16, cap = (int64_t)num_cus() * 32;
  return by_type(type, [&](auto t) {
    constexpr int kType = decltype(t)::value;
    auto grid = [&](int64_t n, int64_t per) { return dim3((unsigned)std::min<int64_t>((n + per - 1) / per, cap)); };
    // rows of 16 pieces share waves: 65536 tokens, 8 experts each, 128 bf16 30 us, a wave each 48
    if (p.row_bytes < 16) unpermute_tiny<kType><<<grid(p.T * p.K, kThreads), dim3(kThreads), 0, stream>>>(p);
    else if (pieces <= 16) unpermute_kernel<kType, 16><<<grid((p.T + 3) / 4, 4), dim3(kThreads), 0, stream>>>(p);
    else unpermute_kernel<kType, 64><<<grid(p.T * ((pieces + 63) / 64), 4), dim3(kThreads), 0, stream>>>(p);
    return check_launch("moe_unpermute");
  });
}

int launch_unpermute_backward(const UnpermuteParams& p, int type, hipStream_t stream) {
  const int64_t pieces = (p.row_bytes + 15) / 16, cap = (int64_t)num_cus() * 32;
  return by_type(type, [&](auto t) {
    constexpr int kType = decltype(t)::value;
    auto grid = [&](int64_t n, int64_t per) { return dim3((unsigned)std::min<int64_t>((n + per - 1) / per, cap)); };
    // a token's assignments over several units until there are four workgroups a CU
    // (8 experts of a token, 64 tokens of 2048 bf16: 3.5 us, unsplit 13.3)
    auto go = [&](auto w, auto c, auto lanes) {
      constexpr int W = decltype(w)::value, C = decltype(c)::value, L = decltype(lanes)::value;
      const int64_t tokens = L == 64 ? p.T : (p.T + 3) / 4, in_wg = W < 4 ? 4 : 1;
      const int64_t want = (int64_t)num_cus() * 4 * in_wg;
      const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(p.k, want / tokens));
      const int64_t per = (p.k + splits - 1) / splits, used = (p.k + per - 1) / per;
      unpermute_backward_kernel<kType, W, C, L><<<grid(tokens * used, in_wg), dim3(64 * (W < 4 ? 4 : W)), 0, stream>>>(
          p, (int)used, (int)per);
    };
    // As many waves as a token's row has pieces for, one each lane: more waves than
    // with several pieces a lane, and a token's loads all in flight (16384 tokens, 8
    // experts each, 2048 bf16: 4 waves 224 us, one wave of 4 pieces a lane 230; 2049 tokens,
    // 4 experts, 2100 bf16: 8 waves 19.9, 4 of 4 pieces 21.9; 256 tokens, 4 experts, 8192:
    // 16 waves 10.0, 4 of 4 pieces 10.5).  Two pieces a lane of one wave take less than
    // 4 waves half idle (1000 tokens, 8 experts, 1024 bf16: 7.6, 9.9); rows of 16
    // pieces share waves (65536 tokens, 8 experts, 128 bf16: 59, a wave each 122).
    using std::integral_constant;
    if (p.row_bytes < 16) unpermute_backward_tiny<kType><<<grid(p.T * p.k, kThreads), dim3(kThreads), 0, stream>>>(p);
    else if (pieces <= 16) go(integral_constant<int, 1>{}, integral_constant<int, 1>{}, integral_constant<int, 16>{});
    else if (pieces <= 64) go(integral_constant<int, 1>{}, integral_constant<int, 1>{}, integral_constant<int, 64>{});
    else if (pieces <= 128) go(integral_constant<int, 1>{}, integral_constant<int, 2>{}, integral_constant<int, 64>{});
    else if (pieces <= 256) go(integral_constant<int, 4>{}, integral_constant<int, 1>{}, integral_constant<int, 64>{});
    else if (pieces <= 512) go(integral_constant<int, 8>{}, integral_constant<int, 1>{}, integral_constant<int, 64>{});
    else if (pieces <= 1024) go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, integral_constant<int, 64>{});
    else if (pieces <= 4096) go(integral_constant<int, 16>{}, integral_constant<int, 4>{}, integral_constant<int, 64>{});
    else unpermute_backward_long<kType><<<grid(p.T * p.k, 1), dim3(64 * kLongWaves), 0, stream>>>(p);
    return check_launch("moe_unpermute_backward");
  });
}

}  // namespace

}  // namespace mxmoe

extern "C" int moe_unpermute(const void* y, int type, const float* topk_w, const int32_t* expanded_row_idx, int64_t T,
                             int64_t K, int64_t k, int64_t M, void* out, void* stream) {
  using namespace mxmoe;
  int rc = check_unpermute("moe_unpermute", type, T, K, k, M);
  if (rc) return rc;
  if (T == 0) return MX_OK;
  if (!expanded_row_idx || !out || (M > 0 && !y)) return fail(MX_ERR_INVALID_ARG, "moe_unpermute: null pointer");
  const uintptr_t es = (uintptr_t)elem_bytes(type);
  if (reinterpret_cast<uintptr_t>(y) % es || reinterpret_cast<uintptr_t>(out) % es ||
      reinterpret_cast<uintptr_t>(topk_w) % 4 || reinterpret_cast<uintptr_t>(expanded_row_idx) % 4)
    return fail(MX_ERR_UNSUPPORTED, "moe_unpermute: misaligned pointer");
  UnpermuteParams p{};
  p.y = static_cast<const uint8_t*>(y);
  p.w = topk_w;
  p.eri = expanded_row_idx;
  p.out = static_cast<uint8_t*>(out);
  p.T = T; p.K = K; p.M = M; p.k = (int)k;
  p.row_bytes = K * (int64_t)es;
  const uint64_t row = (uint64_t)p.row_bytes, n = (uint64_t)(T * k);
  const Span o = {out, (uint64_t)T * row};
  if (overlaps(o, {y, (uint64_t)M * row}) || overlaps(o, {topk_w, n * 4}) || overlaps(o, {expanded_row_idx, n * 4}))
    return fail(MX_ERR_INVALID_ARG, "moe_unpermute: the output overlaps an input");
  return launch_unpermute(p, type, as_stream(stream));
}

extern "C" int moe_unpermute_backward(const void* dout, int type, const void* y, const float* topk_w,
                                      const int32_t* expanded_row_idx, int64_t T, int64_t K, int64_t k, int64_t M,
                                      void* dy, float* dw, void* stream) {
  using namespace mxmoe;
  int rc = check_unpermute("moe_unpermute_backward", type, T, K, k, M);
  if (rc) return rc;
  if (dw && M > 0 && !y) return fail(MX_ERR_INVALID_ARG, "moe_unpermute_backward: dw needs y");
  if (T == 0) return MX_OK;
  if (!dout || !expanded_row_idx || (M > 0 && !dy))
    return fail(MX_ERR_INVALID_ARG, "moe_unpermute_backward: null pointer");
  const uintptr_t es = (uintptr_t)elem_bytes(type);
  if (reinterpret_cast<uintptr_t>(dout) % es || reinterpret_cast<uintptr_t>(y) % es ||
      reinterpret_cast<uintptr_t>(dy) % es || reinterpret_cast<uintptr_t>(topk_w) % 4 ||
      reinterpret_cast<uintptr_t>(expanded_row_idx) % 4 || reinterpret_cast<uintptr_t>(dw) % 4)
    return fail(MX_ERR_UNSUPPORTED, "moe_unpermute_backward: misaligned pointer");
  UnpermuteParams p{};
  p.y = static_cast<const uint8_t*>(y);
  p.dout = static_cast<const uint8_t*>(dout);
  p.w = topk_w;
  p.eri = expanded_row_idx;
  p.out = static_cast<uint8_t*>(dy);
  p.dw = dw;
  p.T = T; p.K = K; p.M = M; p.k = (int)k;
  p.row_bytes = K * (int64_t)es;
  const uint64_t row = (uint64_t)p.row_bytes, n = (uint64_t)(T * k);
  const Span in[4] = {{dout, (uint64_t)T * row}, {y, (uint64_t)M * row}, {topk_w, n * 4}, {expanded_row_idx, n * 4}};
  const Span out[2] = {{dy, (uint64_t)M * row}, {dw, n * 4}};
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 4; ++i)
      if (overlaps(out[o], in[i])) return fail(MX_ERR_INVALID_ARG, "moe_unpermute_backward: an output overlaps an input");
  if (overlaps(out[0], out[1])) return fail(MX_ERR_INVALID_ARG, "moe_unpermute_backward: the outputs overlap");
  return launch_unpermute_backward(p, type, as_stream(stream));
}
