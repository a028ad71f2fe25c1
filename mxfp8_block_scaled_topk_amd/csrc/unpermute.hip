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
// with the same result.
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

template <int kType>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(UnpermuteParams p) {
  constexpr int kPer = Elem<kType>::kPer;
  const int64_t pieces = (p.row_bytes + 15) / 16;
  const int64_t total = p.T * pieces;
  for (int64_t it = blockIdx.x * (int64_t)kThreads + threadIdx.x; it < total; it += (int64_t)gridDim.x * kThreads) {
    const int64_t t = it / pieces;
    const int64_t at = std::min<int64_t>(16 * (it - t * pieces), p.row_bytes - 16);
    float acc[kPer] = {};
    for (int j = 0; j < p.k; ++j) {
      const int32_t r = p.eri[t * p.k + j];
      if (r < 0 || r >= p.M) continue;
      float v[kPer];
      unpack<kType>(load_piece(p.y + r * p.row_bytes + at), v);
      const float w = p.w ? p.w[t * p.k + j] : 1.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] += w * v[i];
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

// One workgroup per assignment.
template <int kType>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(UnpermuteParams p) {
  constexpr int kPer = Elem<kType>::kPer, kBytes = Elem<kType>::kBytes;
  __shared__ float part[kThreads / 64];
  const int64_t total = p.T * p.k;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int64_t t = i / p.k;
    const int32_t r = p.eri[i];
    const bool real = r >= 0 && r < p.M;
    float sum = 0.0f;
    if (real) {
      const float w = p.w ? p.w[i] : 1.0f;
      if (p.row_bytes >= 16) {
        for (int64_t b = 16 * (int64_t)threadIdx.x; b < p.row_bytes; b += 16 * kThreads) {
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
      } else if (threadIdx.x < p.K) {
        const int64_t at = threadIdx.x * kBytes;
        const float d = load1<kType>(p.dout + t * p.row_bytes + at);
        if (p.dw) sum = d * load1<kType>(p.y + r * p.row_bytes + at);
        store1<kType>(p.out + r * p.row_bytes + at, d * w);
      }
    }
    if (!p.dw) continue;
    sum = wave_sum(sum);
    __syncthreads();   // the previous assignment's partials are read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) p.dw[i] = (part[0] + part[1]) + (part[2] + part[3]);
  }
}

int64_t elem_bytes(int type) { return type == MX_TYPE_F32 ? 4 : 2; }

int check_unpermute(const char* name, int type, int64_t T, int64_t K, int64_t k, int64_t M) {
  if (T < 0 || K <= 0 || k <= 0 || M < 0)
    return fail(MX_ERR_INVALID_ARG, "%s: bad sizes T=%lld K=%lld k=%lld M=%lld", name, (long long)T, (long long)K,
                (long long)k, (long long)M);
  if (type != MX_TYPE_BF16 && type != MX_TYPE_F32 && type != MX_TYPE_F16)
    return fail(MX_ERR_INVALID_ARG, "%s: type must be MX_TYPE_BF16, MX_TYPE_F32 or MX_TYPE_F16, got %d", name, type);
  if (!dims_in_range({T, k, M})) return fail(MX_ERR_UNSUPPORTED, "%s: T, k or M above 2^31 - 1", name);
  if (K > (int64_t)1 << 24) return fail(MX_ERR_UNSUPPORTED, "%s: K=%lld > 2^24", name, (long long)K);
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
  const int64_t total = p.row_bytes < 16 ? p.T * p.K : p.T * ((p.row_bytes + 15) / 16);
  const int64_t grid = std::min<int64_t>((total + kThreads - 1) / kThreads, (int64_t)num_cus() * 32);
  return by_type(type, [&](auto t) {
    constexpr int kType = decltype(t)::value;
    if (p.row_bytes < 16) unpermute_tiny<kType><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(p);
    else unpermute_kernel<kType><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(p);
    return check_launch("moe_unpermute");
  });
}

int launch_unpermute_backward(const UnpermuteParams& p, int type, hipStream_t stream) {
  const int64_t grid = std::min<int64_t>(p.T * p.k, (int64_t)num_cus() * 32);
  return by_type(type, [&](auto t) {
    constexpr int kType = decltype(t)::value;
    unpermute_backward_kernel<kType><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(p);
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
