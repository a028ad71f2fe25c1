// int8_linear and gmm_int8: products of int8 rows with fp32 scales per token and
// per output channel,
//
//   z[t, n] = (sum_k xq[t, k] wq[n, k]) xs[t] ws[n]
//
// the sum exact in int32 (K < 2^17).
#include <algorithm>
#include <cmath>

#include "int8.h"

namespace mxmoe {

int launch_int8_quantize(const uint16_t* x, int64_t rows, int64_t kd, int64_t ld, int8_t* q, float* s,
                         hipStream_t stream);

int launch_int8_32x16(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_32x16_wide(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_32x32(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_48x48(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_64x64(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_tile128(const Int8Params& p, hipStream_t stream, const char* name);
int launch_int8_tile256(const Int8Params& p, hipStream_t stream, const char* name);
bool int8_resident(int64_t T, int64_t K, int64_t N);
int launch_int8_resident(const Int8Params& p, hipStream_t stream, const char* name);

namespace {

constexpr int64_t kMaxK = ((int64_t)1 << 17) - 16;
constexpr int64_t kMaxN = ((int64_t)1 << 27) - 1;   // 16 rows of outputs stay within the 32-bit byte offsets of a store

// The kernels, by their tiles (weight rows x rows of x), the waves that share a
// tile's K, and the workgroups of a CU.
struct Kernel {
  int64_t bn, bm, waves, per_cu;
  int64_t first, round, stage;         // time in 0.01 us: first + rounds (round + stages of a wave * stage)
  int64_t g_first, g_round, g_stage;   // of gmm_int8, which does without 48 x 48 (g_stage = 0)
  int (*launch)(const Int8Params&, hipStream_t, const char*);
};
const Kernel kKernels[] = {   // in mx_int8_kernel's order
    {32, 16, 4, 2, 223, 102, 51, 487, 77, 68, launch_int8_32x16},
    {32, 16, 8, 1, 251, 82, 60, 520, 51, 77, launch_int8_32x16_wide},
    {32, 32, 4, 2, 214, 129, 61, 483, 91, 77, launch_int8_32x32},
    {48, 48, 3, 2, 205, 230, 76, 0, 0, 0, launch_int8_48x48},
    {64, 64, 2, 2, 152, 332, 92, 415, 211, 96, launch_int8_64x64},
    {128, 128, 1, 2, 32, 570, 95, 333, 405, 89, launch_int8_tile128},
    {256, 256, 1, 1, 236, 915, 147, 495, 341, 133, launch_int8_tile256},
};

// Which kernel: the one whose time a line through its measured times says is
// shortest.  Its tiles go over the CUs in rounds; a round costs a part per tile and
// a part per k stage of a wave.  gmm_int8's rows lie with the experts as the device's
// group list says: the host counts a tile for every expert that gets a row when all
// are as likely, and a tile for every bm rows past half a tile per expert.  Fitted
// to all kernels on 400 shapes each (up to 16384 tokens to 8 of 128 experts, K and N
// to 8192, drawn over their logarithms): the choice takes 0.7 % longer than the fastest
// on average (30 % at worst), gmm_int8's 2 % (45 %: few tiles, or experts' rows that
// fall to one side of a tile's height).  (Also measured: 16 x 16 over 8 waves, 64 x 16,
// 64 x 32, 32 x 64, 64 x 96, 80 x 32 to 80 x 64 and 64 x 64 over 4 waves, which win by
// less than 0.5 % on average together; without 48 x 48 the linear's choice takes 1.2 %
// longer: T = 203, K = 2096, N = 4099 13.1 instead of 11.9 us.)
int choose(int64_t M, int64_t K, int64_t rows, int64_t E, bool grouped) {
  const int64_t cus = num_cus(), nk = (K + kStageK - 1) / kStageK;
  auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const double used = grouped ? (double)E * -std::expm1((double)M * std::log1p(-1.0 / (double)std::max<int64_t>(E, 2))) : 0;
  int best = 0;
  int64_t best_us = 0;
  for (int i = 0; i < (int)(sizeof(kKernels) / sizeof(kKernels[0])); ++i) {
    const Kernel& k = kKernels[i];
    if (grouped && k.g_stage == 0) continue;
    const double more = (double)std::max<int64_t>(0, M - E * k.bm / 2) / (double)k.bm;
    const int64_t m_tiles = !grouped ? up(M, k.bm) : E == 1 ? up(M, k.bm) : (int64_t)std::ceil(used + more);
    const int64_t rounds = up(m_tiles * up(rows, k.bn), cus * k.per_cu), stages = up(nk, k.waves);
    const int64_t us = grouped ? k.g_first + rounds * (k.g_round + stages * k.g_stage)
                               : k.first + rounds * (k.round + stages * k.stage);
    if (i == 0 || us < best_us) {
      best = i;
      best_us = us;
    }
  }
  return best;
}

int launch_int8(Int8Params& p, hipStream_t stream, const char* name) {
  p.e.nk = (int)((p.e.K + kStageK - 1) / kStageK);
  p.present = (int)((p.e.K - (int64_t)(p.e.nk - 1) * kStageK) / 16);
  p.cached = p.gl && !p.swiglu && p.e.N % 32 != 0;
  return kKernels[choose(p.e.T, p.e.K, p.rows, p.E, p.gl != nullptr)].launch(p, stream, name);
}

// Tile indices are 32-bit in every kernel, also a round past the last: of tiles of
// 16 x 16 there are four times as many (an output of half a TB).
bool too_many_tiles(int64_t T, int64_t N) { return ((T + 31) / 32) * ((N + 31) / 32) >= (int64_t)1 << 28; }

int check_sizes(const char* name, int64_t T, int64_t K, int64_t N) {
  if (T < 0 || K <= 0 || N <= 0)
    return fail(MX_ERR_INVALID_ARG, "%s: bad sizes rows=%lld K=%lld N=%lld", name, (long long)T, (long long)K,
                (long long)N);
  if (!dims_in_range({T}) || N > kMaxN)
    return fail(MX_ERR_UNSUPPORTED, "%s: rows above 2^31 - 1 or N above 2^27 - 1", name);
  if (K % 16 != 0) return fail(MX_ERR_UNSUPPORTED, "%s: K=%lld is not a multiple of 16", name, (long long)K);
  if (K > kMaxK) return fail(MX_ERR_UNSUPPORTED, "%s: K=%lld >= 2^17", name, (long long)K);
  if (too_many_tiles(T, N)) return fail(MX_ERR_UNSUPPORTED, "%s: 2^28 or more tiles of 32 x 32 outputs", name);
  return MX_OK;
}

int check_experts(int64_t M, int64_t K, int64_t N, int64_t E) {
  const int rc = check_sizes("gmm_int8", M, K, N);
  if (rc) return rc;
  if (E <= 0) return fail(MX_ERR_INVALID_ARG, "gmm_int8: bad E=%lld", (long long)E);
  if (E > kInt8MaxE) return fail(MX_ERR_UNSUPPORTED, "gmm_int8: E=%lld > %d", (long long)E, kInt8MaxE);
  // (an expert's last tile may be partly empty: E more rows of tiles)
  if (too_many_tiles(M + 32 * E, N))
    return fail(MX_ERR_UNSUPPORTED, "gmm_int8: 2^28 or more tiles of 32 x 32 outputs");
  return MX_OK;
}

// Workspace: the int8 form of bf16 tokens.
struct Int8Layout {
  size_t xs, total;
};
Int8Layout int8_layout(int64_t T, int64_t K, int64_t N, int x_is_int8) {
  if (x_is_int8 || int8_resident(T, K, N)) return {0, 0};
  const size_t xs = align_up((size_t)(T * K), 256);
  return {xs, xs + align_up((size_t)T * 4, 256)};
}

}  // namespace

}  // namespace mxmoe

extern "C" size_t int8_linear_workspace_size(int64_t T, int64_t K, int64_t N, int x_is_int8) {
  // 0 for sizes int8_linear rejects
  if (mxmoe::check_sizes("int8_linear", T, K, N) != MX_OK) return 0;
  return mxmoe::int8_layout(T, K, N, x_is_int8).total;
}

extern "C" int int8_linear_kernel(int64_t T, int64_t K, int64_t N, int x_is_int8) {
  using namespace mxmoe;
  const int rc = check_sizes("int8_linear", T, K, N);
  if (rc) return rc;
  if (T == 0) return fail(MX_ERR_INVALID_ARG, "int8_linear_kernel: no tokens");
  return !x_is_int8 && int8_resident(T, K, N) ? MX_INT8_32X16_BF16 : choose(T, K, N, 0, false);
}

extern "C" int gmm_int8_kernel(int64_t M, int64_t N, int64_t K, int64_t E, int swiglu) {
  using namespace mxmoe;
  const int rc = check_experts(M, K, N, E);
  if (rc) return rc;
  if (M == 0) return fail(MX_ERR_INVALID_ARG, "gmm_int8_kernel: no rows");
  return choose(M, K, swiglu ? 2 * N : N, E, true);
}

extern "C" int int8_linear(const void* x, const float* x_s, const void* w_i8, const float* w_s, const void* bias,
                           int bias_type, int activation, const void* residual_bf16, int64_t T, int64_t K, int64_t N,
                           void* y_bf16, void* workspace, size_t ws_bytes, void* stream) {
  using namespace mxmoe;
  int rc = check_sizes("int8_linear", T, K, N);
  if (rc) return rc;
  if (bias && bias_type != MX_TYPE_BF16 && bias_type != MX_TYPE_F32)
    return fail(MX_ERR_INVALID_ARG, "int8_linear: bias_type must be MX_TYPE_BF16 or MX_TYPE_F32, got %d", bias_type);
  if (activation < MX_ACT_NONE || activation > MX_ACT_GELU_TANH)
    return fail(MX_ERR_INVALID_ARG, "int8_linear: unknown activation %d", activation);
  const bool int8_in = x_s != nullptr;
  const Int8Layout L = int8_layout(T, K, N, int8_in);
  if (T > 0 && (!x || !w_i8 || !w_s || !y_bf16 || (L.total > 0 && !workspace)))
    return fail(MX_ERR_INVALID_ARG, "int8_linear: null pointer");
  if (ws_bytes < L.total)
    return fail(MX_ERR_WORKSPACE, "int8_linear: workspace %zu bytes < %zu", ws_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(x) % (int8_in ? 16 : 2) || reinterpret_cast<uintptr_t>(w_i8) % 16 ||
      reinterpret_cast<uintptr_t>(x_s) % 4 || reinterpret_cast<uintptr_t>(w_s) % 4 ||
      reinterpret_cast<uintptr_t>(bias) % (bias_type == MX_TYPE_F32 ? 4 : 2) ||
      reinterpret_cast<uintptr_t>(residual_bf16) % 2 || reinterpret_cast<uintptr_t>(y_bf16) % 2 ||
      (L.total > 0 && reinterpret_cast<uintptr_t>(workspace) % 256))
    return fail(MX_ERR_UNSUPPORTED, "int8_linear: misaligned pointer");
  if (T == 0) return MX_OK;
  // Outputs overlap nothing, except that y may take the residual's place.
  const uint64_t dense = (uint64_t)T * (uint64_t)N * 2;
  const Span in[7] = {{x, (uint64_t)T * (uint64_t)K * (int8_in ? 1 : 2)},
                      {x_s, (uint64_t)T * 4},
                      {w_i8, (uint64_t)N * (uint64_t)K},
                      {w_s, (uint64_t)N * 4},
                      {bias, (uint64_t)N * (bias_type == MX_TYPE_F32 ? 4 : 2)},
                      {workspace, L.total},
                      {residual_bf16, dense}};
  for (int i = 0; i < 7; ++i) {
    if (overlaps({y_bf16, dense}, in[i]) && !(i == 6 && y_bf16 == residual_bf16))
      return fail(MX_ERR_INVALID_ARG, "int8_linear: the output overlaps an input or the workspace");
    if (i != 5 && overlaps(in[5], in[i]))
      return fail(MX_ERR_INVALID_ARG, "int8_linear: the workspace overlaps an input");
  }
  Int8Params p{};
  p.e.T = T;
  p.e.K = K;
  p.e.N = N;
  p.e.bias = bias;
  p.e.bias_f32 = bias_type == MX_TYPE_F32;
  p.e.act = activation;
  p.e.res = static_cast<const uint16_t*>(residual_bf16);
  p.e.y = static_cast<uint16_t*>(y_bf16);
  p.e.stream_res = T * N > (int64_t)48 << 20;
  p.w = static_cast<const int8_t*>(w_i8);
  p.ws = w_s;
  p.rows = N;
  hipStream_t s = as_stream(stream);
  if (int8_in) {
    p.x = static_cast<const int8_t*>(x);
    p.xs = x_s;
  } else if (int8_resident(T, K, N)) {
    p.x = static_cast<const int8_t*>(x);
    p.e.nk = (int)((K + kStageK - 1) / kStageK);
    p.present = (int)((K - (int64_t)(p.e.nk - 1) * kStageK) / 16);
    return launch_int8_resident(p, s, "int8_linear");
  } else {
    int8_t* xq = static_cast<int8_t*>(workspace);
    float* xs = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.xs);
    rc = launch_int8_quantize(static_cast<const uint16_t*>(x), T, K, K, xq, xs, s);
    if (rc) return rc;
    p.x = xq;
    p.xs = xs;
  }
  return launch_int8(p, s, "int8_linear");
}

extern "C" int gmm_int8(const void* a_i8, const float* a_s, const void* w_i8, const float* w_s,
                        const int64_t* group_list, int group_list_type, int swiglu, int64_t M, int64_t N, int64_t K,
                        int64_t E, void* y_bf16, void* stream) {
  using namespace mxmoe;
  int rc = check_experts(M, K, N, E);
  if (rc) return rc;
  if (group_list_type != 0 && group_list_type != 1)
    return fail(MX_ERR_INVALID_ARG, "gmm_int8: group_list_type must be 0 (cumulative) or 1 (count), got %d",
                group_list_type);
  if (!group_list || (M > 0 && (!a_i8 || !a_s || !w_i8 || !w_s || !y_bf16)))
    return fail(MX_ERR_INVALID_ARG, "gmm_int8: null pointer");
  if (reinterpret_cast<uintptr_t>(a_i8) % 16 || reinterpret_cast<uintptr_t>(w_i8) % 16 ||
      reinterpret_cast<uintptr_t>(a_s) % 4 || reinterpret_cast<uintptr_t>(w_s) % 4 ||
      reinterpret_cast<uintptr_t>(group_list) % 8 || reinterpret_cast<uintptr_t>(y_bf16) % 2)
    return fail(MX_ERR_UNSUPPORTED, "gmm_int8: misaligned pointer");
  if (M == 0) return MX_OK;
  const int64_t rows = swiglu ? 2 * N : N;
  const Span in[5] = {{a_i8, (uint64_t)M * (uint64_t)K}, {a_s, (uint64_t)M * 4},
                      {w_i8, (uint64_t)E * (uint64_t)rows * (uint64_t)K}, {w_s, (uint64_t)E * (uint64_t)rows * 4},
                      {group_list, (uint64_t)E * 8}};
  for (const Span& i : in)
    if (overlaps({y_bf16, (uint64_t)M * (uint64_t)N * 2}, i))
      return fail(MX_ERR_INVALID_ARG, "gmm_int8: the output overlaps an input");
  Int8Params p{};
  p.e.T = M;
  p.e.K = K;
  p.e.N = N;
  p.e.y = static_cast<uint16_t*>(y_bf16);
  p.x = static_cast<const int8_t*>(a_i8);
  p.xs = a_s;
  p.w = static_cast<const int8_t*>(w_i8);
  p.ws = w_s;
  p.gl = group_list;
  p.gl_type = group_list_type;
  p.E = (int)E;
  p.rows = rows;
  p.swiglu = swiglu != 0;
  return launch_int8(p, as_stream(stream), "gmm_int8");
}
