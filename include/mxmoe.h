/*
 * mxmoe.h -- C ABI of the MXFP8 block-scaled top-k MoE expert layer for
 * AMD MI355X (gfx950).
 *
 * The layer (sources: "Quantization on Ascend", sglang docs, section on MXFP8
 * for LLM MoE models; "[WIP] Fix offline W8A8 MXFP8 quantization for Qwen3.5
 * on Ascend NPU", sglang PR 32266, commit adding the fused-experts chain):
 *
 *   moe_route_quant     top-k routing with the MX activation quant fused in
 *   gmm_swiglu_mxquant  grouped GEMM1 (gate + up) + SwiGLU + MX requant
 *   gmm_mx              grouped GEMM2 (down), bf16 output
 *   moe_finalize        weighted un-permute and sum of the top-k outputs
 *   moe_mxfp8_forward   the four steps above on one stream
 *   mx_quantize         stand-alone MX quantiser (weights at load time)
 *   moe_route_quant_noalloc
 *                       moe_route_quant without a workspace (allocates nothing)
 *   moe_router          top-k softmax router over a bf16 gate (upstream of
 *                       the layer: produces the ids and weights it takes)
 *   mx_linear           dense MXFP8 linear layer (activation quant + MX GEMM)
 *   mx_linear_fused     dense MXFP8 linear layer with bias, activation and
 *                       residual in its epilogue, bf16 or MXFP8 in and out
 *   mx_add_rmsnorm      residual addition + RMSNorm with MXFP8 and bf16 outputs
 *   moe_route_mx, moe_mxfp8_forward_mx
 *                       routing and the layer for token rows that are already
 *                       MXFP8 (as mx_add_rmsnorm writes them)
 *   int8_quantize, int8_linear, gmm_int8
 *                       the products in int8 with a scale per token and output
 *                       channel: quantiser, dense linear, by expert
 *   moe_permute, moe_unpermute, moe_unpermute_backward
 *                       token rows of any type sorted by expert and back with
 *                       the routing weights, and the gradients
 *   mx_pack_weights, gmm_swiglu_mxquant_packed, gmm_mx_packed,
 *   moe_mxfp8_forward_packed
 *                       load-time weight cast into the GEMMs' tile layout,
 *                       and the GEMMs and the layer reading it
 *   mx_quantize_fp4     MXFP4 (e2m1) quantiser for the W4A8 path's weights
 *   gmm_swiglu_mxquant_w4a8, gmm_mx_w4a8, moe_w4a8_forward
 *                       the GEMMs and the layer with MXFP4 expert weights
 *
 * Formats.  MXFP8 = e4m3 payload bytes plus one e8m0 scale byte (exponent +
 * 127, value 2^(byte-127)) per 32 consecutive elements along the reduction
 * dimension.  A row of Kd elements has ceil(Kd/32) scales, padded with one
 * zero byte when that count is odd, stored as [ceil(Kd/64), 2] pairs: the
 * pair-split layout ("Quantization on Ascend", offline MoE path: [E,N,K/32]
 * scales viewed as [E,N,K/64,2]; PR 32266 Summary, offline partial block-scale
 * layout, worked example K = 4304 -> 135 -> 136 -> 68 pairs).  There is no zero
 * point.  Quantisation: s = floor(log2(amax)) - 8 clamped to [-127, 127]
 * (scale byte s + 127; an all-zero block gets byte 0), payload = e4m3 of
 * x * 2^-s rounded to nearest, ties to even, saturating at +-448, sign kept
 * (so -0 and negative values that round to zero give 0x80).
 *
 * Finite inputs only.  Every bf16/fp32 input (x, bf16 weights, topk_w) must
 * be finite: the pages fix no NaN or infinity convention for MX blocks and
 * the library does not check (a device-side scan would cost a full read).
 * What non-finite inputs produce is not part of the contract; with the
 * current kernels a NaN drops out of its block's amax and encodes as -448
 * times the block scale (code 0xFE), and an infinity sets its block's scale
 * byte to 247 and flushes the block's other elements to zero.  No error is
 * reported for either.
 *
 * Tensors.  Every pointer is a DEVICE pointer unless stated; all tensors are
 * dense row-major.  bf16 is passed as its 16-bit pattern.  Sizes are int64_t.
 *   x            bf16   [T, K]
 *   topk_ids     int32  [T, k]   expert ids in [0, E)
 *   topk_w       fp32   [T, k]   routing weights
 *   w13          uint8  [E, 2I, K]   e4m3; rows [0, I) gate, rows [I, 2I) up
 *   w13_s        uint8  [E, 2I, K/64, 2]
 *   w2           uint8  [E, K, I]    e4m3
 *   w2_s         uint8  [E, K, I/64, 2]
 *   group_list   int64  [E]  type 1: rows per expert (counts);
 *                            type 0: inclusive cumulative counts
 *   M = T*k expanded rows; expert e owns a contiguous run of rows in expert
 *   order, and inside one expert rows keep the order of the flat assignment
 *   index t*k + j (a stable sort).
 *
 * Ownership and execution.  The caller allocates every buffer, including
 * the workspaces (sized by the *_workspace_size queries).  The library never
 * allocates, frees or retains pointers and never synchronises the host.
 * Every call enqueues work on `stream` (a hipStream_t passed as void*; NULL =
 * the null stream) and returns at once; results are ready when the stream
 * reaches them.  Calls on different streams must not share output or
 * workspace buffers.
 *
 * Errors.  Every entry point returns MX_OK (0) or a negative mx_status.
 * Argument checks happen on the host before anything is enqueued; on error
 * nothing is enqueued and mx_last_error() (thread-local) describes why.
 * Data-dependent conditions are handled on the device without faulting:
 * an expert id outside [0, E) is dropped (its expanded_row_idx entry is -1,
 * it counts toward no expert, so sum(group_list) < T*k tells the caller), and
 * group lists are clamped to [0, M] rows.
 *
 * GPU shape limits (MX_ERR_UNSUPPORTED otherwise): every size argument at
 * most 2^31 - 1, and M = T*k at most 2^27 for routing and the layer (below
 * 2^31 for the GEMMs and finalize); GEMM reduction dims (K of GEMM1,
 * I of GEMM2) multiples of 128 and at most 2^20; GEMM2 output dim N a
 * multiple of 256;
 * GEMM1 intermediate size I a multiple of 128 (so the forward needs K % 256
 * == 0 and I % 128 == 0); routing needs K % 32 == 0, K <= 2^24,
 * 1 <= k <= 256 and E <= 1024; mx_quantize takes any Kd >= 1.
 *
 * Alignment (MX_ERR_UNSUPPORTED otherwise): e4m3 payload and bf16 tensors
 * that the GEMMs, routing and finalize read or write (x, xq, a, w, w13, w2,
 * hq, y, out, the forward workspace) start on 16-byte boundaries, their scale
 * tensors (a_s, w_s, w13_s, w2_s, hs) on 4-byte boundaries, h_f32_debug on 16.
 * mx_quantize accepts any alignment (a slower path handles the rest).
 */
#ifndef MXMOE_H
#define MXMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mx_status {
  MX_OK = 0,
  MX_ERR_INVALID_ARG = -1, /* null pointer, non-positive size, k > E, bad group_list_type */
  MX_ERR_UNSUPPORTED = -2, /* a shape the GPU kernels do not handle (see above) */
  MX_ERR_WORKSPACE = -3,   /* workspace smaller than the size query returned */
  MX_ERR_HIP = -4          /* a HIP runtime error at launch */
} mx_status;

/*
 * MX-quantise `rows` rows of `kd` bf16 elements (row stride `ld` elements,
 * ld >= kd) into e4m3 payload q [rows, kd] (row stride kd bytes) and scales
 * s [rows, ceil(kd/64), 2] (odd scale counts padded with a zero byte).
 * Used on expert weights at load time ("Quantization on Ascend", MoE online
 * path: bf16 [E, N, K] expert weights quantised once, 3-D input taken as
 * E*N rows) and for activations that bypass routing.
 */
int mx_quantize(const void* x_bf16, int64_t rows, int64_t kd, int64_t ld,
                void* q_u8, void* s_u8, void* stream);

/*
 * MXFP4-quantise `rows` rows of `kd` bf16 elements (row stride `ld`) into
 * packed e2m1 codes q [rows, kd/2] (element 2i in the low nibble of byte i)
 * and e8m0 scales s [rows, ceil(kd/64), 2]: the weights of the W4A8 path
 * ("Quantization on Ascend", W4A8 implementation notes: weights packed FP4,
 * float4_e2m1fn_x2, two nibbles per byte, one UE8M0 scale per 32 elements;
 * activations stay MXFP8).  Per 32-block: s = floor(log2(amax)) - 2 clamped
 * to [-127, 127] (byte s + 127, an all-zero block gets 0), codes = nearest of
 * +-{0, .5, 1, 1.5, 2, 3, 4, 6} to x * 2^-s, ties to the even code,
 * saturating at 6, sign kept.  kd % 32 == 0 (MX_ERR_UNSUPPORTED otherwise).
 */
int mx_quantize_fp4(const void* x_bf16, int64_t rows, int64_t kd, int64_t ld,
                    void* q_u8, void* s_u8, void* stream);

/* Workspace bytes moe_route_quant needs for T tokens, top-k, E experts
 * (0 when T*k <= 256: the call then accepts a null workspace). */
size_t moe_route_quant_workspace_size(int64_t T, int64_t k, int64_t E);

/*
 * Top-k routing with fused MX activation quant ("Quantization on Ascend",
 * MoE forward: routing quantises the activations in the same op; PR 32266,
 * commit on the fused routing quant: byte-identical to routing then
 * quantising).  Outputs, for M = T*k:
 *   xq                uint8 [M, K]        row p = MX payload of token sorted_row[p] / k
 *   xs                uint8 [M, K/64, 2]  its scales (pair-split)
 *   sorted_row        int32 [M]           flat assignment index t*k+j of row p
 *   expanded_row_idx  int32 [M]           row p of flat assignment i (-1 if its id was invalid)
 *   group_list        int64 [E]           rows per expert (count form, type 1)
 * Rows past sum(group_list) (only when ids were invalid) are left unwritten.
 * One kernel launch.  Its workgroups exchange per-chunk expert counts through
 * the workspace under flags tagged per call, so the workspace needs no
 * clearing; a workgroup that finds the counts not yet published after a
 * bounded number of polls (moe_route_quant_set_wait_limit) counts them from
 * topk_ids itself, so the call always ends and its output never depends on
 * the order the GPU runs the workgroups in.  Called while `stream` is
 * capturing, the call also records a one-thread kernel ahead of the routing
 * kernel that advances a generation word in the workspace, so that every
 * replay of the captured graph tags its flags afresh.
 */
int moe_route_quant(const void* x_bf16, const int32_t* topk_ids,
                    int64_t T, int64_t K, int64_t k, int64_t E,
                    void* xq_u8, void* xs_u8, int32_t* sorted_row,
                    int32_t* expanded_row_idx, int64_t* group_list,
                    void* workspace, size_t ws_bytes, void* stream);

/*
 * moe_route_quant for callers that cannot allocate: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, outputs and results as moe_route_quant minus the workspace:
 * the routing scratch (per-chunk expert counts, the experts' offsets and
 * the flags that publish them) is a 4 MiB device array inside the library, one per GPU, held until the
 * process ends.  The call allocates nothing (no hipMalloc, hipFree or
 * allocating library routine); the caller still passes every input and
 * output.  Sizes whose scratch, moe_route_quant_workspace_size(T, k, E),
 * exceeds 4 MiB (4,194,304 bytes) are rejected with MX_ERR_UNSUPPORTED
 * before anything is enqueued (e.g. E = 128, k = 8: up to 261,056 tokens).
 * Every call on one GPU shares that GPU's array: calls that overlap in time
 * on one GPU (other streams, other host threads) race and must not be
 * issued; calls ordered on one stream are safe.  The array needs no
 * clearing: each call writes every count it reads before reading it, and
 * its flags match only the tag of the call that set them.
 */
int moe_route_quant_noalloc(const void* x_bf16, const int32_t* topk_ids,
                            int64_t T, int64_t K, int64_t k, int64_t E,
                            void* xq_u8, void* xs_u8, int32_t* sorted_row,
                            int32_t* expanded_row_idx, int64_t* group_list,
                            void* stream);

/*
 * How many times a routing workgroup polls for the published expert counts
 * before counting them from topk_ids itself (process-wide, default 2^18;
 * 0 makes every workgroup count for itself: much slower, same output).
 * Applies to launches enqueued after the call; returns the previous value.
 * Negative values are taken as 0.  Meant for tests of that path.
 */
int64_t moe_route_quant_set_wait_limit(int64_t polls);

/*
 * Grouped GEMM1 with SwiGLU and MX requant fused ("Quantization on Ascend",
 * MoE forward: GEMM1 fuses gate/up, SwiGLU and requant and hands back
 * quantised activations plus block scales; "PR #30768 report", key source
 * excerpt: it takes a cumulative group list, the dispatcher produces counts).
 * For expert e and its rows m:
 *   acc = A[m] . W13_e^T (fp32 accumulation), g = acc[:, :I], u = acc[:, I:],
 *   h = silu(g) * u (fp32), (hq, hs) = MX quantisation of h along I.
 *   a      uint8 [M, K], a_s [M, K/64, 2]
 *   hq     uint8 [M, I], hs  [M, I/64, 2]
 *   h_f32_debug  fp32 [M, I] or NULL: when given, also receives h.
 * group_list_type: 0 = cumulative, 1 = count.  Rows not owned by any expert
 * are not written.
 */
int gmm_swiglu_mxquant(const void* a_u8, const void* a_s,
                       const void* w13_u8, const void* w13_s,
                       const int64_t* group_list, int group_list_type,
                       int64_t M, int64_t K, int64_t I, int64_t E,
                       void* hq_u8, void* hs_u8, float* h_f32_debug,
                       void* stream);

/*
 * Grouped MX GEMM with bf16 output (GEMM2, down projection; "Quantization on
 * Ascend", MoE forward: the second grouped GEMM takes the count group list).
 *   y[m, :] = bf16_rne( A[m] . W_e^T )  for the expert e owning row m
 *   a  uint8 [M, Kd], a_s [M, Kd/64, 2];  w uint8 [E, N, Kd], w_s [E, N, Kd/64, 2]
 *   y  bf16 [M, N]
 */
int gmm_mx(const void* a_u8, const void* a_s, const void* w_u8, const void* w_s,
           const int64_t* group_list, int group_list_type,
           int64_t M, int64_t N, int64_t Kd, int64_t E,
           void* y_bf16, void* stream);

/*
 * Tile-packed expert weights: the weights' load-time cast into the layout
 * the GEMMs' LDS ring holds, the counterpart of the pages' cast of expert
 * weights into the matrix unit's tiled format once at load ("PR #30768
 * report", review highlights: the NZ format; PR 32266, the commit casting
 * weights to NZ).  mx_pack_weights rewrites e4m3 weights w [E, N, Kd] into
 * out (same size, E*N*Kd bytes, must not overlap w): for expert e, n-tile
 * nt = 0 .. N/256 - 1 and k stage ks = 0 .. Kd/128 - 1, the 32 KB block at
 * byte ((e*(N/256) + nt)*(Kd/128) + ks)*32768 holds 256 rows of 128 bytes,
 * 16-byte chunk c of block row r at chunk position c ^ ((r/2) % 8).  Block
 * row r is weight row 256*nt + r for kind 0 (GEMM2 weights w2 [E, K, I]);
 * for kind 1 (GEMM1 weights w13 [E, 2I, K], I = N/2) block rows
 * [128h, 128h+64) are gate rows 128*nt + 64h + (0..63) and block rows
 * [128h+64, 128h+128) up rows I + 128*nt + 64h + (0..63), h = 0, 1.
 * Scales are not packed: the *_packed calls take them in the usual
 * [E, N, Kd/64, 2] layout.  Needs N % 256 == 0, Kd % 128 == 0, E <= 1024.
 *
 * gmm_swiglu_mxquant_packed, gmm_mx_packed and moe_mxfp8_forward_packed
 * are gmm_swiglu_mxquant, gmm_mx and moe_mxfp8_forward with w13 packed as
 * kind 1 and w2 (w) packed as kind 0; arguments, results and limits are
 * otherwise the same (the results are identical byte for byte).
 */
int mx_pack_weights(const void* w_u8, int64_t E, int64_t N, int64_t Kd, int kind,
                    void* out_u8, void* stream);

int gmm_swiglu_mxquant_packed(const void* a_u8, const void* a_s,
                              const void* w13_packed, const void* w13_s,
                              const int64_t* group_list, int group_list_type,
                              int64_t M, int64_t K, int64_t I, int64_t E,
                              void* hq_u8, void* hs_u8, float* h_f32_debug,
                              void* stream);

int gmm_mx_packed(const void* a_u8, const void* a_s, const void* w_packed,
                  const void* w_s, const int64_t* group_list, int group_list_type,
                  int64_t M, int64_t N, int64_t Kd, int64_t E, void* y_bf16,
                  void* stream);

/*
 * Finalize: weighted un-permute and sum (PR 32266, fused-experts commit:
 * the chain ends with finalize routing).
 *   out[t, :] = bf16_rne( sum_{j=0}^{k-1} w[t, j] * y[expanded_row_idx[t*k+j], :] )
 * accumulated in fp32 in ascending j, each product and sum rounded to fp32.
 * Entries whose index is outside [0, M) are skipped.
 *   y bf16 [M, K], topk_w fp32 [T, k], expanded_row_idx int32 [T*k], out bf16 [T, K]
 */
int moe_finalize(const void* y_bf16, const float* topk_w,
                 const int32_t* expanded_row_idx, int64_t T, int64_t K,
                 int64_t k, int64_t M, void* out_bf16, void* stream);

/*
 * W4A8 variants ("Quantization on Ascend", W4A8 implementation notes: expert
 * weights packed FP4 with a UE8M0 scale per 32 elements, activations per-token
 * MXFP8).  Same arguments, semantics, limits and errors as gmm_swiglu_mxquant
 * and gmm_mx, except that the weight payload is packed e2m1 (mx_quantize_fp4):
 *   w13 uint8 [E, 2I, K/2] (gate rows [0, I), up rows [I, 2I)),
 *   w   uint8 [E, N, Kd/2]; element 2c in the low nibble of byte c.
 * Scales keep the [.., K/64, 2] layout.  GEMM1's output hq/hs stays MXFP8.
 */
int gmm_swiglu_mxquant_w4a8(const void* a_u8, const void* a_s,
                            const void* w13_u8, const void* w13_s,
                            const int64_t* group_list, int group_list_type,
                            int64_t M, int64_t K, int64_t I, int64_t E,
                            void* hq_u8, void* hs_u8, float* h_f32_debug,
                            void* stream);
int gmm_mx_w4a8(const void* a_u8, const void* a_s, const void* w_u8, const void* w_s,
                const int64_t* group_list, int group_list_type,
                int64_t M, int64_t N, int64_t Kd, int64_t E,
                void* y_bf16, void* stream);

/* Workspace bytes moe_mxfp8_forward needs (holds every intermediate). */
size_t moe_mxfp8_forward_workspace_size(int64_t T, int64_t K, int64_t I,
                                        int64_t E, int64_t k);

/*
 * The whole layer on one stream: moe_route_quant -> gmm_swiglu_mxquant ->
 * gmm_mx -> moe_finalize (PR 32266, fused-experts commit; "Quantization on
 * Ascend", MoE forward).  Weights are pre-quantised (see mx_quantize).
 * out bf16 [T, K].  Intermediates live in the workspace.
 */
int moe_mxfp8_forward(const void* x_bf16, const int32_t* topk_ids,
                      const float* topk_w, const void* w13_u8,
                      const void* w13_s, const void* w2_u8, const void* w2_s,
                      int64_t T, int64_t K, int64_t I, int64_t E, int64_t k,
                      void* out_bf16, void* workspace, size_t ws_bytes,
                      void* stream);

/* moe_mxfp8_forward with tile-packed weights (see mx_pack_weights). */
int moe_mxfp8_forward_packed(const void* x_bf16, const int32_t* topk_ids,
                             const float* topk_w, const void* w13_packed,
                             const void* w13_s, const void* w2_packed,
                             const void* w2_s, int64_t T, int64_t K, int64_t I,
                             int64_t E, int64_t k, void* out_bf16, void* workspace,
                             size_t ws_bytes, void* stream);

/*
 * The whole layer with MXFP4 expert weights (the W4A8 path): as
 * moe_mxfp8_forward with w13 uint8 [E, 2I, K/2] and w2 uint8 [E, K, I/2]
 * packed e2m1 (see gmm_swiglu_mxquant_w4a8); same workspace and layout.
 */
int moe_w4a8_forward(const void* x_bf16, const int32_t* topk_ids,
                     const float* topk_w, const void* w13_u8,
                     const void* w13_s, const void* w2_u8, const void* w2_s,
                     int64_t T, int64_t K, int64_t I, int64_t E, int64_t k,
                     void* out_bf16, void* workspace, size_t ws_bytes,
                     void* stream);

/* Byte offsets of the intermediates inside the forward workspace, so a caller
 * can inspect them after the stream has run.  Fills the 8 offsets in order:
 * xq, xs, sorted_row, expanded_row_idx, group_list, hq, hs, y. */
int moe_mxfp8_forward_workspace_layout(int64_t T, int64_t K, int64_t I,
                                       int64_t E, int64_t k,
                                       size_t* offsets_host);

/*
 * Top-k softmax router over a bf16 gate linear, the step upstream of
 * moe_route_quant ("Quantization on Ascend", MXFP8 for LLM MoE models,
 * implementation notes: the router gate is a plain linear layer, kept in bf16
 * on the online path).  For each token t:
 *   logits[e] = sum_c x[t,c] * gate[e,c] (+ bias[e])   fp32 accumulation of
 *               the exact bf16 products
 *   topk_ids[t, :] = the k largest logits, descending (equal logits: the
 *                    lower expert id first)
 *   topk_w[t, j]   = softmax(logits)[topk_ids[t, j]], divided by the sum of
 *                    the k selected when renormalize != 0
 *   x bf16 [T, K], gate bf16 [E, K], bias fp32 [E] or NULL (-inf allowed:
 *   that expert is never picked while a finite one is left);
 *   topk_ids int32 [T, k], topk_w fp32 [T, k] (the inputs of moe_route_quant,
 *   moe_finalize and moe_mxfp8_forward).
 * Limits: K % 64 == 0, E <= 256 (MX_ERR_UNSUPPORTED); 1 <= k <= E
 * (MX_ERR_INVALID_ARG); x and gate 16-byte aligned.
 */
int moe_router(const void* x_bf16, const void* gate_bf16, const float* bias,
               int64_t T, int64_t K, int64_t E, int64_t k, int renormalize,
               int32_t* topk_ids, float* topk_w, void* stream);

/* Workspace bytes mx_linear needs for T tokens of K features. */
size_t mx_linear_workspace_size(int64_t T, int64_t K);

/*
 * Dense MXFP8 linear layer ("Quantization on Ascend", MXFP8 (dense)
 * implementation notes: weights MX-quantised once at load (see mx_quantize),
 * activations MX-quantised per token at inference, block 32 along K, then the
 * quantised matmul):
 *   (xq, xs) = MX quantisation of x along K (as mx_quantize)
 *   y[t, n]  = bf16_rne( sum over 32-blocks b of 2^(sx[t,b] + sw[n,b]) * (xq[t,b] . wq[n,b]) )
 *   x bf16 [T, K]; w uint8 [N, K] e4m3; w_s uint8 [N, K/64, 2]; y bf16 [T, N].
 * The workspace (mx_linear_workspace_size, 256-byte aligned) holds xq and
 * xs.  Limits as gmm_mx with one group: K % 128 == 0,
 * N % 256 == 0.
 */
int mx_linear(const void* x_bf16, const void* w_u8, const void* w_s,
              int64_t T, int64_t K, int64_t N, void* y_bf16,
              void* workspace, size_t ws_bytes, void* stream);

/* Element types: of a norm's weight and of a linear's bias (bf16, fp32), and of
 * moe_unpermute's rows (all three). */
typedef enum mx_type { MX_TYPE_BF16 = 0, MX_TYPE_F32 = 1, MX_TYPE_F16 = 2 } mx_type;

/*
 * Residual addition, root-mean-square norm and MX quantisation in one pass,
 * the step in front of the router, the layer and the dense linears.  For each
 * of `rows` rows of `kd` elements:
 *   h = x + residual                (h = x without a residual)
 *   n = h / sqrt(mean(h^2) + eps) * weight
 *   residual_out = bf16_rne(h),  y = bf16_rne(n),
 *   (q, s) = MX quantisation of n along kd, as mx_quantize's of a row
 * in fp32 throughout, each output rounded once: the norm reads h before it is
 * rounded to bf16, and q rounds n itself and not y.  Before that rounding n is
 * within 48 * 2^-24 of the n of its h, for any kd.
 *   x         bf16 [rows, kd], row stride ldx >= kd elements
 *   residual  bf16 [rows, kd], row stride ldr >= kd, or NULL (ldr unused)
 *   weight    [kd], bf16 or fp32 (weight_type); a norm that multiplies by
 *             (1 + w) takes 1 + w in fp32
 *   residual_out  bf16 [rows, kd] or NULL (only with a residual)
 *   y         bf16 [rows, kd] or NULL
 *   q, s      uint8 [rows, kd], [rows, ceil(kd/64), 2], or both NULL; at least
 *             one of y and q is given
 * residual_out or y may be x or the residual itself (the same address, dense
 * rows); any other overlap of an output is MX_ERR_INVALID_ARG.  eps is a
 * positive normal float.  Any kd from 1 to 2^24 and any alignment of whole
 * elements (rows of a multiple of 8 elements on 16-byte boundaries, q on 8,
 * take the fast path).  h has to be finite in fp32; a row's squares need not.
 */
int mx_add_rmsnorm(const void* x_bf16, int64_t ldx, const void* residual_bf16,
                   int64_t ldr, const void* weight, int weight_type, float eps,
                   int64_t rows, int64_t kd, void* residual_out_bf16,
                   void* y_bf16, void* q_u8, void* s_u8, void* stream);

/*
 * moe_route_quant for token rows that are MXFP8 already: q uint8 [T, K] and
 * s uint8 [T, K/64, 2] are sent to their experts' rows as they are (xq, xs);
 * the maps, the group list, the workspace (moe_route_quant_workspace_size,
 * on an 8-byte boundary), the limits and the bounded waits are those of
 * moe_route_quant.  q needs 16-byte alignment; s any.  An output that overlaps
 * an input, another output or the workspace is MX_ERR_INVALID_ARG.
 */
int moe_route_mx(const void* q_u8, const void* s_u8, const int32_t* topk_ids,
                 int64_t T, int64_t K, int64_t k, int64_t E, void* xq_u8,
                 void* xs_u8, int32_t* sorted_row, int32_t* expanded_row_idx,
                 int64_t* group_list, void* workspace, size_t ws_bytes,
                 void* stream);

/* Formats of the expert weights of moe_mxfp8_forward_mx: e4m3 rows, packed
 * e2m1 (mx_quantize_fp4), e4m3 tile-packed by mx_pack_weights. */
typedef enum mx_weights { MX_WEIGHTS_E4M3 = 0, MX_WEIGHTS_E2M1 = 1, MX_WEIGHTS_PACKED = 2 } mx_weights;

/*
 * The whole layer on token rows that are MXFP8 already (moe_route_mx in the
 * place of moe_route_quant), with expert weights in any of the layer's
 * formats: moe_mxfp8_forward, moe_w4a8_forward or moe_mxfp8_forward_packed
 * with x's quantisation left out.  Same workspace, layout and limits.
 */
int moe_mxfp8_forward_mx(const void* q_u8, const void* s_u8,
                         const int32_t* topk_ids, const float* topk_w,
                         int weight_format, const void* w13_u8,
                         const void* w13_s, const void* w2_u8, const void* w2_s,
                         int64_t T, int64_t K, int64_t I, int64_t E, int64_t k,
                         void* out_bf16, void* workspace, size_t ws_bytes,
                         void* stream);

/* Activations of mx_linear_fused: none; max(z, 0); z / (1 + e^-z);
 * z Phi(z); (z / 2)(1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))). */
typedef enum mx_activation {
  MX_ACT_NONE = 0, MX_ACT_RELU = 1, MX_ACT_SILU = 2, MX_ACT_GELU = 3, MX_ACT_GELU_TANH = 4
} mx_activation;

/* Workspace bytes mx_linear_fused needs (x_is_mx: x comes as MXFP8). */
size_t mx_linear_fused_workspace_size(int64_t T, int64_t K, int64_t N, int x_is_mx);

/*
 * mx_linear with its epilogue fused and without its limits on the sizes:
 *   z[t, n]   = sum over 32-blocks b of 2^(sx[t,b] + sw[n,b]) * (xq[t,b] . wq[n,b])
 *   out[t, n] = activation(z[t, n] + bias[n]) + residual[t, n]
 * bias, activation and residual in fp32, rounded once: to bf16 (y), or along n
 * to MXFP8 (yq, ys: the x of the next linear, or the rows of moe_route_mx).
 * z is summed as the scaled matrix instruction sums.  Of each 8 consecutive k
 * (from a multiple of 8 on) it truncates the products to multiples of
 * 2^(e - 13), e the largest of their sums of operand exponents (a payload below
 * 2^-6 counts as 2^-6 in its block's scale), so 8 products are off by less than
 * 2^-10 of the largest |x| |w| among them; these sums then add in fp32.  That is
 * far below what rounding the operands to e4m3 changed, but it is not fp32's
 * 2^-24: an MXFP8 output is now and then the neighbouring code of an exact
 * sum's (0.4 % RMS of the outputs), a bf16 one within its own rounding.
 * gmm_swiglu_mxquant and gmm_mx add up with the same instruction.
 *   x         uint8 [T, K] e4m3 with x_s uint8 [T, ceil(K/64), 2], or with a
 *             NULL x_s bf16 [T, K], quantised first (the bytes are those of
 *             mx_quantize; up to 32 tokens of up to 65536 elements together
 *             need no workspace for it while N <= 8192)
 *   w, w_s    uint8 [N, K], [N, ceil(K/64), 2]
 *   bias      [N] bf16 or fp32 (bias_type), or NULL
 *   residual  bf16 [T, N] or NULL
 *   y         bf16 [T, N], or yq uint8 [T, N] and ys uint8 [T, ceil(N/64), 2]
 *             (an odd count of scales padded with a zero byte)
 * y may be the residual itself (the same address); any other overlap of an
 * output or of the workspace is MX_ERR_INVALID_ARG.  Limits: K % 32 == 0,
 * K <= 2^20, fewer than 2^30 tiles of 32 x 32 outputs.  Alignment: MXFP8
 * payloads that are read on 16-byte boundaries, their scales on 4, the workspace
 * on 256.
 */
int mx_linear_fused(const void* x, const void* x_s, const void* w_u8,
                    const void* w_s, const void* bias, int bias_type,
                    int activation, const void* residual_bf16, int64_t T,
                    int64_t K, int64_t N, void* y_bf16, void* yq_u8,
                    void* ys_u8, void* workspace, size_t ws_bytes,
                    void* stream);

/* The kernels of mx_linear_fused, by their tiles (weight rows x tokens). */
typedef enum mx_linear_kernel {
  MX_LINEAR_32X32 = 0,
  MX_LINEAR_64X64 = 1,
  MX_LINEAR_64X96 = 2,
  MX_LINEAR_64X64_TWICE = 3, /* 64 x 64, two workgroups per CU */
  MX_LINEAR_128X128 = 4,
  MX_LINEAR_256X128 = 5,
  MX_LINEAR_256X256 = 6,
  MX_LINEAR_32X32_BF16 = 7   /* 32 x 32, bf16 tokens quantised by each workgroup */
} mx_linear_kernel;

/*
 * Which of them mx_linear_fused takes for a size on the current device (256
 * CUs are assumed where there is none), or a negative mx_status for sizes that
 * it refuses and for T = 0.  For profiles and tests; enqueues nothing.
 */
int mx_linear_fused_kernel(int64_t T, int64_t K, int64_t N, int x_is_mx);

/*
 * The INT8 path: W8A8 with one fp32 scale per token and per output channel, the
 * other 8-bit format beside MXFP8 ("PR #30768 report", implementation breakdown:
 * the activation quantiser goes by type, e4m3 or int8).
 *
 * int8_quantize: `rows` rows of `kd` bf16 elements (row stride `ld` >= kd) to
 * int8 codes q [rows, kd] and scales s fp32 [rows]; the tokens of a product, or a
 * weight's output channels (rows of [N, K] or [E, N, K]) at load time:
 *   s[r] = max(amax[r] * fl(1/127), 2^-126),   amax[r] = max |x[r, :]|
 *   q[r, c] = nearest integer to fl(x[r, c] * fl(1 / s[r])), ties to even
 * with fl and the products rounded to fp32, so that every code is determined;
 * |q| <= 127.  A row with a NaN gets the scale NaN, else one with an infinity the
 * scale infinity, and codes 0 both, so that its products are NaN (and stay NaN through
 * int8_linear's activations).  Any kd from 1 to 2^24, any alignment of whole elements
 * (rows of a multiple of 8 elements on 16-byte boundaries, q on 8, are the fastest).
 */
int int8_quantize(const void* x_bf16, int64_t rows, int64_t kd, int64_t ld,
                  void* q_i8, float* s, void* stream);

/* Workspace bytes int8_linear needs (x_is_int8: x comes as int8). */
size_t int8_linear_workspace_size(int64_t T, int64_t K, int64_t N, int x_is_int8);

/*
 * Dense INT8 linear layer with its epilogue fused:
 *   z[t, n]   = (sum_k xq[t, k] * wq[n, k]) * x_s[t] * w_s[n]
 *   y[t, n]   = bf16_rne( activation(z[t, n] + bias[n]) + residual[t, n] )
 * the sum exact (int32), everything after it in fp32.  Codes may be any int8,
 * -128 among them; scales any fp32.
 *   x         int8 [T, K] with x_s fp32 [T], or with a NULL x_s bf16 [T, K],
 *             quantised first (as int8_quantize; up to 16 tokens of up to 16384
 *             elements together need no workspace for it while N <= 8192)
 *   w, w_s    int8 [N, K], fp32 [N]
 *   bias      [N] bf16 or fp32 (bias_type), or NULL
 *   residual  bf16 [T, N] or NULL;  y bf16 [T, N]
 * y may be the residual itself (the same address); any other overlap of y or of
 * the workspace is MX_ERR_INVALID_ARG.  Limits: K % 16 == 0, K < 2^17 (the sum
 * stays within int32), N < 2^27, fewer than 2^28 tiles of 32 x 32 outputs.
 * Alignment: int8 operands on 16-byte boundaries, the workspace on 256, the rest
 * on their elements.
 */
int int8_linear(const void* x, const float* x_s, const void* w_i8,
                const float* w_s, const void* bias, int bias_type,
                int activation, const void* residual_bf16, int64_t T,
                int64_t K, int64_t N, void* y_bf16, void* workspace,
                size_t ws_bytes, void* stream);

/*
 * Grouped INT8 product over rows sorted by expert (gmm_mx's counterpart), for
 * expert e and its rows m:
 *   z[m, n] = (sum_k a[m, k] * w[e, n, k]) * a_s[m] * w_s[e, n]
 *   y[m, n] = bf16_rne( z[m, n] )                            swiglu == 0
 *   y[m, n] = bf16_rne( silu(z[m, n]) * z[m, N + n] )        swiglu != 0
 *   a  int8 [M, K], a_s fp32 [M]
 *   w  int8 [E, N, K], w_s fp32 [E, N]; with swiglu [E, 2N, K] and [E, 2N], the
 *      gate rows first (as w13)
 *   y  bf16 [M, N]
 * group_list int64 [E], group_list_type 0 = cumulative, 1 = count.  Rows not
 * owned by any expert are not written.  Limits and alignment as int8_linear,
 * E <= 1024; fewer than 2^28 tiles of 32 x 32 outputs for M + 32 E rows.
 */
int gmm_int8(const void* a_i8, const float* a_s, const void* w_i8,
             const float* w_s, const int64_t* group_list, int group_list_type,
             int swiglu, int64_t M, int64_t N, int64_t K, int64_t E,
             void* y_bf16, void* stream);

/* The kernels of int8_linear and gmm_int8, by their tiles (weight rows x rows of
 * x). */
typedef enum mx_int8_kernel {
  MX_INT8_32X16 = 0,
  MX_INT8_32X16_WIDE = 1, /* K over 8 waves, one workgroup per CU */
  MX_INT8_32X32 = 2,
  MX_INT8_48X48 = 3,      /* int8_linear only */
  MX_INT8_64X64 = 4,
  MX_INT8_128X128 = 5,
  MX_INT8_256X256 = 6,
  MX_INT8_32X16_BF16 = 7  /* bf16 tokens quantised by each workgroup */
} mx_int8_kernel;

/*
 * Which of them a size takes on the current device (256 CUs are assumed where
 * there is none), or a negative mx_status for sizes that are refused and for no
 * rows.  For profiles and tests; enqueues nothing.
 */
int int8_linear_kernel(int64_t T, int64_t K, int64_t N, int x_is_int8);
int gmm_int8_kernel(int64_t M, int64_t N, int64_t K, int64_t E, int swiglu);

/*
 * Token rows of any type sorted by expert: moe_route_quant without the
 * quantiser.  Row p of xp is token sorted_row[p] / k's row, byte for byte; with
 * x_s (the scales of int8 rows; xp_s then too) its scale goes along.
 *   x    [T, K] elements of elem_bytes = 1, 2 or 4, row stride ldx >= K elements
 *   x_s  fp32 [T] or NULL, xp_s fp32 [T*k] or NULL
 *   xp   [T*k, K], dense
 * The maps, the group list, the workspace (moe_route_quant_workspace_size, on an
 * 8-byte boundary), the bounded waits and the limits are those of
 * moe_route_quant, but K may be anything from 1 to 2^24 and rows may lie on any
 * boundary of elements.  Rows past sum(group_list) are left unwritten.  An output
 * that overlaps an input, another output or the workspace is MX_ERR_INVALID_ARG.
 * Its gradient is moe_unpermute without weights.
 */
int moe_permute(const void* x, int64_t ldx, int64_t elem_bytes, const float* x_s,
                const int32_t* topk_ids, int64_t T, int64_t K, int64_t k,
                int64_t E, void* xp, float* xp_s, int32_t* sorted_row,
                int32_t* expanded_row_idx, int64_t* group_list, void* workspace,
                size_t ws_bytes, void* stream);

/*
 * Expert rows back to their tokens, weights applied: moe_finalize for rows of
 * any width and type, also without weights.
 *   out[t, :] = round( sum_{j=0}^{k-1} w[t, j] * y[expanded_row_idx[t*k+j], :] )
 * accumulated in fp32 in ascending j, each product and sum rounded to fp32, the
 * result once to the rows' type; w = 1 with a NULL topk_w.  Entries outside
 * [0, M) are skipped; a token with none left gets zeros.
 *   y [M, K], out [T, K] of `type` (mx_type); topk_w fp32 [T, k] or NULL;
 *   expanded_row_idx int32 [T*k]
 * K from 1 to 2^24, k from 1 to 2^20, T*k < 2^31, any alignment of whole elements.
 * out overlaps no input (MX_ERR_INVALID_ARG).
 */
int moe_unpermute(const void* y, int type, const float* topk_w,
                  const int32_t* expanded_row_idx, int64_t T, int64_t K,
                  int64_t k, int64_t M, void* out, void* stream);

/*
 * The gradients of moe_unpermute (and of moe_finalize), for p =
 * expanded_row_idx[t*k+j]:
 *   dy[p, :] = round( w[t, j] * dout[t, :] )            w = 1 with a NULL topk_w
 *   dw[t, j] = sum_c dout[t, c] * y[p, c]  in fp32      (0 where p is no row)
 *   dout [T, K], y and dy [M, K] of `type`; y may be NULL when dw is; dw fp32
 *   [T, k] or NULL.
 * Rows of dy that no entry names are left as they are, so the entries within
 * [0, M) have to be distinct, as moe_permute makes them (of a row named twice the
 * contents are unspecified).  Limits, alignment and overlaps as moe_unpermute.
 */
int moe_unpermute_backward(const void* dout, int type, const void* y,
                           const float* topk_w, const int32_t* expanded_row_idx,
                           int64_t T, int64_t K, int64_t k, int64_t M, void* dy,
                           float* dw, void* stream);

/* Description of the last non-OK status returned on this thread. */
const char* mx_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MXMOE_H */
