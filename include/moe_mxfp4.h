/*
 * moe_mxfp4.h -- C ABI of the MXFP4 mixture-of-experts layer for GB300 (sm_103a).
 *
 * The layer (the MoE block of a gpt-oss-style decoder) is:
 *   router GEMV/GEMM -> top-k with softmax over the selected logits -> per-expert
 *   tile table -> permute -> grouped gate/up GEMM with SwiGLU -> down GEMM with the
 *   weighted top-k combine and unpermute.
 * Sources: "A 297-line kernel file that decodes faster than vLLM" (cloudy.so),
 * section "Where the time went" (rows "Router + top-k", "MoE gate/up + SwiGLU",
 * "MoE down + combine") and section "Optimizations" (rows "MXFP4 MoE on tensor
 * cores", "Per-expert routing tile table", "Fixed decode tiles", "MoE token tile
 * follows tokens per expert"); "triton-kernels" README (bassrehab), section
 * "Quick Start", "Fused MoE Dispatch" (router -> permute -> fused expert FFN ->
 * unpermute, returning output, expert indices and expert weights).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers owned by the caller unless stated otherwise.  The
 *    library never allocates or frees device memory on these paths.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and never synchronise the host, except moe_prepare_weights,
 *    moe_prepare_matvec, moe_get_device_status, moe_route_noalloc_status,
 *    moe_dense_status and moe_tensor_peak.
 *  - The return value is a status: MOE_OK (0) or a negative MOE_ERR_* code.  On an
 *    error nothing has been launched unless the code is MOE_ERR_CUDA.
 *  - Shapes: 1 <= T, T * k <= 2^24, H % 32 == 0 with 32 <= H <= 8192, I % 32 == 0
 *    with 32 <= I <= 16384, 1 <= k <= E <= 256, k <= 32.
 *  - bf16 arrays are raw bf16 bit patterns (uint16_t).
 *  - Expert weights: MXFP4 = FP4 E2M1 codes in blocks of 32 along K sharing one
 *    E8M0 scale, value = E2M1[code] * 2^(scale - 127) (OCP MX v1.0).  Raw layout:
 *    codes [E][rows][K/2] bytes with the even K index in the low nibble, scales
 *    [E][rows][K/32] bytes.  Gate/up rows: gate rows 0..I-1 then up rows I..2I-1
 *    (K = H).  Down rows: H rows (K = I).
 *  - Alignment: every device pointer 16-byte aligned; workspace and prepared
 *    weights 256-byte aligned.
 */
#ifndef MOE_MXFP4_H
#define MOE_MXFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* moe_stream_t; /* same type as cudaStream_t */

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)       /* null pointer, bad alignment, bad flag      */
#define MOE_ERR_UNSUPPORTED_SHAPE (-2) /* shape outside the supported set above      */
#define MOE_ERR_WORKSPACE_TOO_SMALL (-3)
#define MOE_ERR_CUDA (-4)              /* a launch or driver call failed             */
#define MOE_ERR_DEVICE_TIMEOUT (-5)    /* a bounded device-side wait gave up          */
#define MOE_ERR_NAN_SCALE (-6)         /* an E8M0 scale byte of 255 (NaN) in weights */

#define MOE_WEIGHTS_GATEUP 0
#define MOE_WEIGHTS_DOWN 1

#define MOE_ROUTE_FROM_LOGITS 1 /* moe_route: `logits` is an input, skip the GEMV */
/* Gating variants (moe_route flags, moe_forward_gated): the k experts are selected the
 * same way in every one (the k largest logits, ties to the lower index); only their
 * weights differ.  Default (neither flag): softmax over the k selected logits.
 * "triton-kernels" README, "Project Structure" (router: softmax / sigmoid gating +
 * top-k) and "References" (DeepSeek-V3: sigmoid gating).                          */
#define MOE_ROUTE_GATING_SOFTMAX_ALL 2 /* w_j = exp(l_j) / sum over all E of exp(l_e)   */
#define MOE_ROUTE_GATING_SIGMOID 4     /* w_j = sigmoid(l_j) / sum over the k selected  */

/* Static description of a status code; never NULL. */
const char* moe_error_string(int status);

/* ------------------------------------------------------------------ weights
 * One-time re-layout of raw MXFP4 expert weights into the layout the tensor-core
 * kernels stream: the codes stay row major, [E][rows][K/2] (the TMA boxes of 128
 * rows x 256 codes are cut from them directly), and the E8M0 scales are regrouped
 * into 512-byte atoms of 128 rows x 4 MX blocks, the order in which the
 * block-scaled MMA reads them, [E][groups][rows/128][K groups of 128, rounded up to
 * even][512] (groups = 2 for gate/up: gate rows, up rows).  No value is re-quantised;
 * the bytes are only moved ("MXFP4 MoE on tensor cores": weights permuted once at
 * load).
 *   kind  MOE_WEIGHTS_GATEUP: rows = 2*I (gate then up), K = H.
 *         MOE_WEIGHTS_DOWN:   rows = H, K = I.
 *   codes [E][rows][K/2], scales [E][rows][K/32]: device, read only.
 *   dst: device, moe_prepared_weight_bytes(...) bytes, 256-byte aligned, written.
 * Scale bytes of 255 are rejected: the call returns MOE_ERR_NAN_SCALE after the
 * stream has finished (it synchronises `stream`, as a load-time call may).
 */
size_t moe_prepared_weight_bytes(int E, int rows, int K, int kind);
int moe_prepare_weights(const uint8_t* codes, const uint8_t* scales, int E, int rows, int K, int kind,
                        void* dst, size_t dst_bytes, moe_stream_t stream);

/* One-time re-layout of bf16 expert weights for moe_forward_bf16 into the tiles its
 * tensor-core kernels stream, one bulk copy each.  Tile (e, g, m, s) holds rows
 * [128 m, 128 m + 128) of row group g of expert e (gate rows then up rows for
 * gate/up, one group for down) and their values [64 s, 64 s + 64): 128 rows of
 * 128 bytes, the 16-byte chunk c of row r stored at chunk c ^ (r % 8) (the 128-byte
 * swizzle the MMA reads), rows past the group's end zero.  Tiles are ordered
 * [E][groups][ceil(rows per group / 128)][K / 64], followed by one zero tile.  The
 * values are copied unchanged.  The pages' Triton kernels read the weights as
 * stored; this is a layout of this implementation (weights permuted once at load,
 * as for MXFP4).
 *   kind, rows, K: as moe_prepare_weights; rows a multiple of the group count, K a
 *   multiple of 64.
 *   w bf16 [E][rows][K]: device, 16-byte aligned, read only.
 *   dst: device, moe_prepared_weight_bytes_bf16(...) bytes, 256-byte aligned, written.
 * Returns MOE_OK, MOE_ERR_UNSUPPORTED_SHAPE, MOE_ERR_INVALID_ARG,
 * MOE_ERR_WORKSPACE_TOO_SMALL or MOE_ERR_CUDA; asynchronous on `stream`.          */
size_t moe_prepared_weight_bytes_bf16(int E, int rows, int K, int kind);
int moe_prepare_weights_bf16(const uint16_t* w, int E, int rows, int K, int kind, void* dst, size_t dst_bytes,
                             moe_stream_t stream);

/* ------------------------------------------------------------------ sizes
 * Token rows per tile chosen for a shape (16, 64 or 128 from the mean tokens per
 * expert T*k/E; fixed per shape, never autotuned) and the bound on tile count.  */
int moe_tile_rows(int T, int k, int E);
int moe_max_tiles(int T, int k, int E, int tile_rows);

/* Bytes of device workspace needed by moe_forward and the stage calls below for
 * this shape; 0 for an unsupported shape.  The workspace holds routing results,
 * quantised activations, the slot buffer of the combine, arrival counters and a
 * status word.  Zero-fill it once after allocation (cudaMemset); every call leaves
 * its counters at zero again, so it can serve consecutive calls on one stream.
 * Calls that overlap on the GPU must not share a workspace.                       */
size_t moe_workspace_bytes(int T, int H, int I, int E, int k);

/* ------------------------------------------------------------------ stage calls
 * moe_route: logits[t, e] = sum_h x[t, h] * w_router[e, h] (+ router_bias[e]) in
 * fp32; then per token the k largest logits (ties: lower expert index first),
 * listed in that order, and weights = softmax over those k logits (or the gating
 * variant a MOE_ROUTE_GATING_* flag names; both flags at once is invalid).
 *   x bf16 [T, H]; w_router bf16 [E, H]; router_bias f32 [E] or NULL.
 *   logits f32 [T, E]: written, or read when flags has MOE_ROUTE_FROM_LOGITS (then
 *   x, w_router and router_bias may be NULL).
 *   topk_idx i32 [T, k], topk_w f32 [T, k]: written.
 *   workspace: zero-filled once, at least moe_workspace_bytes(T, 32, 32, E, k)
 *   bytes; only its status word and routing arrival counters are used.
 * Source: "Where the time went", row "Router + top-k"; "Quick Start",
 * fused_moe_forward(..., gating="softmax").                                        */
int moe_route(const uint16_t* x, const uint16_t* w_router, const float* router_bias, int T, int H, int E, int k,
              float* logits, int flags, int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
              moe_stream_t stream);

/* moe_route_noalloc: moe_route for callers that cannot allocate device memory.
 * The pages have no counterpart of this entry point; it exists for callers such as
 * a serving runtime that owns a fixed memory pool, or a plugin that is handed only
 * its input and output buffers, which have no way to call cudaMalloc for the
 * workspace moe_route wants.  It computes exactly what moe_route computes, with
 * the same arguments minus the workspace: the small scratch moe_route keeps in
 * the workspace (a status word and the arrival counters of its last-block
 * hand-off) lives instead in a fixed array compiled into the library,
 * 256 + 4 * (8192 / 8 + 1) = 4356 bytes, which every GPU that loads the library
 * holds until the process exits.
 *   T must be <= 8192: larger T returns MOE_ERR_UNSUPPORTED_SHAPE.
 *   The first call on a device looks up the array's device address for that
 *   device (once per device, with it current); make that first call before any
 *   stream capture.  The array is zero when the library loads and every call
 *   leaves its counters at zero again, so no call clears anything before it
 *   launches.
 *   All calls share the one array: calls that overlap on the GPU (on different
 *   streams, or from several threads) race and must be serialised by the caller.
 *   A bounded device wait that gives up sets the array's status word; read it with
 *   moe_route_noalloc_status (a routing whose status is non-zero is not reliable). */
int moe_route_noalloc(const uint16_t* x, const uint16_t* w_router, const float* router_bias, int T, int H, int E,
                      int k, float* logits, int flags, int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/* moe_route_noalloc_status: the device status of moe_route_noalloc on the current
 * device.  The pages have no counterpart of it; it is moe_get_device_status for the
 * fixed array.  Synchronises `stream`, reads the array's status word into *status
 * (bits as in moe_get_device_status; 0 = healthy) and, when it is non-zero, clears
 * the whole array, status word and arrival counters alike.  Returns MOE_OK,
 * MOE_ERR_DEVICE_TIMEOUT when a bit was set, MOE_ERR_INVALID_ARG for a NULL
 * status, or MOE_ERR_CUDA.  Not for the hot path.                                 */
int moe_route_noalloc_status(int* status, moe_stream_t stream);

/* moe_build_tile_table: the per-expert tile table of a routing ("Per-expert
 * routing tile table": each expert writes its own tiles).  Atomic-free counting
 * sort, deterministic:
 *   counts[e] (i32 [E]); offsets (i32 [E+1], exclusive prefix sum, offsets[E] = T*k);
 *   perm[s] (i32 [T*k]) = assignment t*k+j at sorted row s, rows sorted by expert
 *   then ascending t*k+j; inv_perm (i32 [T*k]) its inverse;
 *   tiles (i32 [max_tiles][4]) = {expert, first sorted row, rows (1..tile_rows),
 *   tile*tile_rows}, experts ascending, ceil(counts[e]/tile_rows) tiles each;
 *   num_tiles (i32 [1]).
 *   tile_rows: 16, 64 or 128, or 0 for moe_tile_rows(T, k, E).
 *   topk_idx i32 [T, k] with entries in [0, E): read.                              */
int moe_build_tile_table(const int32_t* topk_idx, int T, int k, int E, int tile_rows, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* tiles, int32_t* num_tiles,
                         moe_stream_t stream);

/* moe_mxfp4_gateup_swiglu: for every tile (expert e, rows of perm) and every
 * hidden feature i: g = x_t . W_gate[e][i], u = x_t . W_up[e][i], h = silu(g) * u.
 * Three launches: every token row of x is encoded once as a sum of four E2M1
 * terms, each with its own E8M0 scale per 32-value block; the encoded rows are
 * gathered by perm (the permute step) into tile order; the GEMM runs.  The
 * weights stay MXFP4 and both operands' scales feed the block-scaled MMA
 * (kind::mxf4) directly.
 * h is left in the workspace, encoded the same way in tile row order, for
 * moe_mxfp4_down_combine.
 *   x bf16 [T, H]; perm, tiles, num_tiles as written by moe_build_tile_table with
 *   the same tile_rows (0 = policy); w_gateup: moe_prepare_weights(MOE_WEIGHTS_GATEUP).
 * Source: "Where the time went", row "MoE gate/up + SwiGLU".                       */
int moe_mxfp4_gateup_swiglu(const uint16_t* x, const int32_t* perm, const int32_t* tiles, const int32_t* num_tiles,
                            int tile_rows, const void* w_gateup, int T, int H, int I, int E, int k, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream);

/* moe_mxfp4_down_combine: y_tj = h_tj . W_down[e_tj]^T for every assignment, then
 * out[t] = sum_{j=0..k-1} topk_w[t, j] * y_tj summed in fp32 in ascending j and
 * rounded once to bf16 -- deterministic run to run.  Reads h from the workspace
 * (written by moe_mxfp4_gateup_swiglu for the same routing).  Two launches: the
 * down GEMM writes w_tj * y_tj into a per-assignment fp32 slot of the workspace,
 * then a combine kernel sums each token's k slots.
 *   topk_w f32 [T, k]; w_down: moe_prepare_weights(MOE_WEIGHTS_DOWN); out bf16 [T, H].
 * Source: "Where the time went", row "MoE down + combine".                         */
int moe_mxfp4_down_combine(const int32_t* perm, const int32_t* tiles, const int32_t* num_tiles, int tile_rows,
                           const float* topk_w, const void* w_down, int T, int H, int I, int E, int k,
                           void* workspace, size_t workspace_bytes, uint16_t* out, moe_stream_t stream);

/* moe_hidden_dequant: expand the workspace's four-term encoded h into f32
 * [T*k, I] rows in assignment order (t*k + j); a test and inspection aid.          */
int moe_hidden_dequant(const int32_t* perm, const int32_t* tiles, const int32_t* num_tiles, int tile_rows, int T,
                       int H, int I, int E, int k, const void* workspace, size_t workspace_bytes, float* h_out,
                       moe_stream_t stream);

/* ------------------------------------------------------------------ whole layer
 * moe_forward_gated: moe_forward with the top-k weights of the gating variant
 * `gating` (0, MOE_ROUTE_GATING_SOFTMAX_ALL or MOE_ROUTE_GATING_SIGMOID; any other
 * value is MOE_ERR_INVALID_ARG).                                                   */
int moe_forward_gated(const uint16_t* x, const uint16_t* w_router, const float* router_bias, const void* w_gateup,
                      const void* w_down, int T, int H, int I, int E, int k, int gating, void* workspace,
                      size_t workspace_bytes, uint16_t* out, int32_t* topk_idx_out, float* topk_w_out,
                      moe_stream_t stream);

/* moe_forward_norm: the step before the layer fused into it, then the layer:
 *   s = bf16(x + residual)                      (the residual stream, returned)
 *   y = bf16(s / sqrt(mean_H(s^2) + eps) * norm_weight)
 *   out = MoE(y)  (moe_forward_gated on y; `gating` as there).
 * Sources: "triton-kernels" README, "Kernels" (rmsnorm_residual_fused) and "Quick
 * Start", "Fused RMSNorm + Residual"; the decode-engine page "A 297-line kernel file
 * that decodes faster than vLLM", "Where the time went", row "RMSNorm + residual".
 * No launch is added: the routing kernel and the encoder each normalise the rows
 * they read (the same bits: one fixed summation order), and the combine kernel
 * writes residual_out.
 *   x, residual bf16 [T, H]; norm_weight bf16 [H]; all 16-byte aligned.
 *   eps: finite and >= 0.
 *   residual_out: bf16 [T, H] or NULL.  It may be x or residual itself: it is
 *   written after every read of both.  It may not be `out`.
 * Errors: MOE_ERR_INVALID_ARG for a NULL or misaligned x, residual or norm_weight,
 * a bad eps or gating value, or residual_out == out.  Everything else is as for
 * moe_forward.                                                                     */
int moe_forward_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* norm_weight, float eps,
                     const uint16_t* w_router, const float* router_bias, const void* w_gateup, const void* w_down,
                     int T, int H, int I, int E, int k, int gating, void* workspace, size_t workspace_bytes,
                     uint16_t* out, uint16_t* residual_out, int32_t* topk_idx_out, float* topk_w_out,
                     moe_stream_t stream);

/* moe_forward_bf16: the same layer with bf16 expert weights instead of MXFP4.
 * This is the "Fused MoE Dispatch" workload of the "triton-kernels" README
 * ("Quick Start"; "MoE Dispatch Results": Mixtral-8x7B, 8 experts, top-2,
 * hidden 4096, ffn 14336): router -> top-k softmax gating -> permute -> gate/up +
 * SwiGLU -> down -> weighted combine + unpermute.
 * Launches:
 *   - routing: as moe_forward;
 *   - permute: bf16 rows of x into tile order;
 *   - gate/up and down: the grouped tcgen05 GEMMs with kind::f16 (bf16 x bf16,
 *     f32 accumulate); h is rounded to bf16 between them.  Tiles are 256 token rows
 *     once T*k >= 256*E (N = 256 MMAs), else moe_tile_rows(T, k, E);
 *   - combine: as moe_forward.
 * Arguments:
 *   x bf16 [T, H]; w_router bf16 [E, H]; router_bias f32 [E] or NULL;
 *   w_gateup: moe_prepare_weights_bf16(MOE_WEIGHTS_GATEUP) of bf16 [E, 2I, H], gate
 *   rows [0, I) then up rows [I, 2I); w_down: moe_prepare_weights_bf16(MOE_WEIGHTS_DOWN)
 *   of bf16 [E, H, I].  All pointers are 16-byte aligned.
 *   workspace: moe_workspace_bytes(T, H, I, E, k) bytes, 256-byte aligned.
 *   out bf16 [T, H].
 *   topk_idx_out / topk_w_out: as moe_forward.
 * Errors:
 *   - MOE_ERR_UNSUPPORTED_SHAPE as moe_forward, and also unless H and I are
 *     multiples of 64;
 *   - MOE_ERR_INVALID_ARG for NULL or misaligned pointers;
 *   - MOE_ERR_WORKSPACE_TOO_SMALL.                                                  */
int moe_forward_bf16(const uint16_t* x, const uint16_t* w_router, const float* router_bias, const uint16_t* w_gateup,
                     const uint16_t* w_down, int T, int H, int I, int E, int k, void* workspace,
                     size_t workspace_bytes, uint16_t* out, int32_t* topk_idx_out, float* topk_w_out,
                     moe_stream_t stream);

/* moe_forward: the whole layer, out = MoE(x), on one stream with no host sync.
 *   x bf16 [T, H]; w_router bf16 [E, H]; router_bias f32 [E] or NULL;
 *   w_gateup / w_down: prepared weights; out bf16 [T, H];
 *   topk_idx_out i32 [T, k] and topk_w_out f32 [T, k]: optional copies (NULL to skip).
 *   workspace: moe_workspace_bytes(T, H, I, E, k) bytes.                           */
int moe_forward(const uint16_t* x, const uint16_t* w_router, const float* router_bias, const void* w_gateup,
                const void* w_down, int T, int H, int I, int E, int k, void* workspace, size_t workspace_bytes,
                uint16_t* out, int32_t* topk_idx_out, float* topk_w_out, moe_stream_t stream);

/* moe_forward_timed: moe_forward that also records caller-created CUDA events
 * (cudaEvent_t, passed as void*) on `stream` around its MOE_FORWARD_STAGES stages:
 * events[i] just before stage i and events[MOE_FORWARD_STAGES] after the last one.
 * The stages are its five launches: route + top-k + tile table, the per-token
 * encoding of x (which waits for routing and writes the tile order itself: the
 * permute step), the gate/up + SwiGLU GEMM, the down GEMM, and the combine.  It
 * gives the per-launch time split ("Where the time went": per-section times of a
 * decode step); an event between two launches also separates them, so the
 * programmatic-launch overlap of consecutive kernels is lost in this form.
 * events must hold MOE_FORWARD_STAGES + 1 valid events.                          */
#define MOE_FORWARD_STAGES 5
int moe_forward_timed(const uint16_t* x, const uint16_t* w_router, const float* router_bias, const void* w_gateup,
                      const void* w_down, int T, int H, int I, int E, int k, void* workspace,
                      size_t workspace_bytes, uint16_t* out, int32_t* topk_idx_out, float* topk_w_out,
                      void* const* events, moe_stream_t stream);

/* Number of kernels moe_forward launches for a shape (for launch accounting):
 * route + top-k + table, encode + permute x, gate/up, down, combine.             */
int moe_forward_launches(int T, int H, int I, int E, int k);

/* moe_tensor_peak: the measured dense tensor-pipe rate of this GPU, in TFLOP/s, for
 * one of the MMA forms the expert GEMMs issue, as the roofline peak of the
 * compute-bound (many-token) workloads.  The pages give no tensor peak for this
 * hardware; the 4096-token prefill case is to be reported against the MXFP4 rate.
 *   kind MOE_PEAK_MXF4: tcgen05 kind::mxf4 block-scaled (E2M1 x E2M1, E8M0 scales,
 *        K = 64 per instruction), the MXFP4 layer's GEMMs;
 *   kind MOE_PEAK_BF16: kind::f16 (bf16 x bf16, K = 16), the bf16-weight layer.
 * One CTA per SM issues mmas_per_sm (8 .. 2^24) MMAs of M = 128, N = 256 back to
 * back into tensor memory; the call times that launch with CUDA events on
 * `stream`, synchronises it and writes 2*M*N*K*mmas*SMs / time to *tflops.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_CUDA, or MOE_ERR_DEVICE_TIMEOUT when
 * the bounded completion wait gave up.  Not for the hot path.                      */
#define MOE_PEAK_MXF4 0
#define MOE_PEAK_BF16 1
int moe_tensor_peak(int kind, int mmas_per_sm, double* tflops, moe_stream_t stream);

/* ------------------------------------------------------------------ dense operators
 * What a decoder's half layer needs beside the experts: the norms before and after a
 * block, a dense gated feed-forward block, and products of a few tokens with MXFP4
 * weights that need no routing.  The pages name the pieces ("triton-kernels" README,
 * "Kernels": rmsnorm_residual_fused, swiglu_fused, the W4A16 GEMM); the operators below
 * are this library's own.  `dtype` is the type of the activations and weights
 * (MOE_DTYPE_BF16 or MOE_DTYPE_F16); every array is contiguous, row major.           */
#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_F16 1
#define MOE_DTYPE_F32 2 /* where a function names it: the norms' stream, out of a projection, rows */

#define MOE_GATE_NONE 0
#define MOE_GATE_FEATURE 1 /* gate [H], of `dtype`                                    */
#define MOE_GATE_TOKEN 2   /* gate f32 [T]                                            */
#define MOE_GATE_FULL 3    /* gate [T, H], of `dtype`                                 */

#define MOE_ACT_SILU 0
#define MOE_ACT_GELU 1 /* tanh form                                                   */
#define MOE_ACT_NONE 2 /* projections only                                            */

/* moe_block_norm: the end of one block and the start of the next in one launch.
 *   n = block / sqrt(mean_H(block^2) + eps) * norm_weight   (n = block without norm_weight)
 *   s = residual_scale * residual + gate * n                rounded to stream_dtype
 *   out = s / sqrt(mean_H(s^2) + eps) * next_weight         of the rounded s
 * All arithmetic is f32; s and out are rounded once.
 *   block [T, H]; norm_weight [H] or NULL; gate by gate_kind (NULL for MOE_GATE_NONE);
 *   residual [T, H] of stream_dtype, or NULL for none; next_weight [H] or NULL;
 *   stream_dtype: dtype or MOE_DTYPE_F32.
 *   residual_out: s, [T, H] of stream_dtype, or NULL when only `out` is wanted; it may
 *   be `residual` itself.  out: [T, H] of dtype; NULL exactly when next_weight is; it
 *   may be `block` itself; outputs overlap inputs in no other way.
 *   1 <= T <= 2^24, H % 8 == 0 with 8 <= H <= 8192; arrays 16-byte aligned (a token
 *   gate 4); eps finite and >= 0; residual_scale finite.
 * Source: "triton-kernels" README, "Kernels" (rmsnorm_residual_fused), with the norm
 * after the block, its gate and the residual scale added.                           */
int moe_block_norm(const void* block, const void* norm_weight, const void* gate, int gate_kind, const void* residual,
                   float residual_scale, const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                   void* residual_out, void* out, moe_stream_t stream);

/* moe_block_norm_8bit: moe_block_norm with `out` in 8 bits, for products with 8-bit
 * activations and for moe_sort_tokens to move: E4M3 codes and scales of the f32 y,
 *   code = E4M3(y (1 / scale)), nearest, ties to even
 *   MOE_SCALE_MX: E8M0 bytes [T, H / 32], scale 2^(byte - 127), one for 32 values: the least
 *     with |y| <= 448 scale (2^-126 at least), so that no value saturates.  H % 32 == 0.
 *     (Powers of two: the product is exact.)
 *   MOE_SCALE_ROW: f32 [T], one for a row: max |y| (1 / 448) (2^-126 at least).  Here 1 / 448,
 *     1 / scale and both products are rounded to f32, so that a y within 4 2^-24 of itself of
 *     a tie between two codes may get the other of the two.
 * A group with an infinite or NaN y has a NaN scale (E8M0 255) and NaN codes.
 *   codes [T, H] bytes, written, and scales: overlap nothing else.  residual_out, or NULL.
 *   out: y rounded to dtype as well (for a router, say), or NULL.  next_weight is needed;
 *   every other argument as for moe_block_norm.  Gradients: moe_block_norm_backward, the
 *   rounding passing d_out through.                                                  */
#define MOE_SCALE_MX 0
#define MOE_SCALE_ROW 1
int moe_block_norm_8bit(const void* block, const void* norm_weight, const void* gate, int gate_kind, const void* residual,
                        float residual_scale, const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                        int scale_kind, void* residual_out, uint8_t* codes, void* scales, void* out, moe_stream_t stream);

/* moe_block_norm_backward: every gradient of moe_block_norm, from the same arguments.
 *   d_residual_out [T, H] of stream_dtype: gradient into s from what reads the stream
 *   later, or NULL for none; d_out [T, H] of dtype: NULL exactly when next_weight is (one
 *   of the two must be given).  residual_out: the s of the forward (needed with
 *   next_weight; the rounding of s passes the gradient through).
 *   d_block [T, H] of dtype: written.  d_residual [T, H] of stream_dtype, or NULL.
 *   d_norm_weight, d_next_weight: f32 [H], or NULL.  d_gate, or NULL: f32 [H] for a
 *   feature gate, f32 [T] for a token gate, [T, H] of dtype for a full gate.
 *   d_block may be `block`, d_residual may be `d_residual_out`; no other aliasing.
 *   workspace: moe_block_norm_workspace_bytes(T, H) bytes, 256-byte aligned, contents
 *   irrelevant before and after.  The weight gradients are summed in a fixed order, so
 *   results repeat bit for bit.                                                     */
size_t moe_block_norm_workspace_bytes(int T, int H);
int moe_block_norm_backward(const void* d_residual_out, const void* d_out, const void* block, const void* norm_weight,
                            const void* gate, int gate_kind, const void* residual_out, float residual_scale,
                            const void* next_weight, float eps, int T, int H, int dtype, int stream_dtype,
                            void* d_block, void* d_residual, float* d_norm_weight, void* d_gate, float* d_next_weight,
                            void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* moe_ffn_forward: a dense gated feed-forward block with 16-bit weights (a shared expert
 * or a dense layer beside the experts).
 *   g = x W_gate^T, u = x W_up^T, h = act(g) * u        one kernel
 *   out = h W_down^T
 * Sums are f32; h is rounded to dtype between the products: in f16 an h beyond 65504 becomes
 * infinite and one below 2^-14 loses bits, where bf16 has f32's range.
 *   x [T, H]; w_gateup [2I, H], gate rows [0, I) then up rows; w_down [H, I]: as stored,
 *   nothing is prepared; out [T, H], which may be x itself.
 *   gateup_out: f32 [T, 2I] (g, then u), written for moe_ffn_backward; NULL to skip.
 *   1 <= T <= 2^24, H and I multiples of 8 from 8 to 2^17; arrays 16-byte aligned,
 *   workspace moe_ffn_workspace_bytes(T, H, I, 0) bytes, 256-byte aligned, contents
 *   irrelevant before and after.  Up to 16 tokens take a kernel that streams the weights
 *   through mma.sync, more the tcgen05 GEMMs.
 * Source: "triton-kernels" README, "Kernels" (swiglu_fused).                        */
size_t moe_ffn_workspace_bytes(int T, int H, int I, int backward);
int moe_ffn_forward(const void* x, const void* w_gateup, const void* w_down, int T, int H, int I, int act, int dtype,
                    float* gateup_out, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* moe_ffn_backward: the gradients of moe_ffn_forward, from its inputs and saved g, u.
 *   dh = d_out W_down;  dg = dh * u * act'(g);  du = dh * act(g);  h = act(g) * u
 *   d_x = [dg du] w_gateup;  d_w_gateup = [dg du]^T x;  d_w_down = d_out^T h
 * dg, du and h are formed in f32 and rounded to dtype as the next products' operands, with
 * f16's range as above: scale d_out where its gradients are small.
 *   d_x [T, H], d_w_gateup [2I, H], d_w_down [H, I] of dtype: overwritten; each may be
 *   NULL (not all).  workspace: moe_ffn_workspace_bytes(T, H, I, 1) bytes.
 *   No output may overlap an input.  Everything else is as for moe_ffn_forward.      */
int moe_ffn_backward(const void* d_out, const void* x, const float* gateup, const void* w_gateup, const void* w_down,
                     int T, int H, int I, int act, int dtype, void* d_x, void* d_w_gateup, void* d_w_down,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* moe_linear_forward: a projection with 16-bit weights and what follows it.
 *   pre = x W^T + bias;  out = act(pre) + residual      f32, rounded once to out_dtype
 *   x [T, K], weight [N, K] of dtype; bias f32 [N] or NULL; residual [T, N] of out_dtype or
 *   NULL; out [T, N] of out_dtype (dtype, or MOE_DTYPE_F32: router logits, a residual stream
 *   kept in f32), which may be `residual` itself and overlap nothing else.
 *   act: MOE_ACT_NONE, _SILU or _GELU.  pre_out: f32 [T, N] for moe_linear_backward, or NULL;
 *   NULL with MOE_ACT_NONE, whose backward does not need it.
 *   The tensor cores cut each step's addends below the largest: of its terms' norm, pre is off by
 *   4.4e-6 rms over 4096 bf16 terms and 4.9e-6 over f16 ones (2.7e-5 and 3.1e-5 the worst of 4
 *   million; f32 products: 6e-7 and 1.1e-6 rms), by more the longer the sum (16384: 1.9e-5 rms).
 *   1 <= T <= 2^24, K and N multiples of 8, K up to 2^17, N up to 2^20; arrays 16-byte
 *   aligned; workspace moe_linear_workspace_bytes(T, K, N, 0) bytes (0: it may be NULL),
 *   256-byte aligned, apart from every other array, contents irrelevant before and after.  Few
 *   tokens take a kernel that streams the weights through mma.sync, batches of up to 128 and
 *   more the tcgen05 ones.
 * The pages have no counterpart ("triton-kernels" README, "Kernels", lists the fused GEMMs
 * of the feed-forward block).                                                        */
size_t moe_linear_workspace_bytes(int T, int K, int N, int backward);
int moe_linear_forward(const void* x, const void* weight, const float* bias, const void* residual, int T, int K, int N, int act,
                       int dtype, int out_dtype, float* pre_out, void* out, void* workspace, size_t workspace_bytes,
                       moe_stream_t stream);

/* moe_linear_backward: the gradients of moe_linear_forward (the residual's is d_out itself).
 *   dp = d_out act'(pre);  d_x = dp W;  d_weight = dp^T x;  d_bias = sum_t dp
 *   d_out [T, N] of out_dtype; pre: what pre_out received, NULL exactly with MOE_ACT_NONE.
 *   dp is formed in f32, summed into d_bias (f32 [N]) in a fixed order, and rounded to dtype
 *   as the products' operand, that of an f32 d_out too (in f16 with f16's range: scale d_out
 *   where it is small): d_x and d_weight are off by about 1.4 of their own rounding.
 *   d_x [T, K], d_weight [N, K] of dtype, d_bias: overwritten; each may be NULL (not all).
 *   weight may be NULL without d_x, x without d_weight.  No output may overlap an input or
 *   another output.
 *   workspace: moe_linear_workspace_bytes(T, K, N, 1) bytes, 256-byte aligned, apart from every
 *   other array; enough for any of these calls.                                      */
int moe_linear_backward(const void* d_out, const void* x, const void* weight, const float* pre, int T, int K, int N, int act,
                        int dtype, int out_dtype, void* d_x, void* d_weight, float* d_bias, void* workspace,
                        size_t workspace_bytes, moe_stream_t stream);

/* moe_sort_tokens: token rows into expert order, for experts of the caller's own (the
 * layer's permute step by itself), in the order of moe_build_tile_table: by expert, then by
 * assignment a = t*k + j.  An index outside [0, E) drops its assignment (a padding token, an
 * expert that lives elsewhere): dropped assignments follow behind all others, as rows of
 * zeros, and their entries of perm and inv_perm are kept as -1 - entry.
 *   offsets i32 [E + 1]: rows of expert e are [offsets[e], offsets[e + 1]); the rows from
 *   offsets[E] on are those of the dropped.
 *   perm i32 [T*k]: assignment at each row.  inv_perm i32 [T, k]: row of each assignment.
 *   rows [T*k] rows of row_bytes: x[perm / k].  row_scales, or NULL: the same of `scales`.
 *   x: [T] rows of row_bytes bytes (of any type), a multiple of 16 up to 65536; scales: [T]
 *   rows of scale_bytes (0 .. 4096; 0 with scales and row_scales NULL).  T, k and E as in the
 *   conventions above.  Rows 16-byte aligned, the i32 arrays 4; scales and row_scales may begin
 *   at any byte.  No output may overlap an input or another output.
 * Source: "Quick Start", "Fused MoE Dispatch" (permute).                             */
int moe_sort_tokens(const void* x, const void* scales, const int32_t* topk_idx, int T, int k, int E, int row_bytes,
                    int scale_bytes, int32_t* offsets, int32_t* perm, int32_t* inv_perm, void* rows, void* row_scales,
                    moe_stream_t stream);

/* moe_unsort_tokens: rows in expert order back to tokens, weighted:
 *   out[t] = sum_j topk_w[t, j] * y[inv_perm[t, j]]      f32, ascending j, rounded once
 * over the j whose inv_perm is in [0, T*k); a token without any gets zeros, and no other row
 * of y is read.  With topk_w NULL (all 1) it is the gradient of moe_sort_tokens: d_x of d_rows.
 *   y [T*k, H], out [T, H] of dtype (MOE_DTYPE_BF16, _F16 or _F32); H a multiple of 8, a row
 *   at most 65536 bytes; y and out 16-byte aligned, the others 4; out may not overlap an input.
 * Source: "Quick Start", "Fused MoE Dispatch" (unpermute).                           */
int moe_unsort_tokens(const void* y, const int32_t* inv_perm, const float* topk_w, int T, int k, int H, int dtype, void* out,
                      moe_stream_t stream);

/* moe_unsort_tokens_backward: the gradients of moe_unsort_tokens.
 *   d_y[inv_perm[t, j]] = topk_w[t, j] * d_out[t]; a dropped assignment's row (-1 - inv_perm):
 *   zeros, so that after moe_sort_tokens every row of d_y is written
 *   d_topk_w[t, j] = sum_h d_out[t, h] * y[inv_perm[t, j], h]   (f32; 0 where dropped)
 * Either may be NULL; y is read for d_topk_w alone, and may be NULL without it.  Types and
 * sizes as for moe_unsort_tokens; no output may overlap an input or the other output. */
int moe_unsort_tokens_backward(const void* d_out, const void* y, const int32_t* inv_perm, const float* topk_w, int T, int k,
                               int H, int dtype, void* d_y, float* d_topk_w, moe_stream_t stream);

/* moe_route_backward: the gradient of moe_route's weights into its logits.
 *   d_topk_w f32 [T, k]; logits f32 [T, E], topk_idx and topk_w as moe_route gave them (the
 *   indices as routed, not with assignments dropped); gating: moe_route's flag, or 0.
 *   d_logits f32 [T, E]: written whole, 0 where the weights do not depend on the logit.
 *   The selection itself has no gradient.  An expert listed twice gets the sum.  An index
 *   outside [0, E) gets nothing; its weight and gradient count in sum_i w_i g_i as given.
 *   A d_topk_w of 0 (a dropped assignment's) counts as 0 whatever its weight, and a token
 *   whose d_topk_w are all 0 gets zeros, also where its weights or logits are not finite (a
 *   mask that leaves no expert).  Arrays 4-byte aligned; d_logits may not overlap an input. */
int moe_route_backward(const float* d_topk_w, const float* logits, const int32_t* topk_idx, const float* topk_w, int T, int k,
                       int E, int gating, float* d_logits, moe_stream_t stream);

/* moe_dense_status: the device status of the dense operators' pipelines (GEMMs, MXFP4
 * products, row copies of the norms and of the sorted tokens) on the current device, as moe_get_device_status (bits and
 * returns) for words that the library holds per GPU: synchronises `stream`, reads them
 * into *status and clears them when set.  A bounded wait that gave up sets a bit (the limit
 * of the GEMMs and of the sorted tokens' rows is moe_set_wait_limit_ns's, the others' 1 s);
 * results of calls since the last reading are then not reliable.  The launch that gave up
 * stays until its copies have landed (20 ms); others are not held up.  Not for the hot path. */
int moe_dense_status(int* status, moe_stream_t stream);

/* moe_prepare_matvec: one-time re-layout of raw MXFP4 weights [rows][K/2] codes and
 * [rows][K/32] scales (as the expert weights of one expert) for moe_matvec_mxfp4.  The
 * bytes are only moved.
 *   kind: MOE_WEIGHTS_DOWN for a plain product, MOE_WEIGHTS_GATEUP for gate rows
 *   [0, rows/2) and up rows [rows/2, rows) (rows even).
 *   1 <= rows <= 2^22, K % 32 == 0 with 32 <= K <= 65536; codes 16-byte aligned; dst
 *   moe_prepared_matvec_bytes(...) bytes, 256-byte aligned.
 * Scale bytes of 255 are rejected with MOE_ERR_NAN_SCALE after the stream has finished
 * (it synchronises `stream`, as a load-time call may).                              */
size_t moe_prepared_matvec_bytes(int rows, int K, int kind);
int moe_prepare_matvec(const uint8_t* codes, const uint8_t* scales, int rows, int K, int kind, void* dst,
                       size_t dst_bytes, moe_stream_t stream);

/* moe_matvec_mxfp4: products of 1 to 64 tokens with prepared MXFP4 weights.
 *   MOE_WEIGHTS_DOWN:   out[t, n] = sum_k x[t, k] W[n, k] + bias[n]        out [T, rows]
 *   MOE_WEIGHTS_GATEUP: g, u the products (+ bias) of gate row i and up row i,
 *                       out[t, i] = act(g) * u                             out [T, rows/2]
 * Sums are f32 in a fixed order, one rounding at the end.  The codes are used exactly;
 * a group whose scale is below 2^-126 of its row's largest counts as zero.  bf16 x is
 * carried as f16 times a power of two per token: values below 2^-28 of their token's
 * largest lose relative precision (absolute error 2^-39 of it).
 *   x [T, K] of dtype; bias f32 [rows] or NULL; act is read for MOE_WEIGHTS_GATEUP.
 *   out may not overlap x (MOE_ERR_INVALID_ARG).
 *   workspace: moe_matvec_workspace_bytes(T, K) bytes (0 where x fits the
 *   kernel's shared memory: then it may be NULL), 256-byte aligned, contents irrelevant
 *   before and after.
 * Source: "triton-kernels" README, "Kernels" (W4A16 GEMM: 4-bit weights with group
 * scales, 16-bit activations), on the layer's MXFP4 format.                         */
size_t moe_matvec_workspace_bytes(int T, int K);
int moe_matvec_mxfp4(const void* x, const void* w, const float* bias, int T, int rows, int K, int kind, int act,
                     int dtype, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* moe_set_wait_limit_ns: how long (ns) each pipeline wait of the expert GEMMs (and of the
 * dense GEMMs and the copies of sorted tokens' rows, whose status moe_dense_status reads) may
 * take before it gives up, for launches made after the call (process-wide; 0 restores the
 * default of 1 s; at most 10 s, else MOE_ERR_INVALID_ARG).  A wait that gives up sets a
 * bit of the workspace status word (moe_get_device_status) or of the dense one, the kernel
 * drops its remaining work, waits (up to 1 s) for the copies and tensor-core
 * operations it has already issued, frees its tensor memory and exits: no trap, and
 * the context stays usable.  Limits under 2 us are polled without suspending the
 * waiting thread, so a limit shorter than the pipeline's own latency (a copy landing
 * takes about a microsecond even from L2) makes waits give up on ordinary calls;
 * that is how failure detection is tested.  The pages have no counterpart of it.   */
int moe_set_wait_limit_ns(unsigned long long ns);

/* Synchronises `stream`, reads the workspace's device status word into *status
 * (bit 0: main-loop wait timed out, bit 1: epilogue wait timed out, bit 2:
 * producer wait timed out; 0 = healthy) and clears it.  Returns MOE_OK, or
 * MOE_ERR_DEVICE_TIMEOUT when any bit was set.  After a timeout the call's outputs
 * are not reliable and the workspace's arrival counters may be left non-zero:
 * zero-fill the workspace again before its next use.  Not for the hot path.        */
int moe_get_device_status(void* workspace, size_t workspace_bytes, int* status, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MXFP4_H */
