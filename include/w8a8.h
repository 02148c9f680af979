/*
 * w8a8.h — C ABI of the MI355X (gfx950) fused W8A8 linear library, libw8a8.so.
 *
 * The operation is the one in the abstract of "Realizing Native INT8 Compute
 * for Diffusion Transformers on Consumer GPUs: A Fused INT8 GEMM Kernel for
 * Ideogram 4.0" (arXiv 2606.14598): activations are quantized to int8 per
 * token, weights per (output) channel, the product is accumulated
 * int8 x int8 -> int32 on the matrix cores, and the per-token x per-channel
 * dequantization plus the bias are folded into the GEMM epilogue, which
 * writes bf16.
 *
 * Conventions shared by every entry point
 *   - All tensors are dense, row-major, in device memory (hipMalloc'd or a
 *     torch device tensor); bf16 values are passed as their uint16_t bits.
 *   - X is [M,K] (one row per token), W is [N,K] (one row per output channel,
 *     the torch nn.Linear layout), Y is [M,N].
 *   - The caller owns every buffer.  The library allocates no device memory,
 *     keeps no pointer after returning and holds no mutable state; it is
 *     thread-safe.
 *   - Work is enqueued asynchronously on `stream` (0 = the null stream);
 *     results are valid once that stream has been synchronised.
 *   - Arguments are validated before anything is launched; on any error
 *     nothing is launched and no output byte is written.  Shapes are checked
 *     first: an empty input (M == 0, or N == 0 for the weight quantizer) is
 *     then a no-op that returns W8A8_OK without looking at the pointers.
 *   - Inputs must be finite.  NaN/Inf inputs are outside the contract and not
 *     checked on the hot path.
 *   - Shape contract: 16 <= K, K % 16 == 0; N >= 1; M >= 0.  The GEMM entry
 *     points also require K <= W8A8_MAX_K, the largest K for which a sum of
 *     K products of codes in [-127, 127] cannot overflow int32.
 *   - Alignment contract: X, W, Xq and Wq 16-byte aligned; scales 4-byte
 *     aligned; Y and bias 2-byte aligned; int32 accumulators 4-byte aligned.
 */
#ifndef W8A8_H_
#define W8A8_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* floor((2^31 - 1) / 127^2): sums of this many +-127*127 products fit int32. */
#define W8A8_MAX_K 133144

typedef enum {
  W8A8_OK = 0,
  W8A8_ERR_NULL = 1,   /* a required pointer is NULL */
  W8A8_ERR_SHAPE = 2,  /* M, N or K outside the shape contract */
  W8A8_ERR_ALIGN = 3,  /* a pointer breaks the alignment contract */
  W8A8_ERR_LAUNCH = 4, /* the HIP runtime rejected a launch (wrong device, no device, ...) */
  W8A8_ERR_ARG = 5,    /* any other invalid argument (e.g. an unknown tile id) */
  W8A8_ERR_SCRATCH = 6, /* more scratch than the no-allocation entry point holds */
  /* Not statuses: these two make every int32 value a valid w8a8_status, so
   * that C++ code may hold and compare any value a C caller passes (without
   * them a value outside 0..7 is undefined behaviour in C++). */
  W8A8_STATUS_RANGE_MIN_ = -2147483647 - 1,
  W8A8_STATUS_RANGE_MAX_ = 2147483647
} w8a8_status;

/* Static, NUL-terminated description of a status code. */
const char *w8a8_status_str(w8a8_status s);

/*
 * Per-output-channel weight quantization (offline, once per layer).
 * For each row n of w [N,K] (bf16 bits):
 *   amax = max_k |w[n,k]|,  w_scale[n] = fl32(amax / 127),
 *   wq[n,k] = clamp(rne(fl32(w[n,k] / w_scale[n])), -127, 127),
 * an all-zero row gives w_scale[n] = 0 and wq[n,:] = 0.
 * Abstract: weights are quantized and their per-channel scale is folded into
 * the epilogue.  Outputs: wq int8 [N,K], w_scale fp32 [N].
 */
w8a8_status w8a8_quantize_weight(const uint16_t *w, int64_t N, int64_t K,
                                 int8_t *wq, float *w_scale, hipStream_t stream);

/*
 * Per-token activation quantization (every forward).  Same row rule as
 * w8a8_quantize_weight applied to each row m of x [M,K]:
 * outputs xq int8 [M,K] and x_scale fp32 [M].
 * Abstract: activations are quantized per token.
 */
w8a8_status w8a8_quantize_act(const uint16_t *x, int64_t M, int64_t K,
                              int8_t *xq, float *x_scale, hipStream_t stream);

/*
 * The fp8 variant of the method (OCP e4m3 codes instead of int8; the pages
 * weigh the int8 path against fp8 alternatives, here the same kernels run
 * both on one GPU).  Codes are uint8 bit patterns of e4m3 (1 sign, 4
 * exponent bits with bias 7, 3 mantissa bits; largest value 448).
 *   quantize:  s = fl32(amax / 448), q = e4m3(fl32(v / s)) (nearest, ties to
 *              even, saturating at +-448); an all-zero row gives s = 0, q = 0.
 *   GEMM:      acc[m,n] = sum_k x[m,k] * w[n,k] accumulated in fp32 on the
 *              matrix cores (v_mfma_f32_32x32x64_f8f6f4).  The products are
 *              exact; each instruction adds a block of 64 of them at the
 *              hardware's own internal precision and order, which the ISA
 *              does not document, so the sums are not those of sequential
 *              fp32 additions and carry no bound of the form
 *              gamma_K * sum |x w|.  Checked against exact sums to the same
 *              output tolerance as the int8 path.
 *   linear:    the same epilogue as w8a8_linear on the fp32 accumulators.
 * Same shape, alignment and error contracts as the int8 entry points; the
 * raw entry writes fp32 accumulators.
 */
w8a8_status w8a8_quantize_weight_fp8(const uint16_t *w, int64_t N, int64_t K, uint8_t *wq,
                                     float *w_scale, hipStream_t stream);
w8a8_status w8a8_quantize_act_fp8(const uint16_t *x, int64_t M, int64_t K, uint8_t *xq,
                                  float *x_scale, hipStream_t stream);
w8a8_status w8a8_linear_fp8(const uint8_t *xq, const float *x_scale, const uint8_t *wq,
                            const float *w_scale, const uint16_t *bias, uint16_t *y,
                            int64_t M, int64_t N, int64_t K, hipStream_t stream);
w8a8_status w8a8_linear_fp8_tile(const uint8_t *xq, const float *x_scale, const uint8_t *wq,
                                 const float *w_scale, const uint16_t *bias, uint16_t *y,
                                 int64_t M, int64_t N, int64_t K, int tile, hipStream_t stream);
w8a8_status w8a8_gemm_f32_fp8(const uint8_t *xq, const uint8_t *wq, float *acc,
                              int64_t M, int64_t N, int64_t K, hipStream_t stream);
w8a8_status w8a8_gemm_f32_fp8_tile(const uint8_t *xq, const uint8_t *wq, float *acc,
                                   int64_t M, int64_t N, int64_t K, int tile, hipStream_t stream);

/*
 * Row-wise dequantization back to bf16 (the slow path's first step):
 *   out[r,k] = bf16_rne( fl32( float(q[r,k]) * scale[r] ) )
 * for q int8 [R,K] and scale fp32 [R]; out is bf16 [R,K].
 * Abstract: the shipped int8 forward this work replaces quantizes
 * weights and activations and then immediately dequantizes them to bf16 for a
 * bf16 matrix multiply.  Provided so that path can be measured against the
 * fused GEMM; it is not part of the fused path.  Shape contract as above
 * (16 <= K, K % 16 == 0, R >= 0; R == 0 is a no-op); q and out 16-byte
 * aligned, scale 4-byte aligned.
 */
w8a8_status w8a8_dequantize_rows(const int8_t *q, const float *scale, int64_t R, int64_t K,
                                 uint16_t *out, hipStream_t stream);

/*
 * Fused W8A8 linear: int8 GEMM with the dequant + bias epilogue.
 *   acc[m,n] = sum_k xq[m,k] * wq[n,k]                 (exact, int32)
 *   y[m,n]   = bf16_rne( fl32( fl32( fl32(float(acc[m,n]) * x_scale[m])
 *                                    * w_scale[n] ) + float(bias[n]) ) )
 * Each fp32 operation is rounded separately (no fused multiply-add), so y is
 * a deterministic function of the inputs.  bias may be NULL (treated as 0).
 * Up to 32 tokens go to the kernel of w8a8_linear_dynamic (from codes, no
 * workspace) where it is the faster one, with the same bits; a tile id given to
 * w8a8_linear_tile is always that tile.  So do w8a8_linear_gelu and
 * w8a8_gated_linear.
 * Abstract: int8 x int8 -> int32 on the matrix cores, per-token x per-channel
 * dequantization and bias folded into the epilogue, bf16 out.
 * Inputs xq [M,K], x_scale [M], wq [N,K], w_scale [N], bias [N]; output y [M,N].
 */
w8a8_status w8a8_linear(const int8_t *xq, const float *x_scale, const int8_t *wq,
                        const float *w_scale, const uint16_t *bias, uint16_t *y,
                        int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * Fused W8A8 linear with GELU in the epilogue (the up-projection of a
 * transformer MLP):
 *   y[m,n] = bf16_rne( gelu( fl32 value of w8a8_linear above ) ),
 *   gelu(v) = v * Phi(v) (exact erf definition), evaluated in fp32 with a
 *   relative error below 3e-5 (below 1e-5 where |gelu| > 1e-6).
 * Abstract: the per-token x per-channel dequantization and the bias are
 * folded into the GEMM epilogue; the activation that follows the linear is
 * folded in the same way, so the pre-activation never reaches memory.  Not
 * bit-reproducible against an fp64 GELU: compare with a tolerance.  Same
 * arguments, contracts and errors as w8a8_linear / w8a8_linear_tile.
 */
w8a8_status w8a8_linear_gelu(const int8_t *xq, const float *x_scale, const int8_t *wq,
                             const float *w_scale, const uint16_t *bias, uint16_t *y,
                             int64_t M, int64_t N, int64_t K, hipStream_t stream);
w8a8_status w8a8_linear_gelu_tile(const int8_t *xq, const float *x_scale, const int8_t *wq,
                                  const float *w_scale, const uint16_t *bias, uint16_t *y,
                                  int64_t M, int64_t N, int64_t K, int tile, hipStream_t stream);

/*
 * Diagnostic entry: the same GEMM main loop, storing the raw int32
 * accumulators acc [M,N] instead of running the epilogue.
 * Abstract: the int8 x int8 -> int32 accumulation is checked bit for bit.
 */
w8a8_status w8a8_gemm_i32(const int8_t *xq, const int8_t *wq, int32_t *acc,
                          int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * Per-shape tile selection (the abstract tunes its kernel for each GEMM shape;
 * here a fixed table chosen from measurements).  w8a8_num_tiles() is the number of
 * compiled tile configurations; w8a8_tile_info() describes one (block rows of
 * X, block rows of W, K bytes per stage, threads; any pointer may be NULL);
 * w8a8_select_tile() returns the id w8a8_linear would use for a shape.
 */
int w8a8_num_tiles(void);
w8a8_status w8a8_tile_info(int tile, int *block_m, int *block_n, int *block_k, int *threads);
int w8a8_select_tile(int64_t M, int64_t N, int64_t K);

/*
 * w8a8_linear / w8a8_gemm_i32 with an explicit tile id (tile < 0 selects as
 * the plain entry points do).  Every tile gives bit-identical results; these
 * exist for tests and tile sweeps.  An unknown id returns W8A8_ERR_ARG.
 */
w8a8_status w8a8_linear_tile(const int8_t *xq, const float *x_scale, const int8_t *wq,
                             const float *w_scale, const uint16_t *bias, uint16_t *y,
                             int64_t M, int64_t N, int64_t K, int tile, hipStream_t stream);
w8a8_status w8a8_gemm_i32_tile(const int8_t *xq, const int8_t *wq, int32_t *acc,
                               int64_t M, int64_t N, int64_t K, int tile, hipStream_t stream);

/*
 * K-split fused linear, for shapes whose output tiles are too few to occupy
 * every compute unit (few tokens and a long K, e.g. the down-projection of a
 * transformer MLP over a small batch).  Same result, bit for bit, as
 * w8a8_linear (or w8a8_linear_gelu when `gelu` is non-zero): the K reduction
 * of each output tile is cut into `splits` equal ranges, each range's exact
 * int32 sums are written to the caller's workspace, and a second pass adds
 * the ranges (exactly, in int32) and applies the same fp32 dequantization,
 * bias (and GELU) epilogue, rounded to bf16.
 * Abstract: int8 x int8 -> int32 on the matrix cores, per-token x
 * per-channel dequantization and bias folded into the epilogue; the pages'
 * GEMM is tuned per shape, and splitting K is this library's answer for
 * shapes with few output tiles.
 *   splits <= 0: chosen by the library's cost model (w8a8_select_splitk);
 *   splits == 1: the plain fused path, no workspace needed;
 *   splits > 1: requires N % 8 == 0, K % (16 * splits) == 0 (else
 *                W8A8_ERR_SHAPE), splits <= 64, y and workspace 16-byte
 *                aligned, and workspace_bytes >=
 *                w8a8_linear_splitk_workspace(M, N, splits) (else W8A8_ERR_ARG).
 *   tile < 0: automatic; else a tile id as for w8a8_linear_tile (its main
 *   tiles are used; W8A8_ERR_ARG if unknown).
 * The workspace (device memory the caller owns, splits * M * N int32) is
 * written and read only by this call's kernels, in stream order; calls that
 * share a workspace must be ordered on one stream.
 */
int w8a8_select_splitk(int64_t M, int64_t N, int64_t K, int *tile);
size_t w8a8_linear_splitk_workspace(int64_t M, int64_t N, int splits);
w8a8_status w8a8_linear_splitk(const int8_t *xq, const float *x_scale, const int8_t *wq,
                               const float *w_scale, const uint16_t *bias, uint16_t *y,
                               int64_t M, int64_t N, int64_t K, int splits, int tile, int gelu,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * w8a8_linear_splitk for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments and result without the workspace.  The int32
 * slices live in a library-owned array of W8A8_NOALLOC_SCRATCH_BYTES (32 MiB)
 * in each GPU's memory, held from the library's load until the process ends;
 * its device address is looked up (hipGetSymbolAddress) on the first call on
 * each device, with that device current.  The call allocates nothing.
 * Every call on one GPU uses that GPU's one array: calls that may overlap on
 * one GPU (different streams, or different host threads without ordering)
 * race on it and must be serialized by the caller; calls in order on one
 * stream are safe.  No state carries from one call to the next (each slice
 * element is written before it is read).  A request whose split needs more
 * than W8A8_NOALLOC_SCRATCH_BYTES (splits * M * N * 4 bytes, splits as
 * resolved when `splits` <= 0) returns W8A8_ERR_SCRATCH before anything is
 * launched.  The current device must be the one `stream` belongs to.
 */
#define W8A8_NOALLOC_SCRATCH_BYTES (32 * 1024 * 1024)
w8a8_status w8a8_linear_splitk_noalloc(const int8_t *xq, const float *x_scale, const int8_t *wq,
                                       const float *w_scale, const uint16_t *bias, uint16_t *y,
                                       int64_t M, int64_t N, int64_t K, int splits, int tile,
                                       int gelu, hipStream_t stream);

/*
 * Diagnostic: the throughput ceiling of w8a8_linear's inner loop on this GPU,
 * on the caller's codes.  The int8 matrix cores run at a power-limited clock
 * that depends on the operand values, so the GEMM's rate is best read against
 * what the same instructions sustain on the same data.  This runs the GEMM's
 * K step exactly (the 256x192 tile's eight wavefronts, fragment reads from
 * LDS one K step ahead of the int8 MFMAs) on one 128-byte K stage of xq
 * [M,K] and wq [N,K] per workgroup, staged in LDS once and looped over
 * `iters` times, with no memory traffic, barriers or epilogue in the loop:
 * 256 workgroups of 512 threads, each 49152 * iters MFMAs of
 * 32x32x32 int8 (65536 int8 operations each).  Time it with events on
 * `stream`.
 * Workgroup g takes rows m0 = (g mod floor(M/256)) * 256 of xq,
 * n0 = (floor(g / floor(M/256)) mod floor(N/192)) * 192 of wq and the K stage
 * k0 = (g mod floor(K/128)) * 128; its eight wavefronts write the sums of
 * their int32 accumulators to sink[g*8 .. g*8+7] (int64, device memory,
 * 2048 entries), which add up to iters * sum over k in the stage of
 * (sum of xq[m0..m0+255, k]) * (sum of wq[n0..n0+191, k]).
 * Requires 256 <= M, 192 <= N, 128 <= K <= W8A8_MAX_K, K % 16 == 0 and
 * 1 <= iters <= 2^40; xq, wq 16-byte and sink 8-byte aligned.  Not part of
 * the fused path; it exists so measurements can be put against the chip's
 * power-limited matrix-core rate.
 */
w8a8_status w8a8_mfma_ceiling(const int8_t *xq, const int8_t *wq, int64_t M, int64_t N, int64_t K,
                              int64_t iters, int64_t *sink, hipStream_t stream);

/*
 * The linear from bf16 activations: w8a8_quantize_act and w8a8_linear (or
 * w8a8_linear_gelu when `gelu` is non-zero) in one call, the same bits.  Up to
 * 32 tokens take a kernel that reads the weight once: up to 16 tokens where
 * K >= 768 or N <= 8192 + 16 K, more where K >= 256 and N <= 8 min(K, 2048)
 * (gated: or K >= 4096).  It is one launch that needs no workspace for at most
 * 16 tokens whose codes take at most 22 KB (one token of K = 22272, five of
 * 4096); for larger codes of 9 to 16 tokens the linear takes it only where
 * N <= 40960 or K >= 8192.  Otherwise the codes are made in the workspace first
 * (then the same kernel, the K-split or the tiled kernel, by shape).
 *   x bf16 [M,K] 16-byte aligned; wq [N,K], w_scale [N], bias [N] or NULL;
 *   y bf16 [M,N] 2-byte aligned; workspace of at least
 *   w8a8_linear_dynamic_workspace(M, N, K) bytes, 16-byte aligned (it may be
 *   less, or NULL, where that one launch can do without).  The workspace
 *   belongs to the call until its work on the stream is done: calls that may
 *   overlap need one each.
 */
size_t w8a8_linear_dynamic_workspace(int64_t M, int64_t N, int64_t K);
w8a8_status w8a8_linear_dynamic(const uint16_t *x, const int8_t *wq, const float *w_scale,
                                const uint16_t *bias, uint16_t *y, int64_t M, int64_t N,
                                int64_t K, int gelu, void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/*
 * Gated product, the first half of a gated feed-forward block: both
 * projections, the activation and the product in one kernel.  wq [2N,K] holds
 * the gate's N rows and below them the up projection's; w_scale and bias [2N]
 * likewise (bias may be NULL).
 *   g[m,n] = w8a8_linear's fp32 value for row n, u[m,n] for row N + n,
 *   y[m,n] = bf16_rne( act(g[m,n]) * u[m,n] ),
 *   act 0: SiLU, v / (1 + exp(-v)); act 1: GELU (exact erf definition); both
 *   in fp32 with a relative error below 3e-5 (but zero where the value itself is
 *   next to the smallest fp32 numbers: SiLU below about -87, GELU below about -13).
 * Contracts as for w8a8_linear with 2N in the place of N; `tile` as for
 * w8a8_linear_tile (every tile gives the same bits).  The dynamic form takes
 * bf16 activations as w8a8_linear_dynamic does, with the same bits as
 * w8a8_quantize_act and w8a8_gated_linear.
 */
#define W8A8_ACT_SILU 0
#define W8A8_ACT_GELU 1
w8a8_status w8a8_gated_linear(const int8_t *xq, const float *x_scale, const int8_t *wq,
                              const float *w_scale, const uint16_t *bias, uint16_t *y,
                              int64_t M, int64_t N, int64_t K, int act, hipStream_t stream);
w8a8_status w8a8_gated_linear_tile(const int8_t *xq, const float *x_scale, const int8_t *wq,
                                   const float *w_scale, const uint16_t *bias, uint16_t *y,
                                   int64_t M, int64_t N, int64_t K, int act, int tile,
                                   hipStream_t stream);
size_t w8a8_gated_linear_dynamic_workspace(int64_t M, int64_t N, int64_t K);
w8a8_status w8a8_gated_linear_dynamic(const uint16_t *x, const int8_t *wq, const float *w_scale,
                                      const uint16_t *bias, uint16_t *y, int64_t M, int64_t N,
                                      int64_t K, int act, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of w8a8_linear for dy bf16 [M,N], the rounding to codes passed
 * straight through:
 *   dx[m,k]  = bf16( sum_n dy[m,n] * w[n,k] ),  w = wq * w_scale,
 *   dw[n,k]  = bf16( sum_m dy[m,n] * x[m,k] ),  x = xq * x_scale,
 *   dbias[n] = bf16( sum_m dy[m,n] ).
 * Each output is bf16 and is left out where its pointer is NULL; dx needs wq
 * and w_scale, dw needs xq and x_scale.  Sums are fp32 (bf16 matrix cores);
 * the values w and x are rounded to bf16 once before their products (for up to
 * 64 tokens of a large weight and 16-byte aligned dx, dy * w_scale in the place
 * of w; the codes are then exact), which leaves an rms error of about 1.4 times
 * that of the outputs' own rounding.  Results do not depend on timing (no
 * atomics).
 * The gated form has wq [2N,K], w_scale, bias and dbias [2N] and dw [2N,K] as
 * w8a8_gated_linear; it needs all of xq, x_scale, wq, w_scale and the
 * forward's bias, forms g and u again from them, and
 *   dg = dy * u * act'(g),  du = dy * act(g)   (fp32; for the products rounded
 *   to bf16 once, with the scale of the other operand, whose codes are exact).
 * Without tokens (M = 0) dw and dbias are set to zeros.
 * Limits (W8A8_ERR_SHAPE): N at most 2^21 for dx, gated N at most 2^20 for any
 * output, M at most 2^21 for dw.  dy, bias and outputs 2-byte aligned
 * (dy is copied where it is not 16-byte aligned, N % 8 != 0, or a long product
 * of N % 64 != 0 repays it).  The workspace as above.
 */
size_t w8a8_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int dx, int dw, int dbias);
w8a8_status w8a8_linear_backward(const uint16_t *dy, const int8_t *xq, const float *x_scale,
                                 const int8_t *wq, const float *w_scale, uint16_t *dx,
                                 uint16_t *dw, uint16_t *dbias, int64_t M, int64_t N, int64_t K,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t w8a8_gated_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int dx, int dw,
                                            int dbias);
w8a8_status w8a8_gated_linear_backward(const uint16_t *dy, const int8_t *xq,
                                       const float *x_scale, const int8_t *wq,
                                       const float *w_scale, const uint16_t *bias, uint16_t *dx,
                                       uint16_t *dw, uint16_t *dbias, int64_t M, int64_t N,
                                       int64_t K, int act, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/*
 * RMS norm of each head of the queries and keys and the position rotation, in
 * one pass over the output of a QKV linear.  q is [M,Hq,D], k [M,Hk,D] (bf16;
 * element (m,h,d) at m * row + h * head + d, so both may lie in one packed
 * QKV matrix).  For each head vector x:
 *   n = x / sqrt(mean(x^2) + eps) * weight          (weight NULL: ones)
 *   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first `rot`
 *   values: (n[i], n[i + rot/2]) or, `interleaved` non-zero, (n[2i], n[2i+1]),
 *   with cos, sin fp32 [P, rot/2] of the row's position (positions int32 [M],
 *   or NULL: m mod P, one sequence of P tokens after another).
 * Arithmetic in fp32, rounded to bf16 once.  A row whose position is outside
 * [0, P) (padding) gets zeros in every head, and in the gradients, and adds
 * nothing to the weights' gradients, also where rot = 0 (the norm alone; P is
 * then looked at only where positions are given).  q_out and k_out may be q and
 * k (same strides) and overlap nothing otherwise, nor each other; Hq or Hk may
 * be 0 (its pointers are then not looked at).
 * The gradient takes the outputs' gradients dq, dk and the inputs q, k, and
 * writes dq_in, dk_in (bf16; they may be dq, dk or q, k with the same strides)
 * and, where not NULL, dq_weight, dk_weight (fp32 [D], summed over rows and
 * heads in a fixed order; they need the workspace).
 * Contract: 16 <= D <= 1024, D and rot multiples of 16, 0 <= rot <= D,
 * M * (Hq + Hk) * (D/16 rounded up to a power of two) <= 2^31, 1 <= P < 2^31,
 * eps >= 0; all bf16 and table pointers 16-byte aligned, strides multiples of
 * 8, weight gradients and positions 4-byte aligned.
 */
w8a8_status w8a8_qk_norm_rope(const uint16_t *q, int64_t q_row, int64_t q_head,
                              const uint16_t *k, int64_t k_row, int64_t k_head,
                              const uint16_t *q_weight, const uint16_t *k_weight,
                              const float *cos, const float *sin, const int32_t *positions,
                              uint16_t *q_out, int64_t q_out_row, int64_t q_out_head,
                              uint16_t *k_out, int64_t k_out_row, int64_t k_out_head,
                              int64_t M, int64_t P, int64_t Hq, int64_t Hk, int64_t D,
                              int64_t rot, float eps, int interleaved, hipStream_t stream);
size_t w8a8_qk_norm_rope_backward_workspace(int64_t M, int64_t Hq, int64_t Hk, int64_t D);
w8a8_status w8a8_qk_norm_rope_backward(
    const uint16_t *dq, int64_t dq_row, int64_t dq_head, const uint16_t *dk, int64_t dk_row,
    int64_t dk_head, const uint16_t *q, int64_t q_row, int64_t q_head, const uint16_t *k,
    int64_t k_row, int64_t k_head, const uint16_t *q_weight, const uint16_t *k_weight,
    const float *cos, const float *sin, const int32_t *positions, uint16_t *dq_in,
    int64_t dq_in_row, int64_t dq_in_head, uint16_t *dk_in, int64_t dk_in_row,
    int64_t dk_in_head, float *dq_weight, float *dk_weight, int64_t M, int64_t P, int64_t Hq,
    int64_t Hk, int64_t D, int64_t rot, float eps, int interleaved, void *workspace,
    size_t workspace_bytes, hipStream_t stream);

/*
 * The residual's addition, the root-mean-square norm of each row and its
 * quantization in one pass, in front of a linear.  For rows of K values:
 *   h = bf16(x + residual)                     (residual NULL: h = x),
 *   v = fl32(h * weight)                       (weight NULL: ones),
 *   s = fl32(max|v| * fl32(1 / 127)), xq = rne(fl32(v / s)) in [-127, 127]
 *   (fp8 non-zero: 1 / 448 and e4m3 codes, nearest, ties to even),
 *   x_scale = fl32(s / sqrt(mean(h^2) + eps)),
 * so xq * x_scale is the normed row on the codes' grid: the norm's factor is
 * common to a row, cancels in the codes and goes into the scale.  (s is a
 * product, not w8a8_quantize_act's quotient max|v| / 127: it may be a step of
 * fp32 away from that.)  Codes are exact functions of the inputs; mean(h^2) is
 * a sum in fp32.  A row whose s is zero (all zeros) has zero codes and scale; one
 * with a NaN or an infinity in h or in h * weight has a scale that is not finite,
 * and so has every output that is made of its codes.
 * h is written where it is not NULL; it may be x or residual and overlaps
 * nothing otherwise, and no other output overlaps anything.
 * The gradient, the rounding to codes passed straight through, for dn (of the
 * normed row) and dh (of h, from what else reads it; may be NULL):
 *   r = 1 / sqrt(mean(h^2) + eps), hh = h r,
 *   dx = bf16( dh + r (dn weight - hh mean(dn weight hh)) )  (x and residual),
 *   dweight = sum over rows of dn hh, fp32, in a fixed order (may be NULL; it
 *   needs the workspace; zeros without rows).
 * dx may be dn, dh or h and overlaps nothing otherwise.  Arithmetic is fp32, each bf16
 * output rounded once.  Of a row of zeros with eps = 0, r is taken as 0.
 * Contract: 16 <= K <= 32768, K % 16 == 0; M times 64 (K <= 1024), 256 (K <
 * 8192) or 1024 below 2^32 - 1024, M <= 2^26; eps >= 0; h of any magnitude
 * (squares that vanish or overflow in fp32 are summed again in range) whose
 * products with the weight, and of the gradient dn * weight * h, are finite in
 * fp32; all bf16 pointers and the codes 16-byte aligned, scales and dweight 4-byte
 * aligned.
 */
w8a8_status w8a8_add_rms_norm_quantize(const uint16_t *x, const uint16_t *residual,
                                       const uint16_t *weight, uint16_t *h, void *xq,
                                       float *x_scale, int64_t M, int64_t K, float eps, int fp8,
                                       hipStream_t stream);
size_t w8a8_add_rms_norm_backward_workspace(int64_t M, int64_t K);
w8a8_status w8a8_add_rms_norm_backward(const uint16_t *dn, const uint16_t *dh, const uint16_t *h,
                                       const uint16_t *weight, uint16_t *dx, float *dweight,
                                       int64_t M, int64_t K, float eps, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/*
 * The linear with a low-rank adapter for each token, of a set of L adapters of
 * rank R that share the weight: a bf16 [L,R,K], b bf16 [L,N,R], scaling fp32
 * [L], ids int32 [M] (the token's adapter; outside [0, L): none).  With
 * i = ids[m] and x = xq * x_scale:
 *   t[m,r] = bf16( scaling[i] * sum_k x[m,k] * a[i][r,k] ),
 *   y[m,n] = bf16( v + sum_r t[m,r] * b[i][n,r] ),  v the fp32 value of w8a8_linear.
 * Sums are fp32; t is rounded because it is an operand of the bf16 matrix
 * cores.  A token without an adapter has the bits of w8a8_linear, and no
 * token's result depends on another adapter's values (be they NaN) or on its
 * neighbours (on their number alone, which may choose another kernel); a value of
 * b that is not finite reaches its channel of its adapter's tokens alone, whichever
 * kernel runs.  Adapters of different ranks are padded with zeros.  Any order of ids
 * is right; long runs of tokens with the same adapter are the fast one.
 * The dynamic form takes bf16 activations, with the same bits as
 * w8a8_quantize_act and w8a8_linear_adapters: one launch for up to four short
 * tokens, two for a few tokens, three or four beyond and for rows of over 16384
 * values.
 * Contract as for w8a8_linear, and 8 <= R <= 128, R % 8 == 0, 1 <= L <= 65536;
 * a and b 16-byte aligned, scaling and ids 4-byte aligned.  Workspace as for
 * w8a8_linear_dynamic (always needed).  `tile` as for w8a8_linear_tile, for
 * tests and sweeps: every tile gives the same bits as each other (a few tokens'
 * kernel and the K split, which tile < 0 may choose, sum the adapters' products
 * in another order).
 */
size_t w8a8_linear_adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int dynamic);
w8a8_status w8a8_linear_adapters(const int8_t *xq, const float *x_scale, const int8_t *wq,
                                 const float *w_scale, const uint16_t *bias, const uint16_t *a,
                                 const uint16_t *b, const float *scaling, const int32_t *ids,
                                 uint16_t *y, int64_t M, int64_t N, int64_t K, int64_t R,
                                 int64_t L, int tile, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);
w8a8_status w8a8_linear_adapters_dynamic(const uint16_t *x, const int8_t *wq,
                                         const float *w_scale, const uint16_t *bias,
                                         const uint16_t *a, const uint16_t *b,
                                         const float *scaling, const int32_t *ids, uint16_t *y,
                                         int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                                         void *workspace, size_t workspace_bytes,
                                         hipStream_t stream);

/*
 * Gradients of w8a8_linear_adapters for dy bf16 [M,N], on frozen codes of the
 * weight, the rounding of the activations to codes passed straight through.
 * With i = ids[m], x and t as above and
 *   u[m,r] = scaling[i] * sum_n dy[m,n] * b[i][n,r]:
 *   dx[m,k]    = bf16( sum_n dy[m,n] * w[n,k] + sum_r u[m,r] * a[i][r,k] ),
 *   da[i][r,k] = bf16( sum over the adapter's tokens of u[m,r] * x[m,k] ),
 *   db[i][n,r] = bf16( sum over the adapter's tokens of dy[m,n] * t[m,r] ),
 * bf16 [M,K], [L,R,K] and [L,N,R]; an adapter without tokens gets zeros.  Each
 * is left out where its pointer is NULL; dx needs wq, w_scale, a and b, da needs
 * b, xq and x_scale, db needs a, xq and x_scale.  Sums are fp32.  Of dx, u and
 * w are rounded to bf16 once; da and db take u (times x's scale) and t to 2^-16, so
 * that their own rounding is the only one that is seen.  No atomics, the same bits
 * from call to call.  Contract as for w8a8_linear_adapters and
 * w8a8_linear_backward; da and db 16-byte aligned; those of w, a and b that are
 * needed in another order (for dx all, for da b) have under 2^24 tiles of 64 by 64
 * values, each adapter's counted by themselves (else W8A8_ERR_SHAPE, workspace 0).
 */
size_t w8a8_linear_adapters_backward_workspace(int64_t M, int64_t N, int64_t K, int64_t R,
                                               int64_t L, int dx, int da, int db);
w8a8_status w8a8_linear_adapters_backward(const uint16_t *dy, const int8_t *xq,
                                          const float *x_scale, const int8_t *wq,
                                          const float *w_scale, const uint16_t *a,
                                          const uint16_t *b, const float *scaling,
                                          const int32_t *ids, uint16_t *dx, uint16_t *da,
                                          uint16_t *db, int64_t M, int64_t N, int64_t K, int64_t R,
                                          int64_t L, void *workspace, size_t workspace_bytes,
                                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H_ */
