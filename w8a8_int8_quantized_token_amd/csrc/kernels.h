// Internal launch interface between the C-ABI layer and the HIP kernels of
// libw8a8 (gfx950).  Not installed; the public ABI is include/w8a8.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {

// Row-wise absmax quantizer: rows of x [R,K] (bf16 bits) -> q int8 [R,K] and
// scale fp32 [R].  Requires K % 16 == 0 and R > 0.
hipError_t launch_quantize_rows(const uint16_t* x, int8_t* q, float* scale,
                                int64_t R, int64_t K, hipStream_t stream);

// The same with e4m3 codes: scale fl32(amax/448), q = e4m3(fl32(x/scale)).
hipError_t launch_quantize_rows_fp8(const uint16_t* x, uint8_t* q, float* scale, int64_t R,
                                    int64_t K, hipStream_t stream);

// Row-wise dequantization: out[r,k] = bf16(fl32(float(q[r,k]) * scale[r])),
// q int8 [R,K] -> out bf16 bits [R,K].  Requires K % 16 == 0 and R > 0.
hipError_t launch_dequantize_rows(const int8_t* q, const float* scale, uint16_t* out, int64_t R,
                                  int64_t K, hipStream_t stream);

// One compiled GEMM tile configuration.
struct TileDesc {
  int block_m;   // rows of X (tokens) per workgroup
  int block_n;   // rows of W (output channels) per workgroup
  int block_k;   // K bytes staged per pipeline step
  int threads;   // workgroup size
};

int num_tiles();
const TileDesc& tile_desc(int tile);
int select_tile(int64_t M, int64_t N, int64_t K);
// K ranges (1 = no split) and plan the split cost model picks for a shape.
int select_splitk(int64_t M, int64_t N, int64_t K, int* tile);

// kBf16ScaleBias: y = bf16(((acc*sx)*sw)+b); kBf16GeluScaleBias: the same
// value through GELU before the bf16 rounding; kRawI32: the accumulators;
// kBf16Plain: the accumulators rounded to bf16.
// Gated (two products, gate and up, with values g and u as above):
// k*Gate: y = bf16(act(g) * u); k*GateGrad: the gradients of g and u.
enum class Epilogue {
  kBf16ScaleBias, kBf16GeluScaleBias, kRawI32, kBf16Plain,
  kSiluGate, kGeluGate, kSiluGateGrad, kGeluGateGrad
};

// int8 GEMM acc[m,n] = sum_k xq[m,k] * wq[n,k] with the chosen epilogue.
// For the bf16 epilogues `out` is bf16 [M,N] and sx/sw/bias are used (bias
// may be null); for kRawI32 `out` is int32 [M,N].  Shapes already validated.
hipError_t launch_gemm(int tile, Epilogue epi, const int8_t* xq, const int8_t* wq,
                       const float* sx, const float* sw, const uint16_t* bias, void* out,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream);

// K-split int8 GEMM: the main tiles of plan `tile` over `chunks` equal K
// ranges (K % (16 * chunks) == 0), each range's raw int32 sums into its own
// slice partials[c * M * N + m * N + n] (exact; the slices add up to acc).
hipError_t launch_gemm_partials(int tile, const int8_t* xq, const int8_t* wq, int32_t* partials,
                                int64_t M, int64_t N, int64_t K, int chunks, hipStream_t stream);

// Sum of the K-split slices plus the bf16 epilogue (kBf16ScaleBias or
// kBf16GeluScaleBias): y[m,n] from acc = sum_c partials[c][m][n], exactly as
// the fused GEMM's epilogue evaluates it.  Requires N % 8 == 0.
hipError_t launch_splitk_reduce(Epilogue epi, const int32_t* partials, int chunks, const float* sx,
                                const float* sw, const uint16_t* bias, uint16_t* y, int64_t M,
                                int64_t N, hipStream_t stream);

// The fp8 (e4m3) variant: the same tiles and epilogues on
// v_mfma_f32_32x32x64_f8f6f4; for kRawI32 `out` receives the fp32
// accumulators' bits.
hipError_t launch_gemm_fp8(int tile, Epilogue epi, const uint8_t* xq, const uint8_t* wq,
                           const float* sx, const float* sw, const uint16_t* bias, void* out,
                           int64_t M, int64_t N, int64_t K, hipStream_t stream);

// Diagnostic: the fused GEMM's K-step (256x192 tile, eight wavefronts) looped
// `iters` times over one LDS-resident K stage of xq [M,K] and wq [N,K] per
// workgroup, with no memory traffic in the loop; sink int64
// [kCeilingWorkgroups * 8] receives each wavefront's accumulator sum.
// Requires M >= 256, N >= 192, K >= 128 (shapes already validated).
constexpr int kCeilingWorkgroups = 256;
hipError_t launch_mfma_ceiling(const int8_t* xq, const int8_t* wq, int64_t M, int64_t N, int64_t K,
                               int64_t iters, int64_t* sink, hipStream_t stream);

// Activation of a gated product's gate.
enum class GateAct { kSilu = 0, kGelu = 1 };

// The gated int8 product: wq [2N,K] holds the gate's rows and below them the
// up projection's, sw and bias [2N] likewise; y bf16 [M,N] = act(g) * u.
// tile < 0 chooses.
hipError_t launch_gated(int tile, GateAct act, const int8_t* xq, const float* sx, const int8_t* wq,
                        const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                        int64_t K, hipStream_t stream);

// Gradients dg, du of the gated product's two values for dy bf16 [M,ld_dy]
// (rows 16-byte aligned; columns past N zeros or, N % 8 == 0, none), each
// output as far as not null: p bf16 [M,ldp] (columns in blocks of 32: dg *
// sw_gate of 16 channels, du * sw_up of the same, zeros past channel N; ldp =
// 2N rounded up to 64), qt bf16 [2N,ldq] ((dg * sx)^T over (du * sx)^T,
// zeros past column M; ldq = M rounded up to 64), sums fp32
// [gated_grad_sum_rows(), 2N] (column sums over blocks of rows).
int64_t gated_grad_sum_rows(int64_t M, int64_t N, int64_t K);
hipError_t launch_gated_grad(GateAct act, const uint16_t* dy, int64_t ld_dy, const int8_t* xq, const float* sx,
                             const int8_t* wq, const float* sw, const uint16_t* bias, uint16_t* p,
                             int64_t ldp, uint16_t* qt, int64_t ldq, float* sums, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream);

// out bf16 [M,N] = a [M,Kpad] * b [N,Kpad]^T, bf16 with fp32 sums; N and Kpad
// multiples of 8, rows 16-byte aligned.  The sum is cut into gemm_bf16_slices()
// ranges; where they are more than one, their fp32 sums go to slices [ranges,
// M, N] for a JoinJob (out must then be 16-byte aligned) and out is not
// written; with slices null the product is made whole.
int gemm_bf16_slices(int64_t M, int64_t N, int64_t Kpad);
hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* out, float* slices, int64_t M,
                            int64_t N, int64_t Kpad, hipStream_t stream);

// Operand layout of the backward products and the joins after them (see
// backward_layout.hip): one launch each for up to kMaxJobs jobs.
constexpr int kMaxJobs = 4;
struct LayoutJob {
  enum Kind { kTurnCodes, kTurnPaired, kTurnValues, kPadRows } kind;
  const void* in;        // [R,C]: int8 codes or bf16 values
  const float* scale;    // codes: [R] or null
  uint16_t* out;         // [C,ld] (kPadRows: [R,ld])
  float* sums;           // kTurnValues: [ceil(R / span), C] or null
  int64_t R, C, ld, span;
};
struct JoinJob {
  const float* part;     // [P, n]
  uint16_t* out;         // [n]
  int64_t P, n;
  bool slices;           // few long rows (a product's slices, n % 8 == 0), or many short ones
  int64_t blocks;        // set by the launch
};
// The input's gradient of few tokens from the codes as they are: fp32 slices
// [few_grad_slices()][M][K] for launch_finish to join.  d is dy [M,N] (any
// address; `scale` that of the rows of q), or gated launch_gated_grad's p.
constexpr int64_t kFewGradTokens = 64;
int few_grad_slices(int64_t M, int64_t N, int64_t K, bool gated);
hipError_t launch_few_grad(const uint16_t* d, int64_t ldd, const int8_t* q, const float* scale, float* slices,
                           int64_t M, int64_t N, int64_t K, bool gated, hipStream_t stream);
int64_t transpose_sum_span(int64_t R, int64_t C);   // kTurnValues' rows of one block of sums
hipError_t launch_prepare(const LayoutJob* jobs, int n, hipStream_t stream);
hipError_t launch_finish(const JoinJob* jobs, int n, hipStream_t stream);
hipError_t launch_zero(void* p, int64_t halves, hipStream_t stream);   // 16-bit zeros

// The linear (act: 0 none, 1 GELU) or gated pair (act: a GateAct) for at most
// kFewTokens tokens, from bf16 x, or from codes and scales where those are
// given (xq not null; needed where few_tokens_in_lds() says no).
constexpr int64_t kFewTokens = 32;
bool few_tokens_in_lds(int64_t M, int64_t K);
hipError_t launch_few_tokens(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq,
                             const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, int act, bool gated, hipStream_t stream);

// Queries or keys [M, heads, D]: element (m, h, d) at p[m * row + h * head + d].
struct RopeView {
  uint16_t* p;
  int64_t row, head;
};
struct RopeArgs {
  RopeView q, k;     // inputs
  RopeView qo, ko;   // forward: outputs; gradient: the outputs' gradients
  const uint16_t *qw, *kw;      // norm weights bf16 [D], or null
  const float *cos, *sin;       // [P, rot / 2]
  const int32_t* positions;     // [M], or null: row m has position m % P
  int64_t M, P;
  int Hq, Hk, D, rot;
  float eps;
};
hipError_t launch_norm_rope(const RopeArgs& a, bool interleaved, hipStream_t stream);
// part fp32 [norm_rope_grad_rows(), D] (null: no weight gradients).
int64_t norm_rope_grad_rows(int64_t M, int64_t Hq, int64_t Hk, int D);
hipError_t launch_norm_rope_grad(const RopeArgs& a, const RopeView& dq, const RopeView& dk, bool interleaved,
                                 float* part, float* dqw, float* dkw, hipStream_t stream);

}  // namespace w8a8
