// Gradients of the gated product's two values on the kernel of gemm_kernel.h:
// g and u are formed again from the codes (exactly the forward's), and the
// epilogue turns them and dy into
//   dg = dy * u * act'(g),  du = dy * act(g)
// in fp32, written as the first operands of the input's and the weight's
// gradients (scaled, rounded to bf16 once) and as column sums (fp32) for the
// bias's.  The products themselves never reach memory.
#include "gemm_kernel.h"

namespace w8a8 {
namespace {

// One launch on one tile size: the partial sums' rows belong to it.
int grad_cfg(int64_t M, int64_t N, int64_t K) {
  int best = k192;
  double cost = launch_cost(k192, M, 2 * N, K);
  for (int c = 0; c < kNumCfg; ++c) {
    const double x = launch_cost(c, M, 2 * N, K);
    if (x < cost * 0.999) best = c, cost = x;
  }
  return best;
}

// Rows of a wavefront in each configuration.
template <class T>
constexpr int wave_rows() { return T::TM; }
constexpr int kWaveRows[kNumCfg] = {wave_rows<CfgSplit>(), wave_rows<CfgWhole>(), wave_rows<Cfg192>(),
                                    wave_rows<CfgTail>(), wave_rows<Cfg256x128>(), wave_rows<Cfg128>(),
                                    wave_rows<Cfg64>()};

}  // namespace

int64_t gated_grad_sum_rows(int64_t M, int64_t N, int64_t K) {
  const int c = grad_cfg(M, N, K);
  const int64_t bm = kCfgs[c].block_m;
  return (M + bm - 1) / bm * (bm / kWaveRows[c]);
}

hipError_t launch_gated_grad(GateAct act, const uint16_t* dy, const int8_t* xq, const float* sx,
                             const int8_t* wq, const float* sw, const uint16_t* bias, uint16_t* p,
                             int64_t ldp, uint16_t* qt, int64_t ldq, float* sums, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream) {
  GradArgs a;
  a.w = wq + N * K;
  a.sw = sw + N;
  a.bias = bias ? bias + N : nullptr;
  a.dy = dy;
  a.dy_vec = N % 8 == 0 && reinterpret_cast<uintptr_t>(dy) % 16 == 0;
  a.p = p;
  a.ldp = (int)ldp;
  a.p_up = (int)(ldp / 2);
  a.qt = qt;
  a.ldq = (int)ldq;
  a.dbp = sums;
  const int c = grad_cfg(M, N, K);
  const KSplit whole{(int)K, 1, 0};
  if (act == GateAct::kGelu)
    return launch_cfg<OpI8, Epilogue::kGeluGateGrad>(c, {xq, wq, sx, sw, bias, nullptr, a}, M, N, K, N, stream, whole);
  return launch_cfg<OpI8, Epilogue::kSiluGateGrad>(c, {xq, wq, sx, sw, bias, nullptr, a}, M, N, K, N, stream, whole);
}

}  // namespace w8a8
