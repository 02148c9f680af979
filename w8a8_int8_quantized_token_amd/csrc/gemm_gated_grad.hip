// Gradients of the gated product's two values on the kernel of gemm_kernel.h:
// g and u are formed again from the codes (exactly the forward's), and the
// epilogue turns them and dy into
//   dg = dy * u * act'(g),  du = dy * act(g)
// in fp32, written as the first operands of the input's and the weight's
// gradients (scaled, rounded to bf16 once) and as column sums (fp32) for the
// bias's.  The products themselves never reach memory.
//
// Bound by its epilogue as much as by the matrix cores: 2 bytes in and 8 out
// per channel and token besides 4K operations.  4096 x 8192 x 2048, all
// outputs: 195 to 213 us (264 before the loads of dy ran ahead of the stores, the
// stores were whole 64-byte pieces and the sums went through DPP), of which
// the same product with the forward's epilogue is 134 and the 335 MB at the
// rate of a large copy 62.  Matrix pipes busy 0.33 of the cycles, 350 MB read and
// 300 written.
#include "gemm_kernel.h"

namespace w8a8 {
namespace {

// The tiles compiled for it, cheapest by the cost of launch_cost(): the split
// rings are left out (their epilogue spills or was slower at every size
// first measured: 4096 x 8192 x 2048 with all outputs, 256x256 whole ring 264
// us, split 275, 256x192 293).
constexpr int kGradCfgs[] = {kWhole256, kTail128x256, k128, k64};

int grad_cfg(int64_t M, int64_t N, int64_t K) {
  int best = kWhole256;
  double cost = launch_cost(best, M, 2 * N, K);
  for (const int c : kGradCfgs) {
    const double x = launch_cost(c, M, 2 * N, K);
    if (x < cost * 0.999) best = c, cost = x;
  }
  return best;
}

int wave_rows(int cfg) {
  return cfg == kWhole256 ? CfgWhole::TM : cfg == kTail128x256 ? CfgTail::TM : cfg == k128 ? Cfg128::TM : Cfg64::TM;
}

template <Epilogue EPI, int kWant>
hipError_t launch_want(int cfg, const Operands<EPI>& o, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  using Op = OpI8Want<kWant>;
  const KSplit whole{(int)K, 1, 0};
  switch (cfg) {
    case kWhole256: return launch_t<CfgWhole, Op, EPI>(o, M, N, K, N, s, whole);
    case kTail128x256: return launch_t<CfgTail, Op, EPI>(o, M, N, K, N, s, whole);
    case k128: return launch_t<Cfg128, Op, EPI>(o, M, N, K, N, s, whole);
    default: return launch_t<Cfg64, Op, EPI>(o, M, N, K, N, s, whole);
  }
}

template <Epilogue EPI>
hipError_t launch_epi(int cfg, const Operands<EPI>& o, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  switch ((o.extra.p ? kWantP : 0) | (o.extra.qt ? kWantQ : 0) | (o.extra.dbp ? kWantSums : 0)) {
    case 1: return launch_want<EPI, 1>(cfg, o, M, N, K, s);
    case 2: return launch_want<EPI, 2>(cfg, o, M, N, K, s);
    case 3: return launch_want<EPI, 3>(cfg, o, M, N, K, s);
    case 4: return launch_want<EPI, 4>(cfg, o, M, N, K, s);
    case 5: return launch_want<EPI, 5>(cfg, o, M, N, K, s);
    case 6: return launch_want<EPI, 6>(cfg, o, M, N, K, s);
    case 7: return launch_want<EPI, 7>(cfg, o, M, N, K, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

int64_t gated_grad_sum_rows(int64_t M, int64_t N, int64_t K) {
  const int c = grad_cfg(M, N, K);
  const int64_t bm = kCfgs[c].block_m;
  return (M + bm - 1) / bm * (bm / wave_rows(c));
}

hipError_t launch_gated_grad(GateAct act, const uint16_t* dy, int64_t ld_dy, const int8_t* xq, const float* sx,
                             const int8_t* wq, const float* sw, const uint16_t* bias, uint16_t* p,
                             int64_t ldp, uint16_t* qt, int64_t ldq, float* sums, int64_t M,
                             int64_t N, int64_t K, hipStream_t stream) {
  GradArgs a;
  a.w = wq + N * K;
  a.sw = sw + N;
  a.bias = bias ? bias + N : nullptr;
  a.dy = dy;
  a.ld_dy = (int)ld_dy;
  a.p = p;
  a.ldp = (int)ldp;
  a.qt = qt;
  a.ldq = (int)ldq;
  a.dbp = sums;
  const int c = grad_cfg(M, N, K);
  if (act == GateAct::kGelu)
    return launch_epi<Epilogue::kGeluGateGrad>(c, {xq, wq, sx, sw, bias, nullptr, a}, M, N, K, stream);
  return launch_epi<Epilogue::kSiluGateGrad>(c, {xq, wq, sx, sw, bias, nullptr, a}, M, N, K, stream);
}

}  // namespace w8a8
