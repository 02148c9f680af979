// The gated product on the kernel of gemm_kernel.h: for codes xq [M,K] and the
// stacked weight [gate; up] wq [2N,K],
//   g = ((acc_gate*sx)*sw)+b,  u = ((acc_up*sx)*sw)+b,  y = bf16(act(g) * u)
// in one launch.  The int8 main loop is the linear's; W's LDS rows alternate
// 16 gate and 16 up rows of the same channels, so that a lane holds both
// values of a channel and neither product leaves the registers.
//
// Bound by the matrix cores at many tokens (4MNK operations against
// MK + 2NK + 2MN bytes): 8192 x 12288 x 4096 675 to 730 us, 2.3 to 2.4 POPS at
// the package's power limit (1.67 GHz, matrix pipes busy 0.66 of the cycles), where
// the linear of the same 24576 rows takes 820 us for its twice as many outputs.
// Tiles by the linear's cost model for 2N channels, which counts one workgroup per
// compute unit; the smaller tiles have two or three here, so for a few hundred
// tokens its rounds are too many.
#include "gemm_kernel.h"

namespace w8a8 {

hipError_t launch_gated(int tile, GateAct act, const int8_t* xq, const float* sx, const int8_t* wq,
                        const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                        int64_t K, hipStream_t stream) {
  const UpArgs up{wq + N * K, sw + N, bias ? bias + N : nullptr};
  if (tile < 0) tile = choose_tile(M, 2 * N, K);
  if (act == GateAct::kGelu)
    return launch_plan<OpI8, Epilogue::kGeluGate>(tile, {xq, wq, sx, sw, bias, y, up}, M, N, K, stream);
  return launch_plan<OpI8, Epilogue::kSiluGate>(tile, {xq, wq, sx, sw, bias, y, up}, M, N, K, stream);
}

}  // namespace w8a8
