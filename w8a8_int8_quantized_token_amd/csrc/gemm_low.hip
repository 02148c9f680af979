// The int8 linear with low-rank adapters on the kernel of gemm_kernel.h:
//   y = bf16(((acc*sx)*sw)+b + sum_r t[m,r] b[id(m)][n,r]).
// The second product is an epilogue (add_low): the sums are in fp32 before the
// only rounding, and y is written once.  Bound by the int8 product; its passes,
// one for each 16 ranks of each adapter that a wavefront's tokens have, come on
// top (us, this kernel / the linear): 8192 x 12288 x 4096 in runs of 512 tokens,
// rank 16 409 / 382, rank 64 438 / 367; 2048 x 4096 x 4096, sixteen adapters in runs,
// rank 16 39.5 / 39.7, rank 64 42.9 / 39.5, mixed 43.7 / 39.2 and 74.8 / 39.4.
#include "gemm_kernel.h"

namespace w8a8 {

hipError_t launch_gemm_low(int tile, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                           const uint16_t* bias, const Low& low, uint16_t* y, int64_t M, int64_t N, int64_t K,
                           hipStream_t stream) {
  const LowArgs args{low.t, low.b, low.ids, N * low.R, (int)low.ldt, (int)low.R, (int)low.count};
  if (tile < 0) {
    tile = choose_tile(M, N, K);
    // the 128x256 tiles where the linear takes 256x128 ones (us, 256x128 / 128x256, of
    // adapters in runs and mixed: 2048 x 4096 x 4096, rank 16 55.8 / 51.6 and 65.8 / 59.9,
    // rank 64 58.9 / 54.8 and 97 / 100; 1024 x 8192 x 4096 52.8 / 48.6 and 54.0 / 49.8; 4096
    // x 2048 x 2048 38.2 / 34.7 and 40.3 / 36.4; 1536 x 5120 x 5120 65.6 / 59.3 and 69.9 / 63.2)
    if (kPlans[tile].main == k256x128) --tile;
  }
  // the plans of the 256x256 split ring are those of its whole-stage form here
  if (tile < kNumPlans && kPlans[tile].main == kSplit256) tile += 2;
  static_assert(kPlans[2].main == kWhole256 && kPlans[3].main == kWhole256 && kPlans[2].tail == kPlans[0].tail &&
                    kPlans[3].tail == kPlans[1].tail && kPlans[5].main == kTail128x256 && kPlans[6].main == k256x128,
                "the order of the plans");
  return launch_plan<OpI8, Epilogue::kBf16ScaleBiasLow>(tile, {xq, wq, sx, sw, bias, y, args}, M, N, K, stream);
}

}  // namespace w8a8
