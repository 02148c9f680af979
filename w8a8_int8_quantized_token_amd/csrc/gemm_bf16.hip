// bf16 x bf16 -> fp32 product on the kernel of gemm_kernel.h (out[m,n] =
// bf16(sum_k a[m,k] b[n,k]), both operands contiguous along k): the products
// of the backward passes.  v_mfma_f32_32x32x16_bf16 takes 16 bytes per lane
// and operand, as the int8 MFMA does, so stages, swizzle, ring and schedule
// are the int8 ones with K counted in bytes; only the MFMA differs.
#include "gemm_kernel.h"

namespace w8a8 {

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* out, int64_t M,
                            int64_t N, int64_t Kpad, hipStream_t stream) {
  const int64_t kb = 2 * Kpad;   // bytes per row
  return launch_plan<OpB16, Epilogue::kBf16Plain>(
      choose_tile(M, N, kb),
      {reinterpret_cast<const int8_t*>(a), reinterpret_cast<const int8_t*>(b), nullptr, nullptr, nullptr, out, {}},
      M, N, kb, stream);
}

}  // namespace w8a8
