// The int8 and fp8 (e4m3) products on the kernel of gemm_kernel.h: plan
// choice, the K-split choice and the launches.
#include "gemm_kernel.h"

namespace w8a8 {

int num_tiles() { return kNumPlans; }
const TileDesc& tile_desc(int tile) { return kCfgs[kPlans[tile].main]; }
int select_tile(int64_t M, int64_t N, int64_t K) { return choose_tile(M, N, K); }

// ---- K split ----
// When to split K, from sweeps on MI355X over every plan and range count
// (M = 256 ... 4096 tokens, N = 3072 / 12288, K = 3072 / 12288): a split pays
// only when the unsplit launch leaves most compute units idle and K is long.
// Its cost is the int32 slices (4 bytes per output and range, written by the
// GEMM and read back by a second pass that also writes the bf16 output) plus
// one more kernel boundary; on the 768px DiT shapes (200+ tiles) that cost
// exceeded what balancing the last round saved, e.g. 2304x3072x3072 33.6 us
// unsplit vs 50+ us in two ranges.  Measured wins: 256x3072x12288 43.4 -> 32.8
// us (8 ranges), 512x3072x12288 58.1 -> 44.1 us (4 ranges), both on 256x128
// tiles.  Rule: 256x128 tiles; split only if they number at most 64 and
// K >= 4096; double the range count while the work items stay within one
// round of 256 and each range keeps at least 768 bytes of K.
constexpr int kSplitPlan = 6;   // 256x128 main tiles

int select_splitk(int64_t M, int64_t N, int64_t K, int* tile) {
  const TileDesc& d = kCfgs[kPlans[kSplitPlan].main];
  const int64_t tiles = ((M + d.block_m - 1) / d.block_m) * ((N + d.block_n - 1) / d.block_n);
  int chunks = 1;
  if (N % 8 == 0 && tiles <= 64 && K >= 4096)
    while (tiles * chunks * 2 <= kCUs && K % (16 * chunks * 2) == 0 && K / (chunks * 2) >= 768) chunks *= 2;
  if (tile) *tile = chunks > 1 ? kSplitPlan : select_tile(M, N, K);
  return chunks;
}

namespace {

template <class Op>
hipError_t launch_epi(int tile, Epilogue epi, const int8_t* xq, const int8_t* wq, const float* sx,
                      const float* sw, const uint16_t* bias, void* out, int64_t M, int64_t N,
                      int64_t K, hipStream_t stream) {
  switch (epi) {
    case Epilogue::kBf16ScaleBias:
      return launch_plan<Op, Epilogue::kBf16ScaleBias>(tile, {xq, wq, sx, sw, bias, out, {}}, M, N, K, stream);
    case Epilogue::kBf16GeluScaleBias:
      return launch_plan<Op, Epilogue::kBf16GeluScaleBias>(tile, {xq, wq, sx, sw, bias, out, {}}, M, N, K, stream);
    case Epilogue::kRawI32:
      return launch_plan<Op, Epilogue::kRawI32>(tile, {xq, wq, nullptr, nullptr, nullptr, out, {}}, M, N, K, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gemm(int tile, Epilogue epi, const int8_t* xq, const int8_t* wq,
                       const float* sx, const float* sw, const uint16_t* bias, void* out,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  return launch_epi<OpI8>(tile, epi, xq, wq, sx, sw, bias, out, M, N, K, stream);
}

hipError_t launch_gemm_partials(int tile, const int8_t* xq, const int8_t* wq, int32_t* partials,
                                int64_t M, int64_t N, int64_t K, int chunks, hipStream_t stream) {
  if (tile < 0 || tile >= kNumPlans || chunks < 1 || K % (16 * chunks) != 0) return hipErrorInvalidValue;
  const KSplit ks{(int)K, chunks, M * N};
  return launch_cfg<OpI8, Epilogue::kRawI32>(kPlans[tile].main, {xq, wq, nullptr, nullptr, nullptr, partials, {}},
                                             M, N, K / chunks, N, stream, ks);
}

hipError_t launch_gemm_fp8(int tile, Epilogue epi, const uint8_t* xq, const uint8_t* wq,
                           const float* sx, const float* sw, const uint16_t* bias, void* out,
                           int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  return launch_epi<OpF8>(tile, epi, reinterpret_cast<const int8_t*>(xq),
                          reinterpret_cast<const int8_t*>(wq), sx, sw, bias, out, M, N, K, stream);
}

}  // namespace w8a8
