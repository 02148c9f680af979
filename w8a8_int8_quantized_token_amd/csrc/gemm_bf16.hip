// bf16 x bf16 -> fp32 product on the kernel of gemm_kernel.h (out[m,n] =
// bf16(sum_k a[m,k] b[n,k]), both operands contiguous along k): the products
// of the backward passes.  v_mfma_f32_32x32x16_bf16 takes 16 bytes per lane
// and operand, as the int8 MFMA does, so stages, swizzle, ring and schedule
// are the int8 ones with K counted in bytes; only the MFMA differs.
//
// Few output tiles and a long sum (an input's gradient over few tokens) leave
// compute units idle, so K is then cut into ranges whose fp32 sums go to
// slices of a workspace and are joined, in order, by a second kernel.
#include "gemm_kernel.h"

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight outputs of a row per thread; N % 8 == 0.
__global__ __launch_bounds__(256) void join_slices_kernel(const f32x4* __restrict__ part, int chunks, int64_t slice,
                                                          u32x4* __restrict__ out, int64_t groups) {
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
    f32x4 lo = f32x4{0, 0, 0, 0}, hi = lo;
    for (int c = 0; c < chunks; ++c) {
      const f32x4* p = part + (c * slice + g * 8) / 4;
      lo += __builtin_nontemporal_load(p);
      hi += __builtin_nontemporal_load(p + 1);
    }
    const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    const u32x2 a = pack4_bf16(f), b = pack4_bf16(f + 4);
    out[g] = u32x4{a[0], a[1], b[0], b[1]};
  }
}

// Tile and number of K ranges, by a model of the time in us (measured on
// MI355X over 16 shapes from 16 x 1024 x 2048 to 8192 x 4096 x 24576, every
// tile and 1 to 8 ranges; the choice was within 7% of the best at each):
//   launch + rounds * (tile overhead + stages * max(stage, power)) + join,
// stage the time of 128 K bytes of a tile alone on its compute unit, power
// the same with all units busy, when the chip's power limit holds the whole
// launch to about 1250 TFLOP/s.  Ranges pay where tiles leave units idle:
// 1037 x 2064 x 10944: 106 us whole, 72 in three; 777 x 1168 x 4608: 32 us
// whole, 25 in three; 4096 x 4096 x 4096: 110 us whole, 162 in two.
struct Cost {
  double tile_us, stage_us;
  int ring;
};
constexpr Cost kCost[kNumCfg] = {{6.0, 0.97, 6}, {6.0, 1.04, 2}, {5.0, 0.72, 6}, {4.0, 0.56, 3},
                                 {4.0, 0.70, 3}, {1.2, 0.52, 4}, {0.7, 0.38, 3}};
constexpr int64_t kMaxSlices = int64_t(1) << 29;   // bytes of workspace a split may take

struct Choice {
  int cfg, chunks;
};

double cost_us(int cfg, int chunks, int64_t M, int64_t N, int64_t kb) {
  const TileDesc& d = kCfgs[cfg];
  const int64_t tiles = (M + d.block_m - 1) / d.block_m * ((N + d.block_n - 1) / d.block_n) * chunks;
  // 64-byte-stage tiles run several workgroups per unit; a round is still
  // counted as one tile per unit
  const int64_t rounds = (tiles + kCUs - 1) / kCUs;
  const int64_t range = (kb + 128 * chunks - 1) / (128 * chunks) * 128;
  const int64_t per = d.block_k, ring = kCost[cfg].ring;
  const int64_t stages = ((range + per - 1) / per + ring - 1) / ring * ring;
  const double active = (double)std::min<int64_t>(tiles, kCUs);
  const double power = active * (double)(d.block_m * d.block_n) * 128.0 / 1250e6;   // 2 * 64 operations a byte pair
  const double stage = std::max(kCost[cfg].stage_us, power) * (double)per / 128.0;
  double us = 4.0 + (double)rounds * (kCost[cfg].tile_us + (double)stages * stage);
  if (chunks > 1) us += 3.0 + (double)chunks * (double)(M * N) * 8.0 / 4.5e6;
  return us;
}

Choice choose(int64_t M, int64_t N, int64_t kb) {
  Choice best{kWhole256, 1};
  double us = cost_us(best.cfg, 1, M, N, kb);
  for (int cfg = 0; cfg < kNumCfg; ++cfg)
    for (const int chunks : {1, 2, 3, 4, 6, 8}) {
      if (chunks > 1 && (kb < 512 * chunks || M * N * 4 * chunks > kMaxSlices)) break;
      const double c = cost_us(cfg, chunks, M, N, kb);
      if (c < us * 0.999) best = {cfg, chunks}, us = c;
    }
  return best;
}

}  // namespace

hipError_t launch_gemm_bf16_cfg(int cfg, int chunks, const uint16_t* a, const uint16_t* b, uint16_t* out,
                                float* part, int64_t M, int64_t N, int64_t Kpad, hipStream_t stream) {
  const int64_t kb = 2 * Kpad;   // bytes per row
  const int8_t *pa = reinterpret_cast<const int8_t*>(a), *pb = reinterpret_cast<const int8_t*>(b);
  if (chunks <= 1) {
    const KSplit whole{(int)kb, 1, 0};
    return launch_cfg<OpB16, Epilogue::kBf16Plain>(cfg, {pa, pb, nullptr, nullptr, nullptr, out, {}}, M, N, kb, N,
                                                   stream, whole);
  }
  // ranges of whole stages
  const int64_t range = (kb + 128 * chunks - 1) / (128 * chunks) * 128;
  const KSplit ks{(int)kb, (int)((kb + range - 1) / range), M * N};
  const hipError_t e = launch_cfg<OpB16, Epilogue::kRawI32>(cfg, {pa, pb, nullptr, nullptr, nullptr, part, {}}, M, N,
                                                            range, N, stream, ks);
  if (e != hipSuccess) return e;
  const int64_t groups = M * N / 8;
  hipLaunchKernelGGL(join_slices_kernel, dim3((unsigned)std::min<int64_t>((groups + 255) / 256, 256 * 16)), dim3(256),
                     0, stream, reinterpret_cast<const f32x4*>(part), ks.chunks, M * N,
                     reinterpret_cast<u32x4*>(out), groups);
  return hipGetLastError();
}

int64_t gemm_bf16_slices(int64_t M, int64_t N, int64_t Kpad) {
  const Choice c = choose(M, N, 2 * Kpad);
  return c.chunks > 1 ? 4 * M * N * c.chunks : 0;
}

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* out, float* slices, int64_t M,
                            int64_t N, int64_t Kpad, hipStream_t stream) {
  Choice c = choose(M, N, 2 * Kpad);
  if (reinterpret_cast<uintptr_t>(out) % 16 != 0) c.chunks = 1;   // the join writes 16 bytes at a time
  return launch_gemm_bf16_cfg(c.cfg, c.chunks, a, b, out, slices, M, N, Kpad, stream);
}

}  // namespace w8a8
