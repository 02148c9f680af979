// bf16 x bf16 -> fp32 product on the kernel of gemm_kernel.h (out[m,n] =
// bf16(sum_k a[m,k] b[n,k]), both operands contiguous along k): the products
// of the backward passes.  v_mfma_f32_32x32x16_bf16 takes 16 bytes per lane
// and operand, as the int8 MFMA does, so stages, swizzle, ring and schedule
// are the int8 ones with K counted in bytes; only the MFMA differs.
//
// Few output tiles and a long sum (an input's gradient over few tokens) leave
// compute units idle, so K is then cut into ranges whose fp32 sums go to
// slices of a workspace and are joined, in order, by a later launch.
#include "gemm_kernel.h"

namespace w8a8 {
namespace {

// Tile and number of K ranges, by a model of the time in us, fitted to
// measurements on MI355X of every tile with 1 to 8 ranges at 22 shapes from
// 16 x 1024 x 2048 to 8192 x 4096 x 24576 (its choice was the fastest, or
// within 12% of it, at each; 2% in the mean):
//   4 + rounds * (tile + stages * max(stage, power)) + join,
// stage the time of 128 K bytes of a tile alone on its compute unit, power
// the same when `rate` TFLOP/s is what the whole chip's power limit allows.
// Ranges pay where tiles leave units idle: 1037 x 2064 x 10944: 106 us whole,
// 70 in ranges; 777 x 1168 x 4608: 32 us whole, 25 in three; but 4096 x 4096
// x 4096: 110 us whole, 162 in two.
struct Cost {
  double tile_us, stage_us, rate;
  int ring;
};
constexpr Cost kCost[kNumCfg] = {{2.0, 1.12, 1330, 6}, {2.2, 1.28, 1425, 2}, {2.6, 0.88, 1570, 6},
                                 {3.4, 0.56, 1250, 3}, {2.4, 0.79, 1140, 3}, {0.3, 0.45, 800, 4},
                                 {0.2, 0.24, 450, 3}};
constexpr int64_t kMaxSlices = int64_t(1) << 29;   // bytes of workspace a split may take

struct Choice {
  int cfg, chunks;
};

// Bytes of a range: whole 128-byte stages (chunks ranges, or one fewer).
int64_t range_bytes(int64_t kb, int chunks) { return (kb + 128 * chunks - 1) / (128 * chunks) * 128; }

double cost_us(int cfg, int chunks, int64_t M, int64_t N, int64_t kb) {
  const TileDesc& d = kCfgs[cfg];
  const Cost& c = kCost[cfg];
  const int64_t items = (M + d.block_m - 1) / d.block_m * ((N + d.block_n - 1) / d.block_n) * chunks;
  const double tiles = (double)items;
  const int resident = cfg == k64 ? 3 : cfg == k128 ? 2 : 1;   // as kResident
  // tiles that share a compute unit overlap by about a quarter
  const double rounds = resident == 1 ? (double)((items + kCUs - 1) / kCUs)
                        : items <= kCUs ? 1.0
                        : items <= kCUs * resident ? 1.0 + (tiles / kCUs - 1.0) * 0.75
                                                   : tiles / kCUs;
  const int64_t range = range_bytes(kb, chunks);
  const int64_t stages = ((range + d.block_k - 1) / d.block_k + c.ring - 1) / c.ring * c.ring;
  // 128 operations per output and 128 bytes of K
  const double power = (double)std::min<int64_t>(items, kCUs) * (double)(d.block_m * d.block_n) * 128.0 / (c.rate * 1e6);
  const double us = 4.0 + rounds * (c.tile_us + (double)stages * std::max(c.stage_us, power) * d.block_k / 128.0);
  return chunks > 1 ? us + 1.8 + (double)chunks * (double)M * (double)N * 1.6e-6 : us;
}

Choice cheapest(int64_t M, int64_t N, int64_t kb) {
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

// The model takes about a microsecond, and a backward pass asks three times
// for each of its products (workspace size, layout, launch): the last shapes'
// choices are kept per thread.
Choice choose(int64_t M, int64_t N, int64_t kb) {
  struct Entry {
    int64_t M, N, kb;
    Choice c;
  };
  thread_local Entry last[4] = {};
  thread_local unsigned next = 0;
  for (const Entry& e : last)
    if (e.M == M && e.N == N && e.kb == kb) return e.c;
  Entry& e = last[next++ % 4];
  e = {M, N, kb, cheapest(M, N, kb)};
  return e.c;
}

}  // namespace

int gemm_bf16_slices(int64_t M, int64_t N, int64_t Kpad) {
  const int64_t kb = 2 * Kpad;
  const int64_t range = range_bytes(kb, choose(M, N, kb).chunks);
  return (int)((kb + range - 1) / range);
}

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* out, float* slices, int64_t M,
                            int64_t N, int64_t Kpad, hipStream_t stream) {
  const int64_t kb = 2 * Kpad;   // bytes per row
  const int8_t *pa = reinterpret_cast<const int8_t*>(a), *pb = reinterpret_cast<const int8_t*>(b);
  const Choice c = choose(M, N, kb);
  const int64_t range = range_bytes(kb, c.chunks);
  const int ranges = (int)((kb + range - 1) / range);
  if (ranges == 1 || slices == nullptr) {
    const KSplit whole{(int)kb, 1, 0};
    return launch_cfg<OpB16, Epilogue::kBf16Plain>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, out, {}}, M, N, kb, N,
                                                   stream, whole);
  }
  const KSplit ks{(int)kb, ranges, M * N};
  return launch_cfg<OpB16, Epilogue::kRawI32>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, slices, {}}, M, N, range, N,
                                              stream, ks);
}

}  // namespace w8a8
