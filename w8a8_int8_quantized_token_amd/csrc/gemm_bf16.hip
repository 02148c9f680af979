// bf16 x bf16 -> fp32 product on the kernel of gemm_kernel.h (out[m,n] =
// bf16(sum_k a[m,k] b[n,k]), both operands contiguous along k): the products
// of the backward passes.  v_mfma_f32_16x16x32_bf16 takes 16 bytes per lane
// and operand, as the int8 MFMA does, so stages, swizzle, ring and schedule
// are the int8 ones with K counted in bytes; the MFMA, its fragments and the
// epilogue differ.
//
// Few output tiles and a long sum (an input's gradient over few tokens) leave
// compute units idle, so K is then cut into ranges whose fp32 sums go to
// slices of a workspace and are joined, in order, by a later launch.
#include "gemm_kernel.h"

namespace w8a8 {
namespace {

// Tiles: the int8 product's large ones, and small ones with 128-byte stages
// (64 values; the int8 ones have 64-byte stages, whose barrier every 256
// cycles of MFMAs cost these a third: 777 x 1168 x 4608 on 64x64 tiles 31 us
// with 64-byte stages, 20 with 128).  Four of them: the smallest tile's time is
// its requests' latency over the stages in flight (three 20.7 us, four 17.9,
// six 18.3).
using Cfg128s2 = Tile<128, 128, 128, 2, 2, 2>;
using Cfg128s4 = Tile<128, 128, 128, 2, 2, 4>;
using Cfg64s4 = Tile<64, 64, 128, 2, 2, 4>;
using Cfg64x128 = Tile<64, 128, 128, 2, 2, 3>;
using Cfg128x64 = Tile<128, 64, 128, 2, 2, 3>;
enum BfCfg { kBf256, kBfWhole256, kBf192, kBf128x256, kBf128s2, kBf128s4, kBf64, kBf64x128, kBf128x64, kNumBf };
const TileDesc kBfTiles[kNumBf] = {desc<CfgSplit>(), desc<CfgWhole>(), desc<Cfg192>(), desc<CfgTail>(), desc<Cfg128s2>(),
                                   desc<Cfg128s4>(), desc<Cfg64s4>(), desc<Cfg64x128>(), desc<Cfg128x64>()};

// Tiles with adapters: those whose K loop has the registers for it.
bool low_tile(int cfg, bool raw) { return cfg != kBf256 && cfg != kBf192 && (cfg != kBfWhole256 || !raw); }

template <Epilogue EPI>
hipError_t launch_bf16(int cfg, const Operands<EPI>& o, int64_t M, int64_t N, int64_t K, hipStream_t s, KSplit ks) {
  if constexpr (kLow<EPI>) {
    if (!low_tile(cfg, EPI == Epilogue::kRawLow)) return hipErrorInvalidValue;
    switch (cfg) {
      case kBfWhole256:
        if constexpr (EPI != Epilogue::kRawLow) return launch_t<CfgWhole, OpB16, EPI>(o, M, N, K, N, s, ks);
        else return hipErrorInvalidValue;
      case kBf128x256: return launch_t<CfgTail, OpB16, EPI>(o, M, N, K, N, s, ks);
      case kBf128s2: return launch_t<Cfg128s2, OpB16, EPI>(o, M, N, K, N, s, ks);
      case kBf128s4: return launch_t<Cfg128s4, OpB16, EPI>(o, M, N, K, N, s, ks);
      case kBf64: return launch_t<Cfg64s4, OpB16, EPI>(o, M, N, K, N, s, ks);
      case kBf64x128: return launch_t<Cfg64x128, OpB16, EPI>(o, M, N, K, N, s, ks);
      default: return launch_t<Cfg128x64, OpB16, EPI>(o, M, N, K, N, s, ks);
    }
  } else
  switch (cfg) {
    case kBf256: return launch_t<CfgSplit, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBfWhole256: return launch_t<CfgWhole, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf192: return launch_t<Cfg192, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf128x256: return launch_t<CfgTail, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf128s2: return launch_t<Cfg128s2, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf128s4: return launch_t<Cfg128s4, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf64: return launch_t<Cfg64s4, OpB16, EPI>(o, M, N, K, N, s, ks);
    case kBf64x128: return launch_t<Cfg64x128, OpB16, EPI>(o, M, N, K, N, s, ks);
    default: return launch_t<Cfg128x64, OpB16, EPI>(o, M, N, K, N, s, ks);
  }
}

// Tile and number of K ranges, by a model of the time in us, fitted to
// measurements on MI355X of every tile with 1 to 8 ranges at 44 shapes from 16
// x 1024 x 2048 to 8192 x 4096 x 24576 (its choice was within 9% of the
// fastest at each, 1% in the mean):
//   3.77 + rounds * (tile + stages * max(stage, power)) + join,
// stage the time of 128 K bytes of a tile alone on its compute unit, power the
// same at `rate` TFLOP/s over the whole chip.  All are fitted numbers, no
// properties of the chip: a rate above the 1.83 PFLOP/s that a loop of nothing
// but fragment reads and MFMAs reaches (the whole 256x256 ring's) never binds, and
// that tile's times are its stages' alone.  The measurements are of products by
// themselves with their operands just laid out; in a whole backward pass large
// ones take longer (4096^3 86 us by the model, 96 alone, 103 to 109 in the pass),
// and a choice by a percent says nothing there: 4096 x 2048 x 16384 is 191 as two
// ranges by the model and 192 whole on 128x256 tiles; the two ranges take 256 + 17.
// Ranges pay where tiles leave units idle: 128 x 8192 x 24576: 133 us whole, 92
// in ranges; 512 x 512 x 8192: 23.8 us whole, 13.9 in ranges; but 4096 x 4096 x
// 4096: 100 us whole, 149 in two.
struct Cost {
  double tile_us, stage_us, rate;
  int ring, resident;   // stages of the ring; workgroups per compute unit (kResident)
};
constexpr Cost kCost[kNumBf] = {
    {3.98, 1.172, 1494, 6, 1}, {2.69, 1.244, 2705, 2, 1}, {3.03, 0.881, 1686, 6, 1},
    {3.17, 0.576, 1497, 3, 1}, {0.11, 0.376, 842, 2, 2},  {1.78, 0.363, 1210, 4, 1},
    {0.18, 0.166, 627, 4, 2},  {0.39, 0.235, 813, 3, 2},  {0.21, 0.260, 853, 3, 2}};
constexpr int64_t kMaxSlices = int64_t(1) << 29;   // bytes of workspace a split may take

struct Choice {
  int cfg, chunks;
};

// Bytes of a range: whole 128-byte stages (chunks ranges, or one fewer).
int64_t range_bytes(int64_t kb, int chunks) { return (kb + 128 * chunks - 1) / (128 * chunks) * 128; }

double cost_us(int cfg, int chunks, int64_t M, int64_t N, int64_t kb) {
  const TileDesc& d = kBfTiles[cfg];
  const Cost& c = kCost[cfg];
  const int64_t range = range_bytes(kb, chunks), ranges = (kb + range - 1) / range;
  const int64_t items = (M + d.block_m - 1) / d.block_m * ((N + d.block_n - 1) / d.block_n) * ranges;
  const int64_t stages = (range / 128 + c.ring - 1) / c.ring * c.ring;
  // a tile more on a compute unit that has one costs 0.72 of it
  const double r = c.resident, q = (double)items / kCUs;
  const double rounds = c.resident == 1 ? (double)((items + kCUs - 1) / kCUs)
                        : q <= 1.0      ? 1.0
                        : q <= r        ? 1.0 + (q - 1.0) * 0.717
                                        : q * (1.0 + (r - 1.0) * 0.717) / r;
  // 128 operations per output and 128 bytes of K
  const double power = (double)std::min<int64_t>(items, kCUs) * (double)(d.block_m * d.block_n) * 128.0 / (c.rate * 1e6);
  const double us = 3.77 + rounds * (c.tile_us + (double)stages * std::max(c.stage_us, power));
  return ranges > 1 ? us + 2.5 + (double)ranges * (double)M * (double)N * 1.35e-6 : us;
}

Choice cheapest(int64_t M, int64_t N, int64_t kb, bool low) {
  Choice best{kBfWhole256, 1};
  double us = cost_us(best.cfg, 1, M, N, kb);
  for (int cfg = 0; cfg < kNumBf; ++cfg)
    for (const int chunks : {1, 2, 3, 4, 6, 8}) {
      if (low && !low_tile(cfg, chunks > 1)) continue;
      if (chunks > 1 && (kb < 512 * chunks || M * N * 4 * chunks > kMaxSlices)) break;
      const double c = cost_us(cfg, chunks, M, N, kb);
      if (c < us * 0.999) best = {cfg, chunks}, us = c;
    }
  return best;
}

// The model takes about a microsecond, and a backward pass asks three times
// for each of its products (workspace size, layout, launch): the last shapes'
// choices are kept per thread.
Choice choose(int64_t M, int64_t N, int64_t kb, bool low) {
  struct Entry {
    int64_t M, N, kb;
    bool low;
    Choice c;
  };
  thread_local Entry last[8] = {};
  thread_local unsigned next = 0;
  for (const Entry& e : last)
    if (e.M == M && e.N == N && e.kb == kb && e.low == low) return e.c;
  Entry& e = last[next++ % 8];
  e = {M, N, kb, low, cheapest(M, N, kb, low)};
  return e.c;
}

}  // namespace

int gemm_bf16_slices(int64_t M, int64_t N, int64_t Kpad, bool low) {
  const int64_t kb = 2 * Kpad;
  const int64_t range = range_bytes(kb, choose(M, N, kb, low).chunks);
  return (int)((kb + range - 1) / range);
}

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* b, uint16_t* out, float* slices, int64_t M,
                            int64_t N, int64_t Kpad, const Low* low, hipStream_t stream) {
  const int64_t kb = 2 * Kpad;   // bytes per row
  const int8_t *pa = reinterpret_cast<const int8_t*>(a), *pb = reinterpret_cast<const int8_t*>(b);
  const Choice c = choose(M, N, kb, low != nullptr);
  const int64_t range = range_bytes(kb, c.chunks);
  const int ranges = (int)((kb + range - 1) / range);
  const KSplit whole{(int)kb, 1, 0}, ks{(int)kb, ranges, M * N};
  const bool one = ranges == 1 || slices == nullptr;
  if (low != nullptr) {
    const LowArgs args{low->t, low->b, low->ids, N * low->R, (int)low->ldt, (int)low->R, (int)low->count};
    if (one)
      return launch_bf16<Epilogue::kBf16PlainLow>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, out, args}, M, N, kb, stream, whole);
    return launch_bf16<Epilogue::kRawLow>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, slices, args}, M, N, range, stream, ks);
  }
  if (one)
    return launch_bf16<Epilogue::kBf16Plain>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, out, {}}, M, N, kb, stream, whole);
  return launch_bf16<Epilogue::kRawI32>(c.cfg, {pa, pb, nullptr, nullptr, nullptr, slices, {}}, M, N, range, stream, ks);
}

}  // namespace w8a8
