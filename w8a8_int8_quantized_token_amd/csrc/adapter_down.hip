// The first product of a low-rank adapter, of the adapter that each row (token)
// is assigned:
//   t[m,r] = bf16(scaling[id] * scale[m] * sum_k X[m,k] P[id][r,k]),  id = ids[m],
// zeros where id is outside [0, count) and in the columns from R up to the next
// multiple of 16.  X is int8 codes with one scale per row, bf16 activations that
// are quantized on the way (codes and scales are outputs too, the same as
// quantize_rows'), or bf16 values.  t is rounded to bf16 once, from fp32 sums:
// it is the operand of the next product, on the bf16 matrix cores, whose result
// is rounded to bf16 with the linear's; t's rounding is up to 2^-8 of each of its
// terms, of either sign.  For the matrices' gradients, whose sums are long, the
// values come out in two bf16 parts instead (`two_parts`).
//
// Few rows: a workgroup takes one row and 16 ranks, a wavefront two of them,
// with the lanes along k (M K R fused multiply-adds, and P read once for each
// row, from L2 where rows share an adapter).  More rows: a workgroup takes 32
// rows of one adapter at a time on the bf16 matrix cores (codes are exact in
// bf16), its wavefronts a range of k each.
//
// Bound by reading X where ranks are few: 8192 rows of 4096 codes, rank 16, 13 us
// warm and 23 from cold memory (a copy of these bytes: 21); 16 rows, quantized
// on the way, 4.6.  Where they are many, by P, which every 32 rows read from
// L2 anew: 8192 rows, rank 64, codes of 4096 and values of 8192: 74 us warm, 570
// MB at 7.7 TB/s, which is what the lines that a compute unit's L1 can have
// outstanding allow (with all rows of P the same one: 36).  Tiles of 64 rows
// halve P's share but leave half the compute units idle at that size (72).
#include "adapter_sum.h"
#include "kernels.h"
#include "quant_codes.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWave = 64, kWaves = 8, kThreads = kWave * kWaves;
constexpr u32x4 kZeros = {0, 0, 0, 0};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
// v in two bf16 parts, the high half its leading bits, the low half the rest.
// Both have v's sign and neither is a zero unless v is, so that the products with
// an infinity are the same infinity: a rest of nothing is taken as 2^-17 of v.
__device__ __forceinline__ uint32_t two_parts(float v) {
  const uint32_t bits = __float_as_uint(v) | (__float_as_uint(v) % 65536 != 0 || v == 0.0f ? 0u : 0x40u);
  const float high = __uint_as_float(bits & 0xffff0000u), rest = __uint_as_float(bits) - high;
  return (bits & 0xffff0000u) | (fabsf(v) < INFINITY ? pack2(rest, 0.0f) : bits >> 16);
}
// Eight bf16 values of a row of K from column k on, zeros past its end, from
// any 2-byte address.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int k, int K) {
  u32x4 v = kZeros;
  if (k + 8 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) v[e / 2] |= (uint32_t)row[k + e] << (16 * (e % 2));
  }
  return v;
}
__device__ __forceinline__ int adapter_of(const Down& a, int64_t m) {
  const int id = a.ids[m];
  return id >= 0 && id < a.count ? id : -1;
}

// ---- one row per workgroup ----

enum class Rows { kCodes, kQuantize, kValues };
constexpr int kRanks = 16;          // of a workgroup, two per wavefront
constexpr int kKeep = 4;            // pieces of 8 values that a thread quantizes
constexpr int kMaxFused = kKeep * kThreads * 8;

template <Rows R>
__device__ __forceinline__ void down_row(const Down& a) {
  __shared__ __attribute__((aligned(16))) u32x2 codes[R == Rows::kQuantize ? kMaxFused / 8 : 1];
  __shared__ uint32_t amax[kWaves];
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t m = blockIdx.x;
  const int pieces = (a.K + 7) / 8;
  const int r0 = blockIdx.y * kRanks + 2 * wave;   // this wavefront's two ranks (R is even)
  [[maybe_unused]] u32x4 v[kKeep];
  if constexpr (R == Rows::kQuantize) {
    const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + m * a.K);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int c = threadIdx.x + i * kThreads;
      v[i] = c < pieces ? x[c] : kZeros;
    }
  }
  const int id = adapter_of(a, m);
  float scale = 1.0f;
  if constexpr (R == Rows::kCodes) scale = a.scale[m];
  const bool on = id >= 0 && r0 < a.R;
  const RankRows rows(a.p + max(id, 0) * a.p_stride + (int64_t)min(r0, a.R - 2) * a.ldp, a.ldp, pieces, on);
  RankPieces w;   // the first ones are on the way while the codes are made
  rows.load(lane, w);
  if constexpr (R == Rows::kQuantize) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = absmax_bits(top, v[i][e]);
    top = wave_max(max(top & 0xffffu, top >> 16));
    if (lane == 0) amax[wave] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWaves; ++k) top = max(top, amax[k]);
    const RowScale rs = row_scale<false>(top);
    scale = top ? rs.s : 0.0f;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c < pieces) {
        const u32x2 q = top ? quant_chunk<false>(v[i], rs.xs, rs.ss, rs.r) : u32x2{0, 0};
        codes[c] = q;
        if (blockIdx.y == 0) reinterpret_cast<u32x2*>(a.codes + m * a.K)[c] = q;
      }
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) a.code_scale[m] = scale;
    __syncthreads();
  }
  float sum[2] = {0.0f, 0.0f};
  if (on) {
    for (int c0 = lane; c0 < pieces; c0 += kSumSteps * kWave) {
      if (c0 > lane) rows.load(c0, w);
      float x[kSumSteps][8];
#pragma unroll
      for (int s = 0; s < kSumSteps; ++s) {
        const int c = c0 + s * kWave;
        if constexpr (R == Rows::kValues) {
          unpack8(c < pieces ? load8(static_cast<const uint16_t*>(a.x) + m * a.K, c * 8, a.K) : kZeros, x[s]);
        } else {
          u32x2 q = u32x2{0, 0};
          if (c < pieces) {
            if constexpr (R == Rows::kQuantize) q = codes[c];
            else q = reinterpret_cast<const u32x2*>(static_cast<const int8_t*>(a.x) + m * a.K)[c];
          }
          codes4(q[0], x[s]);
          codes4(q[1], x[s] + 4);
        }
      }
      add_ranks(w, x, sum);
    }
    const float f = a.scaling[id];
#pragma unroll
    for (int k = 0; k < 2; ++k) sum[k] = sum_lanes(sum[k]) * scale * f;
  }
  if (lane == 0) {
    if (a.t != nullptr) *reinterpret_cast<uint32_t*>(a.t + m * a.ldt + r0) = pack2(sum[0], sum[1]);
    if (a.parts != nullptr) {
      const float f = a.parts_scale == nullptr ? 1.0f : id >= 0 ? a.parts_scale[m] : 0.0f;
      *reinterpret_cast<u32x2*>(a.parts + m * a.ldt + r0) = u32x2{two_parts(sum[0] * f), two_parts(sum[1] * f)};
    }
  }
}

template <Rows R>
__global__ __launch_bounds__(kThreads) void down_row_kernel(Down a) {
  down_row<R>(a);
}

// ---- 32 rows of one adapter at a time ----

constexpr int kTileRows = 32, kChunk = 256, kIds = kChunk / kWave;
// A workgroup's LDS: the wavefronts' sums, and each wavefront's list of rows.
template <int kTiles>
struct Lds {
  f32x4 part[kWaves][kTiles][2][kWave];
  uint16_t list[kWaves][kChunk];
};

// The rows of a chunk are sorted by their adapters, each adapter's rows cut into
// tiles of 32, and the tiles dealt to `slots` workgroups: so the work is that of
// the tiles, in whatever order the ids come.  (Blocks of 32 rows in the rows'
// own order, each going through all the adapters that it has: as fast for long
// runs, but 38 us and not 15 for 2048 rows of 4096 codes with sixteen adapters
// mixed, 129 and not 25 for 8192.)
//
// A step is 64 or 128 values of k, a quarter of them in a row in each lane
// (both operands are dealt alike), 16 bytes for an MFMA.  Each wavefront has a
// range of k of its own and walks it in order, so that a row's sum is the same
// whatever rows share its tile.  (Starts that differ from tile to tile, so that
// not all wavefronts read the same place of rows that are pages apart: no faster
// on codes, 8192 rows of 4096 values 36 us and not 37.)  kDepth steps of loads are
// in flight.
template <Rows R, int kTiles>
__device__ __forceinline__ void down_block(const Down& a, int64_t chunk, int rank_block, int slot, int slots,
                                           Lds<kTiles>& lds) {
  constexpr bool kCodes = R == Rows::kCodes;
  constexpr int kMma = kCodes && kTiles < 4 ? 4 : 2;     // MFMAs of a step and tile
  constexpr int kLane = kMma * 8, kStepK = 4 * kLane;    // values of a lane and of a step
  constexpr int kDepth = kTiles == 1 ? 3 : 2;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int l16 = lane % 16, h = lane / 16;
  const int64_t m0 = chunk * kChunk;
  const int first = rank_block * kTiles * 16;   // rank
  int id[kIds];
  uint64_t left[kIds];   // lanes whose rows are still to come
#pragma unroll
  for (int j = 0; j < kIds; ++j) {
    const int64_t m = m0 + j * kWave + lane;
    id[j] = m < a.M ? adapter_of(a, m) : -1;
    left[j] = __builtin_amdgcn_ballot_w64(id[j] >= 0);
  }
  auto zeros = [&](int64_t m) __attribute__((always_inline)) {
    for (int r = first; r < min(first + 16 * kTiles, a.ldt); r += 8) {
      if (a.t != nullptr) *reinterpret_cast<u32x4*>(a.t + m * a.ldt + r) = kZeros;
    }
  };
  if (slot == 0) {
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      const int64_t m = m0 + j * kWave + lane;
      if (j == wave && m < a.M && id[j] < 0) zeros(m);
    }
  }

  constexpr int kWords = kCodes ? kMma / 2 : kMma;   // 16-byte words of a lane's values of x
  struct Step {
    u32x4 p[kTiles][kMma], x[2][kWords];
  };
  const int steps = (a.K + kStepK - 1) / kStepK, per = (steps + kWaves - 1) / kWaves;
  const int from = wave * per, here = max(min(per, steps - from), 0);   // this wavefront's steps
  int64_t row[2];
  // Step n of the wavefront's; past its end zeros.
  auto load = [&](const uint16_t* p, int n, Step& v) __attribute__((always_inline)) {
    const int k = n < here ? (from + n) * kStepK + kLane * h : a.ldp;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < kWords; ++g) {
        v.x[i][g] = kZeros;
        const int at = k + g * (kCodes ? 16 : 8);
        if (at < a.K) {
          if constexpr (kCodes)
            v.x[i][g] = *reinterpret_cast<const u32x4*>(static_cast<const int8_t*>(a.x) + row[i] * a.K + at);
          else v.x[i][g] = load8(static_cast<const uint16_t*>(a.x) + row[i] * a.K, at, a.K);
        }
      }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int r = min(first + t * 16 + l16, a.R - 1);
#pragma unroll
      for (int g = 0; g < kMma; ++g) {
        v.p[t][g] = kZeros;
        if (k + 8 * g < a.ldp) v.p[t][g] = *reinterpret_cast<const u32x4*>(p + (int64_t)r * a.ldp + k + 8 * g);
      }
    }
  };
  // (the control flow is the same in all wavefronts)
  for (int tile = 0;;) {
    int ad = -1;
#pragma unroll
    for (int j = kIds - 1; j >= 0; --j)
      if (left[j] != 0) ad = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(left[j]));
    if (ad < 0) break;
    uint64_t with[kIds];
    int rows = 0;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      with[j] = __builtin_amdgcn_ballot_w64(id[j] == ad);
      left[j] &= ~with[j];
      rows += __popcll(with[j]);
    }
    const int tiles = (rows + kTileRows - 1) / kTileRows;
    int mine = slot - tile;   // the first of the adapter's tiles that is this workgroup's
    while (mine < 0) mine += slots;
    tile += tiles;
    if (mine >= tiles) continue;
    int before = 0;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      if (id[j] == ad)
        lds.list[wave][before + __popcll(with[j] & ((uint64_t(1) << lane) - 1))] = (uint16_t)(j * kWave + lane);
      before += __popcll(with[j]);
    }
    const uint16_t* p = a.p + ad * a.p_stride;
    for (; mine < tiles; mine += slots) {
#pragma unroll
      for (int i = 0; i < 2; ++i) row[i] = m0 + lds.list[wave][min(mine * kTileRows + i * 16 + l16, rows - 1)];
      // what the sums are multiplied by: on the way from here on
      const int t = wave / 2, i = wave % 2, r = first + t * 16 + 4 * h;
      const bool writes = t < kTiles && r < a.ldt && mine * kTileRows + i * 16 + l16 < rows;
      const int64_t m = i ? row[1] : row[0];
      const float f = a.scaling[ad], scale = kCodes ? a.scale[m] : 1.0f, s2 = a.parts_scale != nullptr ? a.parts_scale[m] : 1.0f;
      f32x4 acc[kTiles][2];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) acc[t][0] = acc[t][1] = f32x4{0, 0, 0, 0};
      auto multiply = [&](const Step& v) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u32x4 x[kMma];
          if constexpr (kCodes) {
#pragma unroll
            for (int g = 0; g < kMma; ++g) {
              float f[8];
              codes4(v.x[i][g / 2][2 * (g % 2)], f);
              codes4(v.x[i][g / 2][2 * (g % 2) + 1], f + 4);
              x[g] = u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
            }
          } else {
#pragma unroll
            for (int g = 0; g < kMma; ++g) x[g] = v.x[i][g];
          }
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int g = 0; g < kMma; ++g)
              acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v.p[t][g]),
                                                                  __builtin_bit_cast(bf16x8, x[g]), acc[t][i], 0, 0, 0);
        }
      };
      Step ring[kDepth];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) load(p, d, ring[d]);
      for (int n = 0; n < here; n += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
          multiply(ring[d]);
          load(p, n + kDepth + d, ring[d]);
        }
      }
      __syncthreads();   // the sums of the tile before are read
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) lds.part[wave][t][i][lane] = acc[t][i];
      __syncthreads();
      // a wavefront for each 16 ranks by 16 rows; lane: row l16, ranks 4h .. 4h + 3
      if (!writes) continue;
      f32x4 sum = lds.part[0][t][i][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += lds.part[w][t][i][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = r < a.R ? sum[e] * scale * f : 0.0f;
      if (a.t != nullptr) *reinterpret_cast<u32x2*>(a.t + m * a.ldt + r) = u32x2{pack2(sum[0], sum[1]), pack2(sum[2], sum[3])};
      if (a.parts != nullptr) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = r < a.R ? two_parts(sum[e] * s2) : 0u;
        *reinterpret_cast<u32x4*>(a.parts + m * a.ldt + r) = w;
      }
    }
  }
}

// grid (chunks of rows, blocks of ranks, slots); two products share a launch,
// of codes and of values (b, the last grid.z = slots ones).
template <int kTiles>
__global__ __launch_bounds__(kThreads) void down_block_kernel(Down a) {
  __shared__ Lds<kTiles> lds;
  down_block<Rows::kCodes, kTiles>(a, blockIdx.x, blockIdx.y, blockIdx.z, gridDim.z, lds);
}
template <int kTiles>
__global__ __launch_bounds__(kThreads) void down_block_kernel2(Down codes, Down values, int slots) {
  __shared__ Lds<kTiles> lds;
  const int z = blockIdx.z;
  if (codes.M > 0 && z >= slots)   // (the longer rows first)
    down_block<Rows::kCodes, kTiles>(codes, blockIdx.x, blockIdx.y, z - slots, slots, lds);
  else
    down_block<Rows::kValues, kTiles>(values, blockIdx.x, blockIdx.y, z, slots, lds);
}
__global__ __launch_bounds__(kThreads) void down_row_kernel2(Down codes, Down values) {
  if (blockIdx.z == 0) down_row<Rows::kValues>(values);
  else down_row<Rows::kCodes>(codes);
}

// Workgroups to a chunk of rows: one for each tile of long runs; more, for the
// partial tiles of mixed ids, where compute units are idle otherwise (one with
// nothing to do still takes 2 us).
int slots_of(const Down& a, int tiles) {
  const int64_t blocks = (a.M + kChunk - 1) / kChunk * ((a.R + 16 * tiles - 1) / (16 * tiles));
  constexpr int kFull = kChunk / kTileRows;
  return (int)std::max<int64_t>(kFull, std::min<int64_t>((int64_t)kFull + a.count, 256 / blocks));
}
dim3 block_grid(const Down& a, int tiles, int z) {
  return dim3((unsigned)((a.M + kChunk - 1) / kChunk), (unsigned)((a.R + 16 * tiles - 1) / (16 * tiles)), (unsigned)z);
}
// Tiles of 16 ranks to a workgroup: as few as leave no compute unit more than
// one workgroup, since a row of x is read from L2 faster than many ranks are by
// one workgroup (codes, 2048 rows of 4096, 64 ranks: four tiles 21.8 us, one
// 12.5; but 4096 rows of both products, one tile 33.7, four 26.7).
int tiles_of(const Down& a, int products) {
  const int64_t rows = products * ((a.M + kTileRows - 1) / kTileRows);
  int tiles = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
  while (tiles > 1 && rows * ((a.R + 8 * tiles - 1) / (8 * tiles)) <= 256) tiles /= 2;
  return tiles;
}

// Few rows: a workgroup for each row and 16 ranks.  Warm codes, us by rows / in
// tiles, one adapter: K = 4096, rank 16: 256 rows 5.0 / 11.9, 1024 9.0 / 11.9, 1280
// 10.4 / 12.0, 1536 11.9 / 11.8; rank 32: 512 9.1 / 11.9, 768 11.8 / 11.9, 1024 14.9 /
// 11.9; rank 128: 128 8.7 / 11.6, 192 11.6 / 11.7, 256 14.5 / 11.8; K = 1168, rank
// 16: 1024 5.4 / 6.7, 1280 6.2 / 6.6, 1536 6.9 / 6.7.  With sixteen adapters mixed,
// rank 16: 1536 12.4 / 15.3, 2048 15.2 / 15.4; rank 128: 128 15.2 / 14.8.  Both
// products, with da and db, by rows times ranks, one adapter and eight mixed: rank 8
// of 4096 and 4096: 16384 27.8 / 29.4 and 32.5 / 35.9, 20480 31.3 / 30.6 and 35.4 / 36.1,
// 24576 36.5 / 33.8 and 38.0 / 36.3; of 1024 and 8192: 20480 32.3 / 39.4 and 46.7 / 53.7,
// 32768 43.1 / 41.2 and 57.2 / 55.8; of 1168 and 1168: 12288 19.4 / 19.8 and 21.7 /
// 24.2, 20480 23.7 / 21.4 and 26.1 / 25.7; rank 32 of 4096 and 4096: 12288 28.4 / 30.0
// and 35.2 / 38.2, 16384 32.9 / 30.4 and 38.8 / 38.7, 20480 41.3 / 35.3 and 42.6 / 38.9; of
// 1024 and 8192: 16384 36.6 / 41.4 and 50.4 / 57.6, 20480 41.5 / 42.1 and 54.9 / 56.8;
// rank 64 of 2064 and 5466: 16384 33.4 / 30.4 and 59.6 / 59.0, 20480 41.2 / 34.0 and 62.6 /
// 57.8; of 4096 and 12288: 16384 44.7 / 48.9 and 97.7 / 101.9, 20480 51.0 / 49.2 and
// 103.4 / 99.4.
bool by_rows(int64_t M, int64_t R, int products) {
  return M * ((R + 15) / 16 * 16) <= (products == 1 || R <= 16 ? 20480 : 16384);
}

// Codes alone, by the rules of as many products: a gradient's bits do not depend
// on which others are asked for.
hipError_t launch_codes(const Down& a, bool quantize, int products, hipStream_t s) {
  if (a.M < 1 || a.R < 8 || a.R % 8 != 0 || a.ldt < a.R || a.ldt % 16 != 0)
    return hipErrorInvalidValue;
  const dim3 threads(kThreads), rows((unsigned)a.M, (unsigned)(a.ldt / kRanks));
  if (quantize) {
    if (!down_quantizes(a.M, a.K, a.R)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(down_row_kernel<Rows::kQuantize>, rows, threads, 0, s, a);
  } else if (by_rows(a.M, a.R, products)) {
    hipLaunchKernelGGL(down_row_kernel<Rows::kCodes>, rows, threads, 0, s, a);
  } else {
    const int tiles = tiles_of(a, products);
    const dim3 grid = block_grid(a, tiles, slots_of(a, tiles));
    if (tiles == 1) hipLaunchKernelGGL(down_block_kernel<1>, grid, threads, 0, s, a);
    else if (tiles == 2) hipLaunchKernelGGL(down_block_kernel<2>, grid, threads, 0, s, a);
    else hipLaunchKernelGGL(down_block_kernel<4>, grid, threads, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

bool down_quantizes(int64_t M, int64_t K, int64_t R) { return by_rows(M, R, 1) && K <= kMaxFused; }

hipError_t launch_down(const Down& a, bool quantize, hipStream_t s) { return launch_codes(a, quantize, 1, s); }

hipError_t launch_down_pair(const Down* codes, const Down* values, hipStream_t s) {
  if (values == nullptr) return codes != nullptr ? launch_codes(*codes, false, 2, s) : hipSuccess;
  const Down& v = *values;
  Down c{};   // (M = 0: none)
  if (codes != nullptr) c = *codes;
  if (v.M < 1 || v.R < 8 || v.R % 8 != 0 || v.ldt < v.R || v.ldt % 16 != 0 ||
      (c.M > 0 && (c.M != v.M || c.R != v.R || c.ldt != v.ldt)))
    return hipErrorInvalidValue;
  const dim3 threads(kThreads);
  const int both = c.M > 0 ? 2 : 1;
  if (by_rows(v.M, v.R, 2)) {
    hipLaunchKernelGGL(down_row_kernel2, dim3((unsigned)v.M, (unsigned)(v.ldt / kRanks), both), threads, 0, s, c, v);
    return hipGetLastError();
  }
  const int tiles = tiles_of(v, 2), slots = slots_of(v, tiles);
  const dim3 grid = block_grid(v, tiles, both * slots);
  if (tiles == 1) hipLaunchKernelGGL(down_block_kernel2<1>, grid, threads, 0, s, c, v, slots);
  else if (tiles == 2) hipLaunchKernelGGL(down_block_kernel2<2>, grid, threads, 0, s, c, v, slots);
  else hipLaunchKernelGGL(down_block_kernel2<4>, grid, threads, 0, s, c, v, slots);
  return hipGetLastError();
}

}  // namespace w8a8
