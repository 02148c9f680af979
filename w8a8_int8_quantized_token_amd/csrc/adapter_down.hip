// The first product of a low-rank adapter, of the adapter that each row (token)
// is assigned:
//   t[m,r] = bf16(scaling[id] * scale[m] * sum_k X[m,k] P[id][r,k]),  id = ids[m],
// zeros where id is outside [0, count) and in the columns from R up to the next
// multiple of 16.  X is int8 codes with one scale per row, bf16 activations that
// are quantized on the way (codes and scales are outputs too, the same as
// quantize_rows'), or bf16 values.  t is rounded to bf16 once, from fp32 sums:
// it is the operand of the next product, on the bf16 matrix cores, whose result
// is rounded to bf16 with the linear's; t's rounding is 2^-9 of each of its
// terms, of either sign.
//
// Few rows: a workgroup takes one row and 16 ranks, a wavefront two of them,
// with the lanes along k (M K R fused multiply-adds, and P read once for each
// row, from L2 where rows share an adapter).  More rows: a workgroup takes 32
// of them on the bf16 matrix cores (codes are exact in bf16), its wavefronts
// every eighth 64 values of k, and goes through the adapters that its rows
// have one after another; a row takes the sums of its own adapter alone.
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
__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void codes4(uint32_t w, float* f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = (float)(int8_t)(w >> (8 * e));
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
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

using Rows = DownRows;
constexpr int kRanks = 16;          // of a workgroup, two per wavefront
constexpr int kKeep = 4;            // pieces of 8 values that a thread quantizes
constexpr int kMaxFused = kKeep * kThreads * 8;

template <Rows R>
__global__ __launch_bounds__(kThreads) void down_row_kernel(Down a) {
  __shared__ __attribute__((aligned(16))) u32x2 codes[R == Rows::kQuantize ? kMaxFused / 8 : 1];
  __shared__ uint32_t amax[kWaves];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t m = blockIdx.x;
  const int id = adapter_of(a, m);
  const int pieces = (a.K + 7) / 8;
  float scale = 1.0f;
  if constexpr (R == Rows::kCodes) scale = a.scale[m];
  if constexpr (R == Rows::kQuantize) {
    const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + m * a.K);
    u32x4 v[kKeep];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int c = threadIdx.x + i * kThreads;
      v[i] = c < pieces ? x[c] : kZeros;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = absmax_bits(top, v[i][e]);
    }
    top = wave_max(max(top & 0xffffu, top >> 16));
    if (lane == 0) amax[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = max(top, amax[w]);
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
  const int r0 = blockIdx.y * kRanks + 2 * wave;   // this wavefront's two ranks (R is even)
  float sum[2] = {0.0f, 0.0f};
  if (id >= 0 && r0 < a.R) {
    const uint16_t* p0 = a.p + id * a.p_stride + (int64_t)r0 * a.ldp;
    const uint16_t* p1 = p0 + a.ldp;
    constexpr int kSteps = 4;
    for (int c0 = lane; c0 < pieces; c0 += kSteps * kWave) {
      u32x4 w[kSteps][2], v[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int c = c0 + s * kWave;
        w[s][0] = w[s][1] = v[s] = kZeros;
        if (c < pieces) {
          w[s][0] = *reinterpret_cast<const u32x4*>(p0 + c * 8);
          w[s][1] = *reinterpret_cast<const u32x4*>(p1 + c * 8);
          if constexpr (R == Rows::kValues) {
            v[s] = load8(static_cast<const uint16_t*>(a.x) + m * a.K, c * 8, a.K);
          } else {
            u32x2 q;
            if constexpr (R == Rows::kQuantize) q = codes[c];
            else q = reinterpret_cast<const u32x2*>(static_cast<const int8_t*>(a.x) + m * a.K)[c];
            v[s][0] = q[0], v[s][1] = q[1];
          }
        }
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        float x[8], y[8];
        if constexpr (R == Rows::kValues) {
          unpack8(v[s], x);
        } else {
          codes4(v[s][0], x);
          codes4(v[s][1], x + 4);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          unpack8(w[s][k], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[k] = fmaf(x[e], y[e], sum[k]);
        }
      }
    }
    const float f = a.scaling[id];
#pragma unroll
    for (int k = 0; k < 2; ++k) sum[k] = wave_sum(sum[k]) * scale * f;
  }
  if (lane == 0) {
    *reinterpret_cast<uint32_t*>(a.t + m * a.ldt + r0) = pack2(sum[0], sum[1]);
    if (a.t2 != nullptr) {
      const float s2 = a.scale2[m];
      *reinterpret_cast<uint32_t*>(a.t2 + m * a.ldt + r0) = pack2(sum[0] * s2, sum[1] * s2);
    }
  }
}

// ---- 32 rows per workgroup ----

constexpr int kBlockRows = 32, kStepK = 64;

// 64 values of k at a time: a lane has 16 consecutive ones of a row, the first
// and the last eight of them for two MFMAs; both operands are dealt alike.
template <Rows R, int kTiles>
__global__ __launch_bounds__(kThreads) void down_block_kernel(Down a) {
  __shared__ f32x4 part[kWaves][kTiles][2][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int l16 = lane % 16, h = lane / 16;
  const int64_t m0 = (int64_t)blockIdx.x * kBlockRows;
  const int first = blockIdx.y * kTiles * 16;   // rank
  int id[2];
  int64_t row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + i * 16 + l16;
    row[i] = min(m, a.M - 1);
    id[i] = m < a.M ? adapter_of(a, m) : -1;
  }
  f32x4 res[kTiles][2];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) res[t][0] = res[t][1] = f32x4{0, 0, 0, 0};

  struct Step {
    u32x4 p[kTiles][2], x[2][2];
  };
  auto load = [&](const uint16_t* p, int s, Step& v) __attribute__((always_inline)) {
    const int k = s * kStepK + 16 * h;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int r = min(first + t * 16 + l16, a.R - 1);
      v.p[t][0] = v.p[t][1] = kZeros;
      if (k < a.K) {   // (rows of p are whole pieces of 16 values)
        const u32x4* from = reinterpret_cast<const u32x4*>(p + (int64_t)r * a.ldp + k);
        v.p[t][0] = from[0];
        v.p[t][1] = from[1];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v.x[i][0] = v.x[i][1] = kZeros;
      if (k < a.K) {
        if constexpr (R == Rows::kValues) {
          const uint16_t* from = static_cast<const uint16_t*>(a.x) + row[i] * a.K;
          v.x[i][0] = load8(from, k, a.K);
          v.x[i][1] = load8(from, k + 8, a.K);
        } else {
          v.x[i][0] = *reinterpret_cast<const u32x4*>(static_cast<const int8_t*>(a.x) + row[i] * a.K + k);
        }
      }
    }
  };
  uint64_t left[2] = {__builtin_amdgcn_ballot_w64(id[0] >= 0), __builtin_amdgcn_ballot_w64(id[1] >= 0)};
  const int steps = (a.K + kStepK - 1) / kStepK;
  while ((left[0] | left[1]) != 0) {
    const int ad = left[0] != 0 ? __builtin_amdgcn_readlane(id[0], __builtin_ctzll(left[0]))
                                : __builtin_amdgcn_readlane(id[1], __builtin_ctzll(left[1]));
#pragma unroll
    for (int i = 0; i < 2; ++i) left[i] &= ~__builtin_amdgcn_ballot_w64(id[i] == ad);
    const uint16_t* p = a.p + ad * a.p_stride;
    f32x4 acc[kTiles][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[t][0] = acc[t][1] = f32x4{0, 0, 0, 0};
    Step now, next;
    load(p, wave, now);
    for (int s = wave; s < steps; s += kWaves) {
      load(p, s + kWaves, next);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        u32x4 x[2];
        if constexpr (R == Rows::kValues) {
          x[0] = now.x[i][0];
          x[1] = now.x[i][1];
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float f[8];
            codes4(now.x[i][0][2 * g], f);
            codes4(now.x[i][0][2 * g + 1], f + 4);
            x[g] = u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
          }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int g = 0; g < 2; ++g)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now.p[t][g]),
                                                                __builtin_bit_cast(bf16x8, x[g]), acc[t][i], 0, 0, 0);
      }
      now = next;
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) res[t][i][e] = id[i] == ad ? acc[t][i][e] : res[t][i][e];
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) part[wave][t][i][lane] = res[t][i];
  __syncthreads();
  // a wavefront for each 16 ranks by 16 rows; lane: row l16, ranks 4h .. 4h + 3
  if (wave >= 2 * kTiles) return;
  const int t = wave / 2, i = wave % 2;
  const int64_t m = m0 + i * 16 + l16;
  const int r = first + t * 16 + 4 * h;
  if (m >= a.M || r >= a.ldt) return;
  f32x4 sum = part[0][t][i][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += part[w][t][i][lane];
  const int ad = i ? id[1] : id[0];
  float f = 0.0f, scale = 1.0f;
  if (ad >= 0) f = a.scaling[ad];
  if constexpr (R == Rows::kCodes) scale = a.scale[m];
  const bool on = ad >= 0 && r < a.R;
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = on ? sum[e] * scale * f : 0.0f;
  *reinterpret_cast<u32x2*>(a.t + m * a.ldt + r) = u32x2{pack2(sum[0], sum[1]), pack2(sum[2], sum[3])};
  if (a.t2 != nullptr) {
    const float s2 = a.scale2[m];
    *reinterpret_cast<u32x2*>(a.t2 + m * a.ldt + r) =
        u32x2{pack2(sum[0] * s2, sum[1] * s2), pack2(sum[2] * s2, sum[3] * s2)};
  }
}

template <Rows R>
hipError_t launch(const Down& a, hipStream_t s) {
  if (a.M <= kDownRows) {
    hipLaunchKernelGGL((down_row_kernel<R>), dim3((unsigned)a.M, (unsigned)(a.ldt / kRanks)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  if constexpr (R != Rows::kQuantize) {
    const unsigned blocks = (unsigned)((a.M + kBlockRows - 1) / kBlockRows);
    if (a.R <= 16) hipLaunchKernelGGL((down_block_kernel<R, 1>), dim3(blocks), dim3(kThreads), 0, s, a);
    else if (a.R <= 32) hipLaunchKernelGGL((down_block_kernel<R, 2>), dim3(blocks), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((down_block_kernel<R, 4>), dim3(blocks, (unsigned)((a.R + 63) / 64)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool down_quantizes(int64_t M, int64_t K) { return M <= kDownRows && K <= kMaxFused; }

hipError_t launch_down(DownRows rows, const Down& a, hipStream_t stream) {
  if (a.M < 1 || a.R < 8 || a.R % 8 != 0 || a.ldt < a.R || a.ldt % 16 != 0) return hipErrorInvalidValue;
  switch (rows) {
    case Rows::kCodes: return launch<Rows::kCodes>(a, stream);
    case Rows::kQuantize: return down_quantizes(a.M, a.K) ? launch<Rows::kQuantize>(a, stream) : hipErrorInvalidValue;
    default: return launch<Rows::kValues>(a, stream);
  }
}

}  // namespace w8a8
