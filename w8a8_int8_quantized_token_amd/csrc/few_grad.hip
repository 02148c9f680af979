// The input's gradient for few tokens, straight from the codes:
//   dx[m,k] = sum_n d[m,n] * q[n,k],
// with d = bf16(dy * w_scale) (linear), or the gated gradient's dg and du in
// blocks of 16 gate and 16 up columns.  The tiled product needs the weight
// turned into bf16 rows of n first, which for few tokens costs more than the
// product: 5 bytes of traffic per code beside the one that is read here.
//
// Bound by reading the weight once.  A wavefront takes 32 rows of q at a time
// and 16 * KB columns: a lane loads KB codes of each of 8 rows (256- or
// 128-byte runs), and byte j of those 8 words' worth of rows, converted (exact
// in bf16), is its fragment of column KB * (lane % 16) + j for
// v_mfma_f32_16x16x32_bf16; no transposition goes through LDS.  The rows are
// dealt to wavefronts and workgroups; a workgroup's eight sums are joined
// through LDS in a fixed order, the workgroups' go to slices, which
// launch_finish joins.
//
// Measured, with the join (turning the weight before a tiled product): 12000 x
// 5408, 1 token 22 us (73), 29 tokens 30 us (75), 64 tokens 39 us (74).
#include "kernels.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWave = 64, kWaves = 8, kThreads = kWave * kWaves;
constexpr int kRowsB = 32;   // rows of q of a step

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

struct FewGrad {
  const uint16_t* d;    // linear: dy [M,N]; gated: [M,ldd], scaled, zeros past the last channel
  int64_t ldd;
  const int8_t* q;      // [N,K], gated [2N,K]
  const float* scale;   // linear: of the rows of q
  float* slices;        // [slices][M][K]
  int M, K, blocks_n, per, col_blocks;   // steps in all and of a slice
  int64_t N;
};

template <int MT, int KB, bool kGated>
__global__ __launch_bounds__(kThreads) void few_grad_kernel(FewGrad a) {
  constexpr int kPart = MT * KB * kWave;   // f32x4 of a wavefront's sums
  __shared__ f32x4 part[kWaves / 2 * kPart];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int l16 = lane % 16, h = lane / 16;
  const int cb = (int)(blockIdx.x % (unsigned)a.col_blocks), slice = (int)(blockIdx.x / (unsigned)a.col_blocks);
  const int col = cb * 16 * KB + l16 * KB;
  // columns past K and rows past N are read at the last ones: the former are
  // not written, and the latter meet zeros of d
  const int at = min(col, a.K - KB);
  const int first = slice * a.per + wave, last = min((slice + 1) * a.per, a.blocks_n);

  f32x4 acc[MT][KB];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < KB; ++j) acc[t][j] = f32x4{0, 0, 0, 0};

  struct Step {
    uint32_t w[8][KB / 4];
    u32x4 d[MT];
  };
  auto load = [&](int b, Step& s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int64_t row;
      if constexpr (kGated) row = min((int64_t)b * 16 + h % 2 * 8 + i, a.N - 1) + h / 2 * a.N;
      else row = min((int64_t)b * kRowsB + h * 8 + i, a.N - 1);
      __builtin_memcpy(s.w[i], __builtin_assume_aligned(a.q + row * a.K + at, KB), KB);
    }
    const int64_t n = (int64_t)b * kRowsB + h * 8;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint16_t* row = a.d + (int64_t)min(t * 16 + l16, a.M - 1) * a.ldd;
      if constexpr (kGated) {
        s.d[t] = *reinterpret_cast<const u32x4*>(row + n);
      } else {
        float v[8];
        if (n + 8 <= a.N) {
          u32x4 r;
          __builtin_memcpy(&r, row + n, 16);
          float sc[8];
          __builtin_memcpy(sc, a.scale + n, 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = __uint_as_float(e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16) * sc[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = n + e < a.N ? __uint_as_float((uint32_t)row[n + e] << 16) * a.scale[n + e] : 0.0f;
        }
        s.d[t] = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
      }
    }
  };
  auto multiply = [&](const Step& s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(s.w[i][j / 4] >> (8 * (j % 4)));
      const u32x4 f = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, s.d[t]),
                                                            __builtin_bit_cast(bf16x8, f), acc[t][j], 0, 0, 0);
    }
  };
  // the next step's loads are on the way while a step is multiplied
  Step now, next;
  if (first < last) load(first, now);
  for (int b = first; b < last; b += kWaves) {
    if (b + kWaves < last) load(b + kWaves, next);
    multiply(now);
    now = next;
  }

  // the upper half of the wavefronts' sums onto the lower half's
#pragma unroll
  for (int half = kWaves / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < KB; ++j) part[(wave - half) * kPart + (t * KB + j) * kWave + lane] = acc[t][j];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < KB; ++j) acc[t][j] += part[wave * kPart + (t * KB + j) * kWave + lane];
    }
    __syncthreads();
  }
  if (wave != 0 || col >= a.K) return;
  // this lane: tokens 4h .. 4h+3 of each 16, columns col .. col + KB - 1
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = t * 16 + 4 * h + e;
      if (m < a.M) {
        f32x4* out = reinterpret_cast<f32x4*>(a.slices + ((int64_t)slice * a.M + m) * a.K + col);
#pragma unroll
        for (int j = 0; j < KB; j += 4) out[j / 4] = f32x4{acc[t][j][e], acc[t][j + 1][e], acc[t][j + 2][e], acc[t][j + 3][e]};
      }
    }
}

// Columns of a lane: 16 up to 32 tokens; with more the sums would not fit the
// registers.
int lane_columns(int64_t M) { return M <= 32 ? 16 : 8; }

template <bool kGated>
hipError_t launch(const FewGrad& a, int slices, hipStream_t stream) {
  const dim3 grid((unsigned)(a.col_blocks * slices));
  if (a.M <= 16) hipLaunchKernelGGL((few_grad_kernel<1, 16, kGated>), grid, dim3(kThreads), 0, stream, a);
  else if (a.M <= 32) hipLaunchKernelGGL((few_grad_kernel<2, 16, kGated>), grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((few_grad_kernel<4, 8, kGated>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

int64_t steps(int64_t N, bool gated) { return gated ? (N + 15) / 16 : (N + kRowsB - 1) / kRowsB; }
// Steps of a slice: about one workgroup per compute unit, each wavefront at
// least one step.
int64_t slice_steps(int64_t M, int64_t N, int64_t K, bool gated) {
  const int64_t cols = 16 * lane_columns(M), blocks = (K + cols - 1) / cols, n = steps(N, gated);
  const int64_t slices = std::max<int64_t>(1, std::min((n + kWaves - 1) / kWaves, 256 / blocks));
  return (n + slices - 1) / slices;
}

}  // namespace

int few_grad_slices(int64_t M, int64_t N, int64_t K, bool gated) {
  const int64_t per = slice_steps(M, N, K, gated);
  return (int)((steps(N, gated) + per - 1) / per);
}

hipError_t launch_few_grad(const uint16_t* d, int64_t ldd, const int8_t* q, const float* scale, float* slices,
                           int64_t M, int64_t N, int64_t K, bool gated, hipStream_t stream) {
  if (M < 1 || M > kFewGradTokens) return hipErrorInvalidValue;
  const int64_t cols = 16 * lane_columns(M);
  const FewGrad a{d, ldd, q, scale, slices, (int)M, (int)K, (int)steps(N, gated), (int)slice_steps(M, N, K, gated),
                  (int)((K + cols - 1) / cols), N};
  const int s = few_grad_slices(M, N, K, gated);
  return gated ? launch<true>(a, s, stream) : launch<false>(a, s, stream);
}

}  // namespace w8a8
