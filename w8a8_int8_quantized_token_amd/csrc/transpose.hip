// Operand layout of the backward products.  The product kernel wants both
// operands contiguous along the summed index, but the input's gradient sums
// over output channels (rows of the weight) and the weight's gradient over
// tokens (rows of the activations), so
//   transpose_codes: int8 [R,C] (times scale[r]) -> bf16 [C, ld], zeros past
//     column R; or, `paired`, the R = 2N rows of a stacked [gate; up] weight
//     with 16 gate columns, the 16 up columns of the same channels, and so on
//     (the order of the gated gradient's columns; zeros for channels past N);
//   transpose_bf16:  bf16 [R,C] -> bf16 [C, ld] the same way, and the fp32
//     sums of each column over blocks of rows;
//   pad_rows:        bf16 [R,C] -> bf16 [R, ld], zeros past column C;
//   sum_rows:        fp32 [P,C] -> bf16 [C], summed over P.
// Codes are small integers and exact in bf16; with a scale each value
// q * scale is rounded to bf16 once.
//
// Bound by memory: R*C*(1+2) and R*C*(2+2) bytes.  A tile of 64 x 64 values
// passes through LDS (rows padded by 4 bytes so that reading down a column
// walks all banks), read in 16-byte pieces and written as 128-byte row pieces.
#include "kernels.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kT = 64;          // tile edge
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ float bf(uint32_t half) { return __uint_as_float(half << 16); }

// Eight values of a row of C from column c on, zeros past its end, from any
// 2-byte address (an unaligned 16-byte load where all eight are there).
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t c, int64_t C) {
  u32x4 v = u32x4{0, 0, 0, 0};
  if (c + 8 <= C) {
    __builtin_memcpy(&v, row + c, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) v[e / 2] |= (uint32_t)row[c + e] << (16 * (e % 2));
  }
  return v;
}

// Source row of output column v (-1: none, a zero).
__device__ __forceinline__ int64_t source_row(int64_t v, int64_t R, bool paired) {
  if (!paired) return v < R ? v : -1;
  const int64_t ch = (v >> 5) * 16 + (v & 15), n = R / 2;
  return ch < n ? ((v >> 4) & 1) * n + ch : -1;
}

// grid (ceil(C/128), ceil(ld/64)); C % 16 == 0, ld % 8 == 0.  64 rows by 128
// columns; a thread turns 8 rows of 4 columns, read as 8 words (LDS rows of 33
// words: the 64 lanes' words lie in 64 banks) and written as four 16-byte
// pieces of 128-byte runs.  33.5 MB of codes to 67 MB: see the figures at
// launch_transpose_codes.
constexpr int kCodeRows = 64, kCodeCols = 128;
template <bool kPaired>
__global__ __launch_bounds__(kThreads) void transpose_codes_kernel(
    const int8_t* __restrict__ q, const float* __restrict__ scale, uint16_t* __restrict__ out,
    int64_t R, int64_t C, int64_t ld) {
  __shared__ uint32_t tile[kCodeRows][kCodeCols / 4 + 1];
  __shared__ __attribute__((aligned(16))) float s_lds[kCodeRows];
  const int tid = threadIdx.x;
  const int64_t c0 = (int64_t)blockIdx.x * kCodeCols;
  const int tr = (tid % 8) * 8, tc = tid / 8;   // this thread's rows and word column when writing
  for (int64_t r0 = (int64_t)blockIdx.y * kCodeRows; r0 < ld; r0 += (int64_t)gridDim.y * kCodeRows) {
    const int r = tid / 8, c = (tid % 8) * 16;
    u32x4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t from = source_row(r0 + i * 32 + r, R, kPaired);
      v[i] = from >= 0 && c0 + c < C ? *reinterpret_cast<const u32x4*>(q + from * C + c0 + c) : u32x4{0, 0, 0, 0};
    }
    if (scale != nullptr && tid < kCodeRows) {
      const int64_t at = source_row(r0 + tid, R, kPaired);
      s_lds[tid] = at >= 0 ? scale[at] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[i * 32 + r][c / 4 + e] = v[i][e];
    __syncthreads();
    if (c0 + tc * 4 < C && r0 + tr < ld) {
      uint32_t w[8];
      float s[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k] = tile[tr + k][tc];
        s[k] = scale != nullptr ? s_lds[tr + k] : 1.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack2((float)(int8_t)(w[2 * e] >> (8 * j)) * s[2 * e],
                       (float)(int8_t)(w[2 * e + 1] >> (8 * j)) * s[2 * e + 1]);
        *reinterpret_cast<u32x4*>(out + (c0 + tc * 4 + j) * ld + r0 + tr) = o;
      }
    }
    __syncthreads();
  }
}

// One workgroup: 64 columns, `span` rows (a multiple of 64).  out may be
// null (sums only), sums may be null.
__global__ __launch_bounds__(kThreads) void transpose_bf16_kernel(
    const uint16_t* __restrict__ x, uint16_t* __restrict__ out, float* __restrict__ sums, int64_t R,
    int64_t C, int64_t ld, int64_t Rpad, int span) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[kT][kT + 2];
  __shared__ float part[kThreads / 8][kT];   // 32 row groups of each column
  const int tid = threadIdx.x;
  const int64_t c0 = (int64_t)blockIdx.x * kT;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  const int64_t first = (int64_t)blockIdx.y * span, last = first + span < Rpad ? first + span : Rpad;
  for (int64_t r0 = first; r0 < last; r0 += kT) {
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int r = it * 32 + tid / 8, c = (tid % 8) * 8;
      u32x4 v = u32x4{0, 0, 0, 0};
      if (r0 + r < R) v = load8(x + (r0 + r) * C, c0 + c, C);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] += bf(v[e] & 0xffffu);
        acc[2 * e + 1] += bf(v[e] >> 16);
        *reinterpret_cast<uint32_t*>(&tile[r][c + 2 * e]) = v[e];
      }
    }
    __syncthreads();
    if (out != nullptr) {
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int id = it * kThreads + tid, c = id / 8, r = (id % 8) * 8;
        if (c0 + c < C && r0 + r < Rpad) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = (uint32_t)tile[r + 2 * e][c] | (uint32_t)tile[r + 2 * e + 1][c] << 16;
          *reinterpret_cast<u32x4*>(out + (c0 + c) * ld + r0 + r) = w;
        }
      }
    }
    __syncthreads();
  }
  if (sums != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[tid / 8][(tid % 8) * 8 + e] = acc[e];
    __syncthreads();
    if (tid < kT && c0 + tid < C) {
      float s = 0.0f;
      for (int g = 0; g < kThreads / 8; ++g) s += part[g][tid];
      sums[(int64_t)blockIdx.y * C + c0 + tid] = s;
    }
  }
}

__global__ __launch_bounds__(kThreads) void pad_rows_kernel(const uint16_t* __restrict__ x,
                                                            uint16_t* __restrict__ out, int64_t R,
                                                            int64_t C, int64_t ld) {
  const int64_t per_row = ld / 8, n = R * per_row;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    *reinterpret_cast<u32x4*>(out + r * ld + c) = load8(x + r * C, c, C);
  }
}

// 32 columns per workgroup, 32 groups of rows with eight loads in flight
// each, joined in a fixed order.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void sum_rows_kernel(const float* __restrict__ part,
                                                               uint16_t* __restrict__ out, int64_t P,
                                                               int64_t C) {
  constexpr int kGroups = kSumThreads / 32;
  __shared__ float s_lds[kGroups][33];
  const int g = threadIdx.x / 32, l = threadIdx.x % 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + l;
  float s = 0.0f;
  if (c < C)
    for (int64_t p = g; p < P; p += 8 * kGroups) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p + i * kGroups < P ? part[(p + i * kGroups) * C + c] : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  s_lds[g][l] = s;
  __syncthreads();
  if (g == 0 && c < C) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t += s_lds[i][l];
    out[c] = __builtin_bit_cast(uint16_t, (__bf16)t);
  }
}

// A fill kernel rather than a memset, which a captured graph would record.
__global__ __launch_bounds__(kThreads) void zero_kernel(uint16_t* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = 0;
}

}  // namespace

hipError_t launch_zero(void* p, int64_t halves, hipStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>((halves + kThreads - 1) / kThreads, 256 * 16);
  hipLaunchKernelGGL(zero_kernel, dim3(grid), dim3(kThreads), 0, stream, static_cast<uint16_t*>(p), halves);
  return hipGetLastError();
}

hipError_t launch_transpose_codes(const int8_t* q, const float* scale, uint16_t* out, int64_t R,
                                  int64_t C, int64_t ld, bool paired, hipStream_t stream) {
  const dim3 grid((unsigned)((C + kCodeCols - 1) / kCodeCols),
                  (unsigned)std::min<int64_t>((ld + kCodeRows - 1) / kCodeRows, 65535));
  if (paired)
    hipLaunchKernelGGL((transpose_codes_kernel<true>), grid, dim3(kThreads), 0, stream, q, scale, out, R, C, ld);
  else
    hipLaunchKernelGGL((transpose_codes_kernel<false>), grid, dim3(kThreads), 0, stream, q, scale, out, R, C, ld);
  return hipGetLastError();
}

// Rows of one workgroup's sums: as many as leave at least about 8 workgroups
// per compute unit, 64 to 1024.
int64_t transpose_sum_span(int64_t R, int64_t C) {
  const int64_t tiles = (C + kT - 1) / kT;
  int64_t span = 64;
  while (span < 1024 && tiles * ((R + 2 * span - 1) / (2 * span)) >= 2048) span *= 2;
  while ((R + span - 1) / span > 65535) span *= 2;
  return span;
}

hipError_t launch_transpose_bf16(const uint16_t* x, uint16_t* out, float* sums, int64_t R, int64_t C,
                                 int64_t ld, int64_t Rpad, hipStream_t stream) {
  const int64_t span = transpose_sum_span(R, C);
  const dim3 grid((unsigned)((C + kT - 1) / kT), (unsigned)((R + span - 1) / span));
  hipLaunchKernelGGL(transpose_bf16_kernel, grid, dim3(kThreads), 0, stream, x, out, sums, R, C, ld, Rpad,
                     (int)span);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const uint16_t* x, uint16_t* out, int64_t R, int64_t C, int64_t ld,
                           hipStream_t stream) {
  const int64_t n = R * (ld / 8);
  const unsigned grid = (unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 256 * 16);
  hipLaunchKernelGGL(pad_rows_kernel, dim3(grid), dim3(kThreads), 0, stream, x, out, R, C, ld);
  return hipGetLastError();
}

hipError_t launch_sum_rows(const float* part, uint16_t* out, int64_t P, int64_t C, hipStream_t stream) {
  hipLaunchKernelGGL(sum_rows_kernel, dim3((unsigned)((C + 31) / 32)), dim3(kSumThreads), 0, stream, part, out,
                     P, C);
  return hipGetLastError();
}

}  // namespace w8a8
