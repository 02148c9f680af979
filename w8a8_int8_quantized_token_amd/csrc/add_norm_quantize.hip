// The residual's addition, the root-mean-square norm of each row and its codes
// in one pass, and the gradient.  For rows x, residual [K] and a weight w:
//   h = bf16(x + residual),  v = fl32(h w),  s = fl32(max|v| * fl32(1 / 127)),
//   q = rne(fl32(v / s))  (e4m3: 1 / 448 and the e4m3 rounding),
//   scale = fl32(s / rms),  rms = sqrt(mean(h^2) + eps).
// The normed value v / rms is never formed: its factor 1 / rms is common to the
// row, so it cancels in v / s and goes into the scale.  h w is exact (8 + 8
// bits), so the codes depend on no order of summation; the sum of squares
// enters the scale alone.  Squares of bf16 values may vanish or overflow in fp32
// (below 2^-75, above 2^64): such a row, found by its sum, is summed again.
//
// Gradient with the rounding to codes passed straight through, for dn (of the
// normed row) and dh (of h, from what else reads it), r = 1 / rms, hh = h r:
//   dx = dresidual = dh + r (dn w - hh mean(dn w hh)),
//   dw = sum over rows of dn hh.
//
// Bound by memory: 7 bytes per value forward (3 without a residual), 8 backward
// (6 without dh).  A row stays in registers between its reductions and its
// codes, so it is read once.  Measured: 16384 x 4096 82 us (5.7 TB/s), e4m3 of
// 1531 x 5136 without a residual 7.5 (3.1 TB/s; the launch and one chain of load,
// maximum, codes), 1 x 4096 2.3 on the GPU, an empty launch; gradient, 8192 x 4096 with dh 46.6
// (5.8 TB/s, 4.8 us of them the weight's sums in a launch of their own: joined
// in the first, its last workgroup would wait for the others' writes across the
// XCDs), 777 x 1168 9.5.
#include "kernels.h"
#include "quant_codes.h"

#include <algorithm>
#include <type_traits>

namespace w8a8 {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWave = 64;

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
// Sum and maximum over the wavefront by DPP exchanges: six trips through LDS
// take longer than a short row.
template <class F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v = f(v, dpp(v, std::integral_constant<int, 0xB1>{}));    // quad_perm [1,0,3,2]
  v = f(v, dpp(v, std::integral_constant<int, 0x4E>{}));    // quad_perm [2,3,0,1]
  v = f(v, dpp(v, std::integral_constant<int, 0x141>{}));   // row_half_mirror
  v = f(v, dpp(v, std::integral_constant<int, 0x140>{}));   // row_mirror
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = f(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  return over_lanes(v, [](float a, float b) { return a + b; });
}
// (a NaN stays: fmaxf would drop it, and a row of NaNs would have finite codes)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_maxf(float v) {
  return over_lanes(v, [](float a, float b) { return larger(a, b); });
}

// Whether fp32 has the sum of squares: 24 bits of it, or eps is so much larger
// that what vanished does not matter.  (The same in all lanes: a scalar branch.)
__device__ __forceinline__ bool in_range(float sq, float eps) {
  return __builtin_amdgcn_ballot_w64(sq < INFINITY && (sq >= 0x1p-100f || eps >= 0x1p-100f)) != 0;
}
// Where it has not, the sum is made again in 64 bits, from the row in registers.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll 1
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// fl32(v / s) for any fp32 |v| <= 448 s, from the correctly rounded r = 1 / s:
// one correction step brings v r within a step of the quotient, and the second
// then rounds it correctly (Markstein's theorem).  (For the bf16 v of
// quant_codes.h one step gives the same codes; v has twice their bits here.)
__device__ __forceinline__ float quotient(float v, float s, float r) {
  float q = v * r;
  q = fmaf(fmaf(-q, s, v), r, q);
  return fmaf(fmaf(-q, s, v), r, q);
}
// The scale of a row, and of tiny rows (s below 2^-100) v and s times 2^100,
// which is exact and keeps 1 / s finite.
template <bool F8>
__device__ __forceinline__ RowScale scale_of(float amax) {
  RowScale rs;
  rs.s = amax * (F8 ? 1.0f / 448.0f : 1.0f / 127.0f);
  rs.xs = rs.s < 0x1p-100f ? 0x1p100f : 1.0f;
  rs.ss = rs.s * rs.xs;
  rs.r = 1.0f / rs.ss;   // correctly rounded
  return rs;
}
// Codes of 8 values.  No clamp: |v| <= amax, so the quotient is at most a few
// steps above 127 (448), which rounds to it.  The even rounding to an integer is
// the addition of 1.5 * 2^23, whose sum has the code in its lowest byte.
template <bool F8>
__device__ __forceinline__ u32x2 quantize8(const float* v, const RowScale& rs) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = quotient(v[e], rs.ss, rs.r);
  if constexpr (F8) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_copysignf(f[e], v[e]);   // (the correction turns -0 into +0)
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
    return u32x2{(uint32_t)lo, (uint32_t)hi};
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = __float_as_uint(f[4 * i + e] + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
    w[i] = lo | hi;
  }
  return u32x2{w[0], w[1]};
}

struct Norm {
  const u32x4 *x, *residual, *weight;   // rows of `chunks` 16-byte pieces; residual, weight or null
  u32x4* h;                             // or null
  u32x2* q;
  float* scale;
  int64_t M;
  int chunks;
  float eps;
};

// kWaves wavefronts to a row (below four of them: four rows to a workgroup),
// kPieces 16-byte pieces to a lane.
template <int kWaves, int kPieces, bool F8>
__global__ __launch_bounds__(kWave * (kWaves > 4 ? kWaves : 4)) void norm_kernel(Norm a) {
  constexpr int kRows = kWaves > 4 ? 1 : 4 / kWaves, kStride = kWaves * kWave;
  __shared__ f32x2 part[kRows > 1 ? 1 : kWaves];
  __shared__ double far_part[kRows > 1 ? 1 : kWaves];
  const int tid = threadIdx.x % kStride;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kStride;
  if (kRows > 1 && row >= a.M) return;   // whole wavefronts, and no barriers with several rows
  const int64_t base = row * a.chunks;

  u32x4 h[kPieces], w[kPieces], other[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = tid + i * kStride;
    h[i] = other[i] = u32x4{0, 0, 0, 0};
    w[i] = u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};   // ones
    if (c < a.chunks) {
      h[i] = __builtin_nontemporal_load(a.x + base + c);
      if (a.residual != nullptr) other[i] = __builtin_nontemporal_load(a.residual + base + c);
      if (a.weight != nullptr) w[i] = a.weight[c];
    }
  }
  float sq = 0.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (a.residual != nullptr) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        h[i][e] = pack2(low(h[i][e]) + low(other[i][e]), high(h[i][e]) + high(other[i][e]));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = low(h[i][e]), hi = high(h[i][e]);
      sq = fmaf(lo, lo, sq);
      sq = fmaf(hi, hi, sq);
      top = larger(top, larger(fabsf(lo * low(w[i][e])), fabsf(hi * high(w[i][e]))));
    }
  }
  if (a.h != nullptr) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int c = tid + i * kStride;
      if (c < a.chunks) a.h[base + c] = h[i];
    }
  }
  sq = wave_sum(sq);
  top = wave_maxf(top);
  if constexpr (kWaves > 1) {
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = f32x2{sq, top};
    __syncthreads();
    sq = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      const f32x2 p = part[k];
      sq += p[0];
      top = larger(top, p[1]);
    }
  }
  const RowScale rs = scale_of<F8>(top);
  const bool zero = rs.s == 0.0f;
  const float n = (float)(a.chunks * 8);
  float far_scale = -1.0f;   // (below 0: not used)
  if (!in_range(sq, a.eps)) {
    double far = 0.0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        far = fma((double)low(h[i][e]), (double)low(h[i][e]), far);
        far = fma((double)high(h[i][e]), (double)high(h[i][e]), far);
      }
    far = wave_sum(far);
    if constexpr (kWaves > 1) {
      if (threadIdx.x % kWave == 0) far_part[threadIdx.x / kWave] = far;
      __syncthreads();
      far = 0.0;
#pragma unroll 1
      for (int k = 0; k < kWaves; ++k) far += far_part[k];
    }
    far_scale = (float)(rs.s / sqrt(far / n + a.eps));
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = tid + i * kStride;
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = low(h[i][e]) * low(w[i][e]);
      v[2 * e + 1] = high(h[i][e]) * high(w[i][e]);
    }
    if (rs.xs != 1.0f) {   // a row of tiny numbers: a subnormal s may be half of what it should be
      const float most = (F8 ? 448.0f : 127.0f) * rs.ss;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_amdgcn_fmed3f(v[e] * rs.xs, -most, most);
    }
    if (c < a.chunks) a.q[base + c] = zero ? u32x2{0, 0} : quantize8<F8>(v, rs);
  }
  if (tid == 0) a.scale[row] = zero ? 0.0f : far_scale < 0.0f ? rs.s / sqrtf(sq / n + a.eps) : far_scale;
}

template <int kWaves, int kPieces>
hipError_t forward(const Norm& a, bool fp8, hipStream_t s) {
  constexpr int kRows = kWaves > 4 ? 1 : 4 / kWaves;
  const dim3 grid((unsigned)((a.M + kRows - 1) / kRows)), block(kWave * (kWaves > 4 ? kWaves : 4));
  if (fp8) hipLaunchKernelGGL((norm_kernel<kWaves, kPieces, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<kWaves, kPieces, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

// ---- gradient ----

struct NormGrad {
  const u32x4 *dn, *dh, *h, *weight;   // dh, weight or null
  u32x4* dx;
  float* part;   // [gridDim.x][8 * chunks], or null
  int64_t M;
  int chunks;
  float eps;
};

// A workgroup takes every gridDim.x-th row and keeps its rows' sums for the
// weight's gradient in registers.  kAhead: the next row's loads are in flight
// meanwhile.  Long rows leave no registers for that, and the longest
// (kReload) none for the row itself, which is then read again after the
// reductions (from the cache).
enum class Rows { kAhead, kKept, kReload };
template <int kThreads, int kPieces, Rows kRows>
__global__ __launch_bounds__(kThreads) void norm_grad_kernel(NormGrad a) {
  constexpr int kWaves = kThreads / kWave;
  constexpr u32x4 kZeros = {0, 0, 0, 0}, kOnes = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  __shared__ f32x2 part[2][kWaves];
  const int tid = threadIdx.x;
  float sum[kPieces][8];
  u32x4 w[kPieces];
  auto weight = [&](int i) __attribute__((always_inline)) {
    const int c = tid + i * kThreads;
    return a.weight != nullptr && c < a.chunks ? a.weight[c] : kOnes;
  };
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if constexpr (kRows != Rows::kReload) w[i] = weight(i);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[i][e] = 0.0f;
  }
  struct Piece {
    u32x4 h, dn, dh;
  };
  auto load = [&](int64_t row, int i, Piece& p) __attribute__((always_inline)) {
    const int c = tid + i * kThreads;
    p.h = p.dn = p.dh = kZeros;
    if (c < a.chunks && row < a.M) {
      const int64_t at = row * a.chunks + c;
      p.h = __builtin_nontemporal_load(a.h + at);
      p.dn = __builtin_nontemporal_load(a.dn + at);
      if (a.dh != nullptr) p.dh = __builtin_nontemporal_load(a.dh + at);
    }
  };
  Piece now[kPieces];
  [[maybe_unused]] Piece next[kPieces];
  auto load_row = [&](int64_t row, Piece* p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) load(row, i, p[i]);
  };
  float sq, along;   // of a row: h^2 and dn w h
  auto reduce = [&](const Piece& p, u32x4 wt, auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float h0 = f(low(p.h[e])), h1 = f(high(p.h[e]));
      sq = fmaf(h0, h0, sq);
      sq = fmaf(h1, h1, sq);
      along = fmaf(low(p.dn[e]) * low(wt[e]), h0, along);
      along = fmaf(high(p.dn[e]) * high(wt[e]), h1, along);
    }
  };
  int parity = 0;
  auto join = [&]() __attribute__((always_inline)) {
    sq = wave_sum(sq);
    along = wave_sum(along);
    // (two buffers: a wavefront is at most one barrier ahead of another)
    if (tid % kWave == 0) part[parity][tid / kWave] = f32x2{sq, along};
    __syncthreads();
    sq = along = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) sq += part[parity][k][0], along += part[parity][k][1];
    parity ^= 1;
  };
  auto sums_of_reloaded = [&](int64_t row, auto f) __attribute__((always_inline)) {
    sq = along = 0.0f;
#pragma unroll 1
    for (int i = 0; i < kPieces; ++i) {
      Piece p;
      load(row, i, p);
      reduce(p, weight(i), f);
    }
    join();
  };
  const float n = (float)(a.chunks * 8);
  // Piece i of dx, and its share of the weight's gradient; t: mean(dn w hh).
  auto put = [&](int64_t row, int i, const Piece& p, u32x4 wt, float r, float t, auto f) __attribute__((always_inline)) {
    const int c = tid + i * kThreads;
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float h0 = f(low(p.h[e])) * r, h1 = f(high(p.h[e])) * r;
      const float d0 = low(p.dn[e]), d1 = high(p.dn[e]);
      sum[i][2 * e] = fmaf(d0, h0, sum[i][2 * e]);
      sum[i][2 * e + 1] = fmaf(d1, h1, sum[i][2 * e + 1]);
      const float g0 = f(fmaf(d0, low(wt[e]), -(h0 * t))), g1 = f(fmaf(d1, high(wt[e]), -(h1 * t)));
      o[e] = pack2(fmaf(r, g0, low(p.dh[e])), fmaf(r, g1, high(p.dh[e])));
    }
    if (c < a.chunks) a.dx[row * a.chunks + c] = o;
  };
  auto plain = [](float v) __attribute__((always_inline)) { return v; };

  if constexpr (kRows == Rows::kAhead) load_row(blockIdx.x, now);
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    if constexpr (kRows == Rows::kAhead) load_row(row + gridDim.x, next);
    else if constexpr (kRows == Rows::kKept) load_row(row, now);
    if constexpr (kRows == Rows::kReload) {
      sums_of_reloaded(row, plain);
    } else {
      sq = along = 0.0f;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) reduce(now[i], w[i], plain);
      join();
    }
    // A row whose squares leave fp32's range (or, with eps = 0, one of zeros): h
    // times a power of two, half of it here and half in r: hh = (h half) (r half),
    // dx = dh + (r half) (half (dn w - hh t)).  Such a row is loaded again, which
    // leaves the others their registers (4096 x 2560 21.8 us; 22.3 with half in every
    // row's products, 21.1 without any of this; in the loop of reloaded rows half costs
    // nothing).
    float half = 1.0f;
    if (kRows != Rows::kReload && in_range(sq, a.eps)) {
      const float r = 1.0f / sqrtf(sq / n + a.eps), t = along * r / n;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) put(row, i, now[i], w[i], r, t, plain);
    } else {
      if (kRows != Rows::kReload || !in_range(sq, a.eps)) {
        half = sq < 1.0f ? 0x1p50f : 0x1p-50f;
        sums_of_reloaded(row, [&](float v) __attribute__((always_inline)) { return v * (half * half); });
      }
      const float power = sq / n + a.eps * half * half * half * half;
      const float r = power == 0.0f ? 0.0f : 1.0f / sqrtf(power), t = along * r / n;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        Piece p;
        load(row, i, p);
        put(row, i, p, weight(i), r * half, t, [&](float v) __attribute__((always_inline)) { return v * half; });
      }
    }
    if constexpr (kRows == Rows::kAhead) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) now[i] = next[i];
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int c = tid + i * kThreads;
    if (c < a.chunks) {
      f32x4* p = reinterpret_cast<f32x4*>(a.part + ((int64_t)blockIdx.x * a.chunks + c) * 8);
      p[0] = f32x4{sum[i][0], sum[i][1], sum[i][2], sum[i][3]};
      p[1] = f32x4{sum[i][4], sum[i][5], sum[i][6], sum[i][7]};
    }
  }
}

// part [rows][K] -> out [K], in a fixed order: 32 columns to a workgroup, 32
// groups of threads walk the rows with eight loads in flight each.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void norm_sum_kernel(const float* __restrict__ part, int rows, int K,
                                                               float* __restrict__ out) {
  constexpr int kGroups = kSumThreads / 32;
  __shared__ float lds[kGroups][33];
  const int l = threadIdx.x % 32, g = threadIdx.x / 32, e = blockIdx.x * 32 + l;
  float s = 0.0f;
  if (e < K)
    for (int b = g; b < rows; b += 8 * kGroups) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b + i * kGroups < rows ? part[(int64_t)(b + i * kGroups) * K + e] : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  lds[g][l] = s;
  __syncthreads();
  if (g == 0 && e < K) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t += lds[i][l];
    out[e] = t;
  }
}

// Threads of the gradient's workgroups, and their number: about one row in flight
// for each wavefront that the compute units hold (512 workgroups of 256 threads,
// 256 of 512), and more where short rows leave the weight's sums cheap (16384 x
// 1024: 512 workgroups 37.7 us, 1024 31.7; 1024 x 1024: 8.7, 9.4).  Us by 256 / 512
// threads, with a residual's gradient: 100 rows of 2064 6.4 / 6.1, of 3840 7.2 / 6.8;
// 777 of 2064 11.8 / 10.5, of 3840 13.7 / 11.8; 4096 of 2064 22.5 / 23.6, of 2816 23.7 /
// 24.9, of 3584 26.7 / 26.7, of 4096 29.0 / 28.2; 16384 of 2064 60 / 69, of 2816 67 / 72,
// of 3584 80.2 / 81.6, of 4096 88.3 / 87.2.
int grad_threads(int64_t M, int64_t K) {
  if (K > 16384) return 1024;
  return K >= 3584 || (K > 2048 && M <= 1024) ? 512 : 256;
}

template <int kThreads, int kPieces, Rows kRows>
hipError_t backward(const NormGrad& a, int rows, hipStream_t s) {
  hipLaunchKernelGGL((norm_grad_kernel<kThreads, kPieces, kRows>), dim3((unsigned)rows), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

// Wavefronts to a row of the forward pass.  Us by 1 / 4 / 16 of them, with a
// residual: 16384 x 512 14.2 / 21.2 / 58, 4096 x 1024 8.3 / 9.0 / 17.1, 1024 x 1024
// 4.9 / 4.5 / 6.3; 16384 x 4096 80.9 / 73.6 / 86.8, 512 x 4096 9.0 / 5.0 / 4.7, 200 x
// 5136 12.1 / 5.5 / 4.7, 1531 x 5136 18.7 / 14.1 / 14.7; 512 x 8192 - / 8.9 / 7.9,
// 16384 x 8192 - / 164 / 161, 8192 x 12288 - / 128 / 120.
int norm_waves(int64_t M, int64_t K) {
  if (K >= 8192 || (K >= 4096 && M <= 512)) return 16;
  return K <= 1024 && M >= 4096 ? 1 : 4;
}

// A launch has under 2^32 threads.
bool norm_fits(int64_t M, int64_t K) {
  return K <= kMaxNorm && M * norm_waves(M, K) * kWave < (int64_t(1) << 32) - 1024;
}

hipError_t launch_add_norm_quantize(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* h,
                                    void* q, float* scale, int64_t M, int64_t K, float eps, bool fp8, hipStream_t s) {
  const auto in = [](const uint16_t* p) { return reinterpret_cast<const u32x4*>(p); };
  const Norm a{in(x), in(residual), in(weight), reinterpret_cast<u32x4*>(h), static_cast<u32x2*>(q), scale, M, (int)(K / 8), eps};
  const int waves = norm_waves(M, K), pieces = (a.chunks + waves * kWave - 1) / (waves * kWave);
  if (waves == 1) return pieces == 1 ? forward<1, 1>(a, fp8, s) : forward<1, 2>(a, fp8, s);
  if (waves == 4) {
    if (pieces == 1) return forward<4, 1>(a, fp8, s);
    if (pieces == 2) return forward<4, 2>(a, fp8, s);
    return pieces == 3 ? forward<4, 3>(a, fp8, s) : forward<4, 4>(a, fp8, s);
  }
  if (pieces == 1) return forward<16, 1>(a, fp8, s);
  return pieces == 2 ? forward<16, 2>(a, fp8, s) : forward<16, 4>(a, fp8, s);
}

int64_t norm_grad_rows(int64_t M, int64_t K) {
  return std::min<int64_t>(M, K <= 1024 && M >= 4096 ? 1024 : 128 * 1024 / grad_threads(M, K));
}

hipError_t launch_add_norm_grad(const uint16_t* dn, const uint16_t* dh, const uint16_t* h, const uint16_t* weight,
                                uint16_t* dx, float* part, float* dweight, int64_t M, int64_t K, float eps,
                                hipStream_t s) {
  const auto in = [](const uint16_t* p) { return reinterpret_cast<const u32x4*>(p); };
  const NormGrad a{in(dn), in(dh), in(h), in(weight), reinterpret_cast<u32x4*>(dx), part, M, (int)(K / 8), eps};
  const int rows = (int)norm_grad_rows(M, K);
  hipError_t e;
  if (K <= 2048) e = backward<256, 1, Rows::kAhead>(a, rows, s);
  else if (grad_threads(M, K) == 256) e = backward<256, 2, Rows::kAhead>(a, rows, s);
  else if (K <= 4096) e = backward<512, 1, Rows::kAhead>(a, rows, s);
  else if (K <= 8192) e = backward<512, 2, Rows::kAhead>(a, rows, s);
  else if (K <= 16384) e = backward<512, 4, Rows::kKept>(a, rows, s);
  else e = backward<1024, 4, Rows::kReload>(a, rows, s);
  if (e != hipSuccess || part == nullptr) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((K + 31) / 32)), dim3(kSumThreads), 0, s, part, rows, (int)K, dweight);
  return hipGetLastError();
}

}  // namespace w8a8
