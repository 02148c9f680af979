// RMS norm of each query and key head with the position rotation in the same
// pass, and its gradient.  For a head x [D], weight w, r = 1/sqrt(mean(x^2) +
// eps), n = x r w, and each pair (a, b) of the first `rot` values turned by its
// row's angle:
//   (a, b) -> (a cos - b sin, b cos + a sin).
// Gradient, with dn the gradient turned back (sin -> -sin), xh = x r:
//   dx = r (dn w - xh mean(dn w xh)),  dw = sum over rows and heads of dn xh.
//
// Bound by memory: 4 bytes per value forward (6 backward).  A head belongs to
// D/16 lanes (rounded up to a power of two), 16 values each: two 16-byte
// loads, whose pairs are both in the lane in either pairing (a lane takes
// values 8u.. and rot/2 + 8u.. when the halves are paired, 16u.. when
// neighbours are), so the rotation needs no exchange and the norm one
// reduction over the head's lanes.  All arithmetic is fp32, rounded to bf16
// once.  The weight's gradient is kept in registers over a workgroup's heads
// and joined by a second small kernel in a fixed order.
//
// Measured: 16384 tokens of 24 + 24 heads of 128 values 78 us, 5.2 TB/s (a
// large copy 5.1 to 5.4); gradient of 8192 tokens of 32 + 8 heads 46 us, 5.5
// TB/s, and 4.7 us for the second kernel.
#include "kernels.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWave = 64;
// Workgroups of the gradient kernel, each a row of weight sums (8192 x 40
// heads: 1024 46 + 4.7 us, 512 53 + 4.7, 2048 47 + 5.4).
constexpr int kMaxSumBlocks = 1024;

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
  return v;
}

// Sum over the G lanes of a head.
template <int G>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// Where lane u of a head has its 16 values: [lo, lo+8) and [hi, hi+8).  Units
// past the rotation take the rest of the head, first half and second half.
template <bool kInterleaved>
__device__ __forceinline__ void unit_of(int u, int D, int rot, int& lo, int& hi) {
  if (kInterleaved) {
    lo = 16 * u;
    hi = lo + 8;
  } else if (u < rot / 16) {
    lo = 8 * u;
    hi = rot / 2 + lo;
  } else {
    lo = rot + 8 * (u - rot / 16);
    hi = lo + (D - rot) / 2;
  }
}

// cos and sin of the lane's 8 pairs; a lane past the rotation turns by nothing.
__device__ __forceinline__ void load_turn(const RopeArgs& a, int64_t pos, int u, float* c, float* s) {
  if (u < a.rot / 16) {
    const int64_t at = pos * (a.rot / 2) + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 cv = *reinterpret_cast<const f32x4*>(a.cos + at + 4 * i);
      const f32x4 sv = *reinterpret_cast<const f32x4*>(a.sin + at + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) c[4 * i + e] = cv[e], s[4 * i + e] = sv[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.0f, s[e] = 0.0f;
  }
}

// The lane's 16 norm weights (1 without a weight).
__device__ __forceinline__ void load_weight(const uint16_t* w, int lo, int hi, float* f) {
  if (w != nullptr) {
    unpack8(*reinterpret_cast<const u32x4*>(w + lo), f);
    unpack8(*reinterpret_cast<const u32x4*>(w + hi), f + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = 1.0f;
  }
}

// Turns the pairs of v[16]: neighbours (interleaved) or v[e], v[8+e].
template <bool kInterleaved, bool kBack>
__device__ __forceinline__ void turn(float* v, const float* c, const float* s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = kInterleaved ? 2 * e : e, j = kInterleaved ? 2 * e + 1 : 8 + e;
    const float a = v[i], b = v[j], t = kBack ? -s[e] : s[e];
    v[i] = fmaf(a, c[e], -(b * t));
    v[j] = fmaf(b, c[e], a * t);
  }
}

// One head of one row per G lanes.
template <int G, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(RopeArgs a, uint32_t heads, uint32_t items) {
  const uint32_t item = (blockIdx.x * kThreads + threadIdx.x) / G;
  const int u = threadIdx.x % G;
  const bool on = item < items && u < a.D / 16;
  const uint32_t m = item / heads, hh = item - m * heads;
  const bool is_k = hh >= (uint32_t)a.Hq;
  const int64_t h = is_k ? hh - a.Hq : hh;
  int lo, hi;
  unit_of<kInterleaved>(u, a.D, a.rot, lo, hi);
  float v[16], w[16], c[8], s[8];
  int64_t pos = 0;
  bool turned = false;
  uint16_t* y = nullptr;
  float sq = 0.0f;
  if (on) {
    const RopeView& x = is_k ? a.k : a.q;
    const RopeView& o = is_k ? a.ko : a.qo;
    const uint16_t* xr = x.p + (int64_t)m * x.row + h * x.head;
    y = o.p + (int64_t)m * o.row + h * o.head;
    const u32x4 x0 = *reinterpret_cast<const u32x4*>(xr + lo), x1 = *reinterpret_cast<const u32x4*>(xr + hi);
    pos = a.positions ? (int64_t)a.positions[m] : (int64_t)(m % (uint32_t)a.P);
    turned = pos >= 0 && pos < a.P;
    load_turn(a, turned ? pos : 0, u, c, s);
    load_weight(is_k ? a.kw : a.qw, lo, hi, w);
    unpack8(x0, v);
    unpack8(x1, v + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) sq = fmaf(v[e], v[e], sq);
  }
  sq = head_sum<G>(sq);
  if (!on) return;
  const float r = __builtin_amdgcn_rsqf(sq / (float)a.D + a.eps);
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = v[e] * r * w[e];
  turn<kInterleaved, false>(v, c, s);
  // (chosen after the turn: a padding row's angles are the table's first row's)
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = turned ? v[e] : 0.0f;
  *reinterpret_cast<u32x4*>(y + lo) = pack8(v);
  *reinterpret_cast<u32x4*>(y + hi) = pack8(v + 8);
}

// Workgroups 0 .. qblocks-1 walk the query heads, the others the key heads.
template <int G, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void norm_rope_grad_kernel(RopeArgs a, RopeView dq, RopeView dk,
                                                                  int qblocks, float* __restrict__ part) {
  __shared__ float lds[kThreads / kWave][1024];
  const bool is_k = (int)blockIdx.x >= qblocks;
  const uint32_t block = is_k ? blockIdx.x - qblocks : blockIdx.x;
  const uint32_t blocks = is_k ? gridDim.x - qblocks : qblocks;
  const uint32_t heads = is_k ? a.Hk : a.Hq, items = (uint32_t)a.M * heads;
  const RopeView x = is_k ? a.k : a.q, dy = is_k ? a.ko : a.qo, dx = is_k ? dk : dq;
  const int u = threadIdx.x % G;
  const bool has = u < a.D / 16;
  int lo, hi;
  unit_of<kInterleaved>(has ? u : 0, a.D, a.rot, lo, hi);
  float w[16], sum[16];
  load_weight(is_k ? a.kw : a.qw, lo, hi, w);
#pragma unroll
  for (int e = 0; e < 16; ++e) sum[e] = 0.0f;
  constexpr uint32_t kPer = kThreads / G;
  // every lane of a wavefront makes the same number of steps
  for (uint32_t first = block * kPer; first < items; first += blocks * kPer) {
    const uint32_t item = first + threadIdx.x / G;
    const bool on = has && item < items;
    const uint32_t m = item / heads, h = item - m * heads;
    float v[16], d[16], c[8], s[8];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = d[e] = 0.0f;
    bool turned = false;
    float sq = 0.0f, along = 0.0f;
    if (on) {
      const uint16_t* xr = x.p + (int64_t)m * x.row + (int64_t)h * x.head;
      const uint16_t* dr = dy.p + (int64_t)m * dy.row + (int64_t)h * dy.head;
      const u32x4 x0 = *reinterpret_cast<const u32x4*>(xr + lo), x1 = *reinterpret_cast<const u32x4*>(xr + hi);
      const u32x4 d0 = *reinterpret_cast<const u32x4*>(dr + lo), d1 = *reinterpret_cast<const u32x4*>(dr + hi);
      const int64_t pos = a.positions ? (int64_t)a.positions[m] : (int64_t)(m % (uint32_t)a.P);
      turned = pos >= 0 && pos < a.P;
      load_turn(a, turned ? pos : 0, u, c, s);
      unpack8(x0, v);
      unpack8(x1, v + 8);
      unpack8(d0, d);
      unpack8(d1, d + 8);
      turn<kInterleaved, true>(d, c, s);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (!turned) d[e] = 0.0f;
        sq = fmaf(v[e], v[e], sq);
        along = fmaf(d[e] * w[e], v[e], along);
      }
    }
    sq = head_sum<G>(sq);
    along = head_sum<G>(along);
    if (on) {
      const float r = __builtin_amdgcn_rsqf(sq / (float)a.D + a.eps);
      const float t = along * r / (float)a.D;   // mean(dn w xh)
      float o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float xh = v[e] * r;
        o[e] = turned ? r * fmaf(d[e], w[e], -(xh * t)) : 0.0f;
        if (turned) sum[e] = fmaf(d[e], xh, sum[e]);
      }
      uint16_t* orow = dx.p + (int64_t)m * dx.row + (int64_t)h * dx.head;
      *reinterpret_cast<u32x4*>(orow + lo) = pack8(o);
      *reinterpret_cast<u32x4*>(orow + hi) = pack8(o + 8);
    }
  }
  if (part == nullptr) return;
  // over the heads of a wavefront, then over the workgroup's wavefronts
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int off = G; off < kWave; off *= 2) sum[e] += __shfl_xor(sum[e], off, kWave);
  const int wave = threadIdx.x / kWave;
  if (threadIdx.x % kWave < G && has) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lds[wave][lo + e] = sum[e];
      lds[wave][hi + e] = sum[8 + e];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.D; e += kThreads)
    part[(int64_t)blockIdx.x * a.D + e] = (lds[0][e] + lds[1][e]) + (lds[2][e] + lds[3][e]);
}

// part [qblocks + kblocks, D] -> dqw, dkw: grid (ceil(D / 32), 2).  Latency
// bound: 32 groups of threads walk the rows, eight loads in flight each
// (1024 rows of 128: 4 us, against 28 us with eight groups and no unrolling).
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void norm_weight_sum_kernel(const float* __restrict__ part, int qblocks,
                                                                      int blocks, int D, float* __restrict__ dqw,
                                                                      float* __restrict__ dkw) {
  constexpr int kGroups = kSumThreads / 32;
  __shared__ float lds[kGroups][33];
  float* const out = blockIdx.y ? dkw : dqw;
  if (out == nullptr) return;
  const int l = threadIdx.x % 32, g = threadIdx.x / 32, e = blockIdx.x * 32 + l;
  const int from = blockIdx.y ? qblocks : 0, to = blockIdx.y ? blocks : qblocks;
  float s = 0.0f;
  if (e < D)
    for (int b = from + g; b < to; b += 8 * kGroups) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b + i * kGroups < to ? part[(int64_t)(b + i * kGroups) * D + e] : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  lds[g][l] = s;
  __syncthreads();
  if (g == 0 && e < D) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t += lds[i][l];
    out[e] = t;
  }
}

int lanes_of(int D) {
  int g = 1;
  while (g * 16 < D) g *= 2;
  return g;
}

template <int G>
hipError_t forward(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  const uint32_t heads = (uint32_t)(a.Hq + a.Hk), items = (uint32_t)a.M * heads;
  const uint32_t per = kThreads / G;
  const dim3 grid((items + per - 1) / per);
  if (interleaved) hipLaunchKernelGGL((norm_rope_kernel<G, true>), grid, dim3(kThreads), 0, stream, a, heads, items);
  else hipLaunchKernelGGL((norm_rope_kernel<G, false>), grid, dim3(kThreads), 0, stream, a, heads, items);
  return hipGetLastError();
}

// Workgroups for the query and key heads, in proportion to their number.
void grad_blocks(int64_t M, int64_t Hq, int64_t Hk, int D, int& qb, int& kb) {
  const int64_t per = kThreads / lanes_of(D);
  const int64_t nq = (M * Hq + per - 1) / per, nk = (M * Hk + per - 1) / per;
  const double f = nq + nk > kMaxSumBlocks ? (double)kMaxSumBlocks / (double)(nq + nk) : 1.0;
  qb = (int)std::max<int64_t>(Hq > 0, (int64_t)(f * (double)nq));
  kb = (int)std::max<int64_t>(Hk > 0, (int64_t)(f * (double)nk));
}

template <int G>
hipError_t backward(const RopeArgs& a, const RopeView& dq, const RopeView& dk, bool interleaved, int qb, int kb,
                    float* part, hipStream_t stream) {
  const dim3 grid((unsigned)(qb + kb));
  if (interleaved)
    hipLaunchKernelGGL((norm_rope_grad_kernel<G, true>), grid, dim3(kThreads), 0, stream, a, dq, dk, qb, part);
  else
    hipLaunchKernelGGL((norm_rope_grad_kernel<G, false>), grid, dim3(kThreads), 0, stream, a, dq, dk, qb, part);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_rope(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  switch (lanes_of(a.D)) {
    case 1: return forward<1>(a, interleaved, stream);
    case 2: return forward<2>(a, interleaved, stream);
    case 4: return forward<4>(a, interleaved, stream);
    case 8: return forward<8>(a, interleaved, stream);
    case 16: return forward<16>(a, interleaved, stream);
    case 32: return forward<32>(a, interleaved, stream);
    default: return forward<64>(a, interleaved, stream);
  }
}

int64_t norm_rope_grad_rows(int64_t M, int64_t Hq, int64_t Hk, int D) {
  int qb, kb;
  grad_blocks(M, Hq, Hk, D, qb, kb);
  return qb + kb;
}

hipError_t launch_norm_rope_grad(const RopeArgs& a, const RopeView& dq, const RopeView& dk, bool interleaved,
                                 float* part, float* dqw, float* dkw, hipStream_t stream) {
  int qb, kb;
  grad_blocks(a.M, a.Hq, a.Hk, a.D, qb, kb);
  hipError_t e;
  switch (lanes_of(a.D)) {
    case 1: e = backward<1>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    case 2: e = backward<2>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    case 4: e = backward<4>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    case 8: e = backward<8>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    case 16: e = backward<16>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    case 32: e = backward<32>(a, dq, dk, interleaved, qb, kb, part, stream); break;
    default: e = backward<64>(a, dq, dk, interleaved, qb, kb, part, stream); break;
  }
  if (e != hipSuccess || part == nullptr) return e;
  hipLaunchKernelGGL(norm_weight_sum_kernel, dim3((unsigned)((a.D + 31) / 32), 2), dim3(kSumThreads), 0, stream, part,
                     qb, qb + kb, a.D, dqw, dkw);
  return hipGetLastError();
}

}  // namespace w8a8
