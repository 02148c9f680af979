// Sums of a row by two ranks of an adapter, shared by the kernels that make an
// adapter's first product for few rows, so that they produce the same bits: the
// lanes of a wavefront along k, pieces of 8 values 64 apart in each lane, added
// in order, then over the lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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
// Sum over the wavefront by DPP exchanges (few_tokens.hip's maximum likewise).
template <int kCtrl>
__device__ __forceinline__ float plus_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum_lanes(float v) {
  v = plus_dpp<0xB1>(v);    // quad_perm [1,0,3,2]
  v = plus_dpp<0x4E>(v);    // quad_perm [2,3,0,1]
  v = plus_dpp<0x141>(v);   // row_half_mirror
  v = plus_dpp<0x140>(v);   // row_mirror
  const uint32_t a = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t b = __float_as_uint(v);
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Pieces of two ranks' rows that are on the way at once.
constexpr int kSumSteps = 4;
struct RankPieces {
  u32x4 w[kSumSteps][2];
};
// The two rows of p, which are the same in all lanes, as buffer ranges (nothing
// where there is no adapter): pieces past their end are zeros, without a branch,
// whose end would wait for the loads.
struct RankRows {
  __amdgpu_buffer_rsrc_t row[2];
  __device__ __forceinline__ RankRows(const uint16_t* p, int64_t ldp, int pieces, bool on) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      row[k] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p + k * ldp), (short)0, on ? pieces * 16 : 0, 0x00020000);
  }
  __device__ __forceinline__ void load(int c0, RankPieces& r) const {
#pragma unroll
    for (int s = 0; s < kSumSteps; ++s)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        r.w[s][k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row[k], (c0 + s * 64) * 16, 0, 0));
  }
};
// x: the row's 8 values of each of the pieces
__device__ __forceinline__ void add_ranks(const RankPieces& r, const float (&x)[kSumSteps][8], float (&sum)[2]) {
#pragma unroll
  for (int s = 0; s < kSumSteps; ++s)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float y[8];
      unpack8(r.w[s][k], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[k] = fmaf(x[s][e], y[e], sum[k]);
    }
}

}  // namespace
}  // namespace w8a8
