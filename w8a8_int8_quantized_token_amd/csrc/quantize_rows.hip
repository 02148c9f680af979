// Per-row absmax int8 quantizer for gfx950: per-token activation quantization
// and per-output-channel weight quantization, as in the abstract of
// "Realizing Native INT8 Compute for Diffusion Transformers on Consumer GPUs"
// (arXiv 2606.14598), with the readings s = fl32(amax/127) and
// q = clamp(rne(fl32(x/s)), -127, 127); an all-zero row gives s = 0, q = 0.
//
// One wavefront owns one row.  The row is read once from HBM with 16-byte
// loads (8 bf16 per lane per load) and kept in registers; the absmax is a
// packed 16-bit integer max over the magnitude bits (for finite bf16 the
// order of |x| equals the order of its bits) followed by a wavefront
// butterfly; the codes are then produced from the registers and written with
// 8-byte stores.  HBM traffic is the algorithmic 3 bytes per element plus
// 4 bytes per row.
//
// The fp8 variant (F8) is the same kernel with s = fl32(amax/448) and codes
// e4m3(fl32(x/s)) (OCP e4m3: nearest, ties to even, largest value 448)
// produced by v_cvt_pk_fp8_f32; the same exhaustive check covers its codes.
#include "kernels.h"
#include "quant_codes.h"

namespace w8a8 {
namespace {

constexpr int kWave = 64;
constexpr int kRowsPerBlock = 4;
constexpr int kThreads = kWave * kRowsPerBlock;

// Row resident in registers: CPL 16-byte chunks per lane, K <= CPL*8*64.
template <int CPL, bool F8>
__global__ __launch_bounds__(kThreads) void quantize_rows_reg(const u32x4* __restrict__ x,
                                                              u32x2* __restrict__ q,
                                                              float* __restrict__ scale,
                                                              int64_t R, int nchunk) {
  const int lane = threadIdx.x % kWave;
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / kWave;
  if (row >= R) return;  // whole wavefront leaves together
  const u32x4* xr = x + row * nchunk;
  u32x2* qr = q + row * nchunk;

  u32x4 v[CPL];
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = lane + i * kWave;
    v[i] = c < nchunk ? __builtin_nontemporal_load(xr + c) : u32x4{0, 0, 0, 0};
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    m = absmax_bits(m, v[i].x);
    m = absmax_bits(m, v[i].y);
    m = absmax_bits(m, v[i].z);
    m = absmax_bits(m, v[i].w);
  }
  m = max(m & 0xffffu, m >> 16);
  m = wave_max(m);

  if (m == 0) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const int c = lane + i * kWave;
      if (c < nchunk) qr[c] = u32x2{0, 0};
    }
    if (lane == 0) scale[row] = 0.0f;
    return;
  }
  const RowScale rs = row_scale<F8>(m);
#pragma unroll
  for (int i = 0; i < CPL; ++i) {
    const int c = lane + i * kWave;
    if (c < nchunk) qr[c] = quant_chunk<F8>(v[i], rs.xs, rs.ss, rs.r);
  }
  if (lane == 0) scale[row] = rs.s;
}

// Any K: two passes over the row (the second one mostly from cache).
template <bool F8>
__global__ __launch_bounds__(kThreads) void quantize_rows_2pass(const u32x4* __restrict__ x,
                                                                u32x2* __restrict__ q,
                                                                float* __restrict__ scale,
                                                                int64_t R, int nchunk) {
  const int lane = threadIdx.x % kWave;
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / kWave;
  if (row >= R) return;
  const u32x4* xr = x + row * nchunk;
  u32x2* qr = q + row * nchunk;
  uint32_t m = 0;
  for (int c = lane; c < nchunk; c += kWave) {
    u32x4 v = xr[c];
    m = absmax_bits(m, v.x);
    m = absmax_bits(m, v.y);
    m = absmax_bits(m, v.z);
    m = absmax_bits(m, v.w);
  }
  m = max(m & 0xffffu, m >> 16);
  m = wave_max(m);
  if (m == 0) {
    for (int c = lane; c < nchunk; c += kWave) qr[c] = u32x2{0, 0};
    if (lane == 0) scale[row] = 0.0f;
    return;
  }
  const RowScale rs = row_scale<F8>(m);
  for (int c = lane; c < nchunk; c += kWave) qr[c] = quant_chunk<F8>(xr[c], rs.xs, rs.ss, rs.r);
  if (lane == 0) scale[row] = rs.s;
}

template <int CPL, bool F8>
hipError_t launch_reg(const uint16_t* x, int8_t* q, float* s, int64_t R, int nchunk,
                      hipStream_t st) {
  const int64_t blocks = (R + kRowsPerBlock - 1) / kRowsPerBlock;
  hipLaunchKernelGGL((quantize_rows_reg<CPL, F8>), dim3((unsigned)blocks), dim3(kThreads), 0, st,
                     reinterpret_cast<const u32x4*>(x), reinterpret_cast<u32x2*>(q), s, R, nchunk);
  return hipGetLastError();
}

template <bool F8>
hipError_t launch_rows(const uint16_t* x, int8_t* q, float* scale, int64_t R, int64_t K,
                       hipStream_t stream) {
  const int nchunk = (int)(K / 8);          // 16-byte chunks per row
  const int cpl = (nchunk + kWave - 1) / kWave;
  if (cpl <= 1) return launch_reg<1, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 2) return launch_reg<2, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 4) return launch_reg<4, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 6) return launch_reg<6, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 8) return launch_reg<8, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 12) return launch_reg<12, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 16) return launch_reg<16, F8>(x, q, scale, R, nchunk, stream);
  if (cpl <= 24) return launch_reg<24, F8>(x, q, scale, R, nchunk, stream);
  const int64_t blocks = (R + kRowsPerBlock - 1) / kRowsPerBlock;
  hipLaunchKernelGGL((quantize_rows_2pass<F8>), dim3((unsigned)blocks), dim3(kThreads), 0, stream,
                     reinterpret_cast<const u32x4*>(x), reinterpret_cast<u32x2*>(q), scale, R,
                     nchunk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const uint16_t* x, int8_t* q, float* scale, int64_t R, int64_t K,
                                hipStream_t stream) {
  return launch_rows<false>(x, q, scale, R, K, stream);
}

hipError_t launch_quantize_rows_fp8(const uint16_t* x, uint8_t* q, float* scale, int64_t R,
                                    int64_t K, hipStream_t stream) {
  return launch_rows<true>(x, reinterpret_cast<int8_t*>(q), scale, R, K, stream);
}

}  // namespace w8a8
