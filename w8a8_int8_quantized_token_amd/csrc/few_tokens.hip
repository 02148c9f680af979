// The int8 linear (and the gated pair of projections) for few tokens, from
// bf16 activations, in one launch: y = bf16(act(((acc*sx)*sw)+b)) with the
// codes and scales of quantize_rows and the same integer sums and epilogue
// arithmetic as the tiled kernel, so the result is the same bits as
// quantize + linear.
//
// Bound by reading the weight once (N*K bytes; the activations, M*K*2 bytes,
// come from L2).  A workgroup of eight wavefronts takes 16 output channels
// (gated: 16 gate and the 16 up rows) at a time; the wavefronts share K, each
// taking 128-byte pieces of the 16 rows in turn, so a workgroup reads 1 KB
// runs of each row.  The product is v_mfma_i32_16x16x64_i8 with weight rows as
// the first operand, whose register layout (16 consecutive K bytes of one row
// per lane) is what a 16-byte load brings: weights never pass through LDS.
// The tokens' codes are the second operand.  They are made by every workgroup
// for itself (its first weight loads are in flight meanwhile) and stay in LDS;
// where they do not fit, quantize_rows makes them first and the lanes load
// them from L2.  The eight partial sums are exact int32 and are joined through
// LDS.
#include "epilogue.h"
#include "kernels.h"
#include "quant_codes.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWave = 64;
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kRows = 16;          // output channels of a group
constexpr int kPairs = 4;          // 128-byte pieces a wavefront has in flight
constexpr int kLds = 160 * 1024;
constexpr int kSkew = 16;          // LDS rows start 4 banks apart

enum class FewAct { kNone, kGelu, kSiluGate, kGeluGate };

// Bytes of one token's codes in LDS: whole 64-byte steps, the row length an
// odd multiple of 16 bytes (16 lanes read the same step of 16 rows).
__host__ __device__ constexpr int64_t code_row(int64_t K) {
  return (K + 63) / 64 * 64 + kSkew;
}
constexpr int red_bytes(int nv) { return kWaves * nv * kWave * 16; }

// kCodes: the codes and scales come from memory (xq, sx); otherwise from x.
template <int MT, FewAct ACT, bool kCodes>
__global__ __launch_bounds__(kThreads) void few_tokens_kernel(
    const uint16_t* __restrict__ x, const int8_t* __restrict__ xq, const float* __restrict__ sx,
    const int8_t* __restrict__ W, const float* __restrict__ sw, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ y, int M, int64_t N, int K, int groups) {
  constexpr bool kGate = ACT == FewAct::kSiluGate || ACT == FewAct::kGeluGate;
  constexpr int NW = kGate ? 2 : 1;      // weight rows per channel
  constexpr int NV = NW * MT;            // accumulators
  extern __shared__ __attribute__((aligned(16))) int8_t lds[];
  v4i* const red = reinterpret_cast<v4i*>(lds);                                  // [wave][v][lane]
  float* const sx_lds = reinterpret_cast<float*>(lds + red_bytes(NV));           // [32]
  uint32_t* const amax_lds = reinterpret_cast<uint32_t*>(sx_lds + 32);           // [4][8]
  int8_t* const codes = reinterpret_cast<int8_t*>(amax_lds + 32);
  const int64_t row_bytes = code_row(K);

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l16 = lane % 16, h = lane / 16;
  const int steps = (K + 63) / 64;
  const int rounds = ((steps + 1) / 2 + kWaves * kPairs - 1) / (kWaves * kPairs);

  // Weight pieces of round r of group g (and, with kCodes, the tokens').
  // Steps past the end are not loaded; the last step's bytes past K repeat
  // the row's last 16, against codes that are zero there.
  struct Piece {
    v4i w[NW][2 * kPairs];
    v4i c[kCodes ? MT : 1][2 * kPairs];
  };
  auto step_of = [&](int r, int u) { return 2 * (wave + kWaves * (r * kPairs + u / 2)) + u % 2; };
  auto load = [&](Piece& p, int g, int r) {
    const int64_t n = min((int64_t)g * kRows + l16, N - 1);
#pragma unroll
    for (int u = 0; u < 2 * kPairs; ++u) {
      const int s = step_of(r, u);
      if (s < steps) {
        const int k = min(s * 64 + h * 16, K - 16);
#pragma unroll
        for (int i = 0; i < NW; ++i)
          p.w[i][u] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(W + (n + i * N) * K + k));
        if constexpr (kCodes) {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const int tok = min(t * 16 + l16, M - 1);
            p.c[t][u] = *reinterpret_cast<const v4i*>(xq + (int64_t)tok * K + k);
            if (s * 64 + h * 16 >= K) p.c[t][u] = v4i{0, 0, 0, 0};
          }
        }
      }
    }
  };

  Piece cur;
  int g = blockIdx.x;
  load(cur, g, 0);

  if constexpr (kCodes) {
    if (tid < M) sx_lds[tid] = sx[tid];
  } else {
    // ---- the tokens' codes: P wavefronts per token ----
    const int P = M == 1 ? 8 : M == 2 ? 4 : M <= 4 ? 2 : 1;
    const int part = wave % P, nchunk = K / 8, stride = P * kWave;
    constexpr int kKeep = 4;   // chunks of 8 values a lane keeps in registers
    for (int m = wave / P; m < M; m += kWaves / P) {
      const u32x4* xr = reinterpret_cast<const u32x4*>(x + (int64_t)m * K);
      u32x4 v[kKeep];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int c = part * kWave + lane + i * stride;
        v[i] = c < nchunk ? xr[c] : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = absmax_bits(mx, v[i][e]);
      for (int c = part * kWave + lane + kKeep * stride; c < nchunk; c += stride) {
        const u32x4 z = xr[c];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = absmax_bits(mx, z[e]);
      }
      mx = wave_max(max(mx & 0xffffu, mx >> 16));
      if (P > 1) {
        // M <= 4: every wavefront comes here exactly once
        if (lane == 0) amax_lds[(wave / P) * kWaves + part] = mx;
        __syncthreads();
        for (int q = 0; q < P; ++q) mx = max(mx, amax_lds[(wave / P) * kWaves + q]);
      }
      const RowScale rs = row_scale<false>(mx);
      int8_t* const row = codes + m * row_bytes;
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int c = part * kWave + lane + i * stride;
        if (c < nchunk)
          *reinterpret_cast<u32x2*>(row + c * 8) = mx ? quant_chunk<false>(v[i], rs.xs, rs.ss, rs.r) : u32x2{0, 0};
      }
      for (int c = part * kWave + lane + kKeep * stride; c < nchunk; c += stride)
        *reinterpret_cast<u32x2*>(row + c * 8) = mx ? quant_chunk<false>(xr[c], rs.xs, rs.ss, rs.r) : u32x2{0, 0};
      const int c = nchunk + lane;   // zeros up to whole steps
      if (part == 0 && c * 8 < steps * 64) *reinterpret_cast<u32x2*>(row + c * 8) = u32x2{0, 0};
      if (part == 0 && lane == 0) sx_lds[m] = mx ? rs.s : 0.0f;
    }
    // M == 3: the wavefronts of the fourth token slot take part in the
    // barrier of the reduction above
    if (P == 2 && wave / P >= M) __syncthreads();
  }
  __syncthreads();

  for (; g < groups; g += gridDim.x) {
    v4i acc[NW][MT];
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][t] = v4i{0, 0, 0, 0};

    for (int r = 0; r < rounds; ++r) {
      Piece nxt;
      const bool more = r + 1 < rounds;
      const int ng = more ? g : g + (int)gridDim.x;
      if (ng < groups) load(nxt, ng, more ? r + 1 : 0);
#pragma unroll
      for (int u = 0; u < 2 * kPairs; ++u) {
        const int s = step_of(r, u);
        if (s < steps) {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            v4i c;
            if constexpr (kCodes) c = cur.c[t][u];
            else c = *reinterpret_cast<const v4i*>(codes + min(t * 16 + l16, M - 1) * row_bytes + s * 64 + h * 16);
#pragma unroll
            for (int i = 0; i < NW; ++i) acc[i][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(cur.w[i][u], c, acc[i][t], 0, 0, 0);
          }
        }
      }
      cur = nxt;
    }

    // ---- join the eight sums; one wavefront per 16 tokens writes them ----
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t) red[(wave * NV + i * MT + t) * kWave + lane] = acc[i][t];
    __syncthreads();
    if (wave < MT) {
      v4i sum[NW];
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        sum[i] = v4i{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum[i] += red[(w * NV + i * MT + wave) * kWave + lane];
      }
      const int tok = wave * 16 + l16;
      if (tok < M) {
        const float sa = sx_lds[tok];
        const int64_t n0 = (int64_t)g * kRows + 4 * h;
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t n = min(n0 + e, N - 1);
          float v = dequant((float)sum[0][e], sa, sw[n], bias ? __uint_as_float((uint32_t)bias[n] << 16) : 0.0f);
          if constexpr (ACT == FewAct::kGelu) v = gelu(v);
          if constexpr (kGate) {
            const float up = dequant((float)sum[NW - 1][e], sa, sw[N + n],
                                     bias ? __uint_as_float((uint32_t)bias[N + n] << 16) : 0.0f);
            v = (ACT == FewAct::kGeluGate ? gelu(v) : silu(v)) * up;
          }
          o[e] = v;
        }
        const uint32_t lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{o[0], o[1]}), bf16x2));
        const uint32_t hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{o[2], o[3]}), bf16x2));
        uint16_t* out = y + (int64_t)tok * N + n0;
        if (n0 + 3 < N && reinterpret_cast<uintptr_t>(out) % 8 == 0) {
          *reinterpret_cast<u32x2*>(out) = u32x2{lo, hi};
        } else {
          const uint16_t b[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n0 + e < N) out[e] = b[e];
        }
      }
    }
    __syncthreads();
  }
}

// LDS of a launch whose codes are made in it.
int64_t lds_bytes(int64_t M, int64_t K, int nv) { return red_bytes(nv) + 256 + M * code_row(K); }

template <int MT, FewAct ACT, bool kCodes>
hipError_t launch(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                  const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  constexpr int NV = (ACT == FewAct::kSiluGate || ACT == FewAct::kGeluGate ? 2 : 1) * MT;
  const int64_t lds = kCodes ? red_bytes(NV) + 256 : lds_bytes(M, K, NV);
  const int64_t groups = (N + kRows - 1) / kRows;
  const int64_t resident = lds <= kLds / 2 ? 512 : 256;
  const auto kern = few_tokens_kernel<MT, ACT, kCodes>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)std::min(groups, resident)), dim3(kThreads), (size_t)lds, stream, x, xq,
                     sx, wq, sw, bias, y, (int)M, N, (int)K, (int)groups);
  return hipGetLastError();
}

template <FewAct ACT>
hipError_t launch_act(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                      const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (xq != nullptr)
    return M <= 16 ? launch<1, ACT, true>(x, xq, sx, wq, sw, bias, y, M, N, K, s)
                   : launch<2, ACT, true>(x, xq, sx, wq, sw, bias, y, M, N, K, s);
  return M <= 16 ? launch<1, ACT, false>(x, xq, sx, wq, sw, bias, y, M, N, K, s)
                 : launch<2, ACT, false>(x, xq, sx, wq, sw, bias, y, M, N, K, s);
}

}  // namespace

bool few_tokens_in_lds(int64_t M, int64_t K, bool gated) {
  return lds_bytes(M, K, (gated ? 2 : 1) * (M <= 16 ? 1 : 2)) <= kLds;
}

hipError_t launch_few_tokens(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq,
                             const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, int act, bool gated, hipStream_t stream) {
  if (M < 1 || M > kFewTokens || (xq == nullptr && !few_tokens_in_lds(M, K, gated))) return hipErrorInvalidValue;
  if (gated)
    return act == static_cast<int>(GateAct::kGelu)
               ? launch_act<FewAct::kGeluGate>(x, xq, sx, wq, sw, bias, y, M, N, K, stream)
               : launch_act<FewAct::kSiluGate>(x, xq, sx, wq, sw, bias, y, M, N, K, stream);
  return act ? launch_act<FewAct::kGelu>(x, xq, sx, wq, sw, bias, y, M, N, K, stream)
             : launch_act<FewAct::kNone>(x, xq, sx, wq, sw, bias, y, M, N, K, stream);
}

}  // namespace w8a8
