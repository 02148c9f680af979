// The int8 linear (and the gated pair of projections) for few tokens, from
// bf16 activations, in one launch: y = bf16(act(((acc*sx)*sw)+b)) with the
// codes and scales of quantize_rows and the same integer sums and epilogue
// arithmetic as the tiled kernel, so the result is the same bits as
// quantize + linear.
//
// Bound by reading the weight once (N*K bytes; the activations come from L2),
// below about 20 MB by the launch and the way through one group.  A workgroup
// of eight wavefronts takes 16 output channels (gated: 16 gate and the 16 up
// rows) at a time, each wavefront every eighth 128-byte piece of K.  A piece
// of 16 rows goes straight to the wavefront's own LDS ring (buffer_load ...
// lds, one to five pieces ahead, no barriers): a request then reads 128-byte
// runs of eight rows, and the workgroup 1 KB runs, where loads straight into
// the MFMA's register layout read 64-byte runs of sixteen rows (a plain read
// of 96 MB: 5.4 TB/s against 4.9).  16-byte chunks are XOR swizzled by row on
// the way in, so the fragment reads do not conflict.  The product is
// v_mfma_i32_16x16x64_i8 with weight rows as the first operand and the tokens'
// codes as the second; the partial sums of the wavefronts are exact int32 and
// are joined through LDS.
//
// Low-rank adapters: their shares t b^T of the workgroup's groups are made at
// the start, while the first pieces of the weight are on the way; for a single
// token or a short one so are t themselves, by every workgroup, which costs less
// than the launch that makes them for more tokens.
//
// Codes: up to kCodeBytes of them (one token of K = 22272, or five of 4096)
// are made by every workgroup for itself while its first pieces are on the
// way, and stay in LDS: one launch.  More tokens would make that the
// bottleneck (16 x 4096: 10 us of each workgroup), so quantize_rows makes them
// first, and they come through the ring beside the weight.
//
// Measured (cold weights, one call after another): 1 x 65536 x 4096 49 us, 5.5
// TB/s; 1 x 12288 x 4096 14 us; gated 1 x 12288 x 4096 21 us, 4.8 TB/s; 16
// x 12288 x 4096 14 us after 4 us for the codes.
#include "adapter_sum.h"
#include "epilogue.h"
#include "kernels.h"
#include "quant_codes.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kWave = 64;
constexpr int kRows = 16;            // output channels of a group
constexpr int kPiece = 128;          // bytes of K of a piece
constexpr int kPieceBytes = kRows * kPiece;
constexpr int kCodeBytes = 22 * 1024;
constexpr int kFewRank = 32;               // ranks of adapters whose first products are made here
constexpr uint32_t kOOB = 0x80000000u;    // buffer offset past any range: reads as zeros
constexpr int kRsrcWord3 = 0x00020000;

enum class FewAct { kNone, kGelu, kSiluGate, kGeluGate };

// Bytes of one token's codes in LDS: whole pieces, the row length an odd
// multiple of 16 bytes (16 lanes read the same chunk of 16 rows).
__host__ __device__ constexpr int64_t code_row(int64_t K) { return (K + kPiece - 1) / kPiece * kPiece + 16; }

template <int MT, FewAct ACT, bool kCodes, bool kLow = false>
struct Few {
  static constexpr bool kGate = ACT == FewAct::kSiluGate || ACT == FewAct::kGeluGate;
  static constexpr int NW = kGate ? 2 : 1;                 // weight rows per channel
  static constexpr int NV = NW * MT;                       // accumulators
  static constexpr int kTiles = NW + (kCodes ? MT : 0);    // 16-row tiles of a piece
  static constexpr int kDma = kPieceBytes / 1024 * kTiles; // requests per piece
  // (their pieces make 1 KB runs of a row: a plain read of 96 MB in that order
  // 5.4 TB/s, with four wavefronts 4.8)
  static constexpr int kWaves = 8;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kSlotBytes = kWaves * kTiles * kPieceBytes;
  static constexpr int kSlots = kTiles == 1 ? 6 : kTiles == 2 ? 4 : kTiles == 3 ? 3 : 2;   // as LDS allows
  static constexpr int kAhead = kThreads / (kRows * NW);   // groups whose scales are in LDS
  // Low-rank adapters: the tokens' shares of the workgroup's groups, fp32, made
  // before the first piece is needed.
  static constexpr int kLowGroup = MT * 16 * kRows * 4;   // bytes of a group
  static constexpr int kLowGroups = kLow ? (MT == 1 ? 24 : 4) : 0;
  // from bf16 activations: the adapters' first products too
  static constexpr int kLowT = kLow && !kCodes ? 16 * kFewRank * 2 : 0;
  static constexpr int kLds =
      kSlots * kSlotBytes + (kCodes ? 0 : kCodeBytes) + 12 * kThreads + 64 + kLowGroups * kLowGroup + kLowT;
  static_assert(kCodes || MT == 1, "codes in LDS are one tile of tokens");
  static_assert(!kLow || ACT == FewAct::kNone, "adapters beside the plain linear");
  static_assert(kLds <= 160 * 1024, "LDS budget");
  static_assert(NV * kWave * 16 <= kTiles * kPieceBytes, "a wavefront's sums fit its part of a slot");
};

template <int n>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  __builtin_amdgcn_sched_barrier(0);
}
// Barrier for LDS contents only: a __syncthreads() would also wait for the
// requests in flight.
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}
// LDS accesses in assembly: for ordinary ones the compiler waits for ring
// requests in flight that it cannot tell apart from them, so the ring would
// run empty at the end of every group.
// What a read needs waited for is waited for explicitly: the requests by
// wait_vmcnt() before it, its own data within the block; writes by the wait
// in barrier().
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void lds_write(uint32_t a, v4i v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(a), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_write(uint32_t a, u32x2 v) {
  asm volatile("ds_write_b64 %0, %1" ::"v"(a), "v"(v) : "memory");
}
__device__ __forceinline__ void lds_write(uint32_t a, uint32_t v) {
  asm volatile("ds_write_b32 %0, %1" ::"v"(a), "v"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds_read_word(uint32_t a) {
  uint32_t r;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(r) : "v"(a) : "memory");
  return r;
}
__device__ __forceinline__ u32x2 lds_read8(uint32_t a) {
  u32x2 r;
  asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(r) : "v"(a) : "memory");
  return r;
}
__device__ __forceinline__ v4i lds_read16(uint32_t a) {
  v4i r;
  asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(r) : "v"(a) : "memory");
  return r;
}
// 16 bytes at each of two and of four addresses
__device__ __forceinline__ void lds_read16x2(uint32_t a0, uint32_t a1, v4i* r) {
  asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(r[0]), "=&v"(r[1])
               : "v"(a0), "v"(a1)
               : "memory");
}
__device__ __forceinline__ void lds_read16x4(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, v4i* r) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
      : "v"(a0), "v"(a1), "v"(a2), "v"(a3)
      : "memory");
}

// Where 16-byte chunk c of row r of a piece lies in LDS: rows of 128 bytes,
// so that reads of one chunk of 16 rows fill all 256 bytes of banks.
__device__ __forceinline__ int swizzled(int r, int c) { return c ^ ((r >> 1) & 7); }

// Sixteen rows of a piece at K byte k0 into LDS: request i brings rows 8i ..
// 8i+7.  Lane p fills chunk p % 8 of row 8i + p / 8 with the chunk of that row
// that belongs there; chunks at or past K and rows past the range are zeros.
// kAux 2: non-temporal (the weight is read once).
template <int kAux>
__device__ __forceinline__ void request_tile(__amdgpu_buffer_rsrc_t r, int8_t* lds, int k0, int K, int lane) {
#pragma unroll
  for (int i = 0; i < kPieceBytes / 1024; ++i) {
    const int row = 8 * i + lane / 8, k = k0 + swizzled(row, lane % 8) * 16;
    const uint32_t o = k < K ? (uint32_t)(row * K + k) : kOOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + i * 1024), 16, (int)o, 0, 0, kAux);
  }
}

__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t o) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
}

// Maximum over the wavefront by DPP exchanges (a tenth of the latency of six
// trips through LDS): within fours, eights, sixteens, then across rows.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t wave_max_dpp(uint32_t v) {
  v = max(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
  v = max(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  v = max(v, dpp<0x141>(v));   // row_half_mirror
  v = max(v, dpp<0x140>(v));   // row_mirror
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// kCodes: the codes and scales come from memory (xq, sx); otherwise from x.
template <int MT, FewAct ACT, bool kCodes, bool kLow>
__global__ __launch_bounds__((Few<MT, ACT, kCodes, kLow>::kThreads)) void few_tokens_kernel(
    const uint16_t* __restrict__ x, const int8_t* __restrict__ xq, const float* __restrict__ sx,
    const int8_t* __restrict__ W, const float* __restrict__ sw, const uint16_t* __restrict__ bias,
    uint16_t* __restrict__ y, int M, int64_t N, int K, int groups, Low low) {
  using F = Few<MT, ACT, kCodes, kLow>;
  constexpr int NW = F::NW, S = F::kSlots, kWaves = F::kWaves, kThreads = F::kThreads;
  __shared__ __attribute__((aligned(16))) int8_t ring[S * F::kSlotBytes];
  __shared__ __attribute__((aligned(16))) int8_t codes[kCodes ? 16 : kCodeBytes];
  __shared__ float sx_lds[kThreads];
  __shared__ __attribute__((aligned(16))) float s_lds[kThreads], b_lds[kThreads];
  __shared__ __attribute__((aligned(16))) uint32_t amax_lds[8];
  __shared__ __attribute__((aligned(16))) float low_lds[kLow ? F::kLowGroups * F::kLowGroup / 4 : 4];
  __shared__ __attribute__((aligned(16))) uint16_t t_lds[kLow && !kCodes ? F::kLowT / 2 : 8];

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int l16 = lane % 16, h = lane / 16;
  const int pieces = (K + kPiece - 1) / kPiece;
  const int per = (pieces + kWaves - 1) / kWaves;   // pieces per wavefront and group (past the end: zeros)
  const int mine = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;   // groups of this workgroup
  const int items = mine * per;

  // Requests of the next item into a slot: the wavefront's pieces of each of
  // the workgroup's groups in turn, then nothing (zeros).
  int r_left = per, r_piece = wave;
  int64_t r_n0 = (int64_t)blockIdx.x * kRows;
  int r_items = items;
  int8_t* const my_ring = ring + wave * (F::kTiles * kPieceBytes);
  auto request = [&](int slot) {
    const bool there = r_items > 0;
    const int64_t n0 = r_n0;
    const int piece = r_piece;
    const int rows = there ? (int)min((int64_t)kRows, N - n0) : 0;
    --r_items;
    r_piece += kWaves;
    if (--r_left == 0) {
      r_left = per;
      r_piece = wave;
      r_n0 += (int64_t)gridDim.x * kRows;
    }
    int8_t* dst = my_ring + slot * F::kSlotBytes;
    auto range = [&](const int8_t* from, int bytes) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(from), (short)0, bytes, kRsrcWord3);
    };
#pragma unroll
    for (int i = 0; i < NW; ++i)
      request_tile<2>(range(W + (there ? (n0 + i * N) * K : 0), rows * K), dst + i * kPieceBytes, piece * kPiece, K, lane);
    if constexpr (kCodes) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
        request_tile<0>(range(xq + (int64_t)m * 16 * K, there ? min(16, M - m * 16) * K : 0),
                        dst + (NW + m) * kPieceBytes, piece * kPiece, K, lane);
    }
  };
  // Channel scales and biases of kAhead groups from gi on, into LDS: a load at
  // the end of each group would wait for the requests in flight there.
  auto scale_row = [&](int first) {
    const int64_t g = (int64_t)blockIdx.x + (int64_t)min(first + tid / (kRows * NW), mine - 1) * gridDim.x;
    return min(g * kRows + tid % kRows, N - 1) + (tid / kRows % NW) * N;
  };
  auto load_scales = [&](int first) {
    const int64_t n = scale_row(first);
    lds_write(lds_address(s_lds + tid), __float_as_uint(sw[n]));
    lds_write(lds_address(b_lds + tid), bias != nullptr ? (uint32_t)bias[n] << 16 : 0u);
  };

  // The small loads go first, so that waiting for them does not wait for the
  // first pieces as well (loads return in order).
  // wavefronts per token when making codes
  const int P = M == 1 ? kWaves : M == 2 ? kWaves / 2 : M <= 4 ? kWaves / 4 : 1;
  const int part = wave % P, nchunk = K / 8, stride = P * kWave;
  constexpr int kKeep = 2;   // chunks of 8 values a lane keeps in registers
  u32x4 v[kKeep];
  auto load_x = [&](int m) {   // zeros past the row, and past the last token
    const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x + (int64_t)min(m, M - 1) * K), (short)0,
                                                     m < M ? 2 * K : 0, kRsrcWord3);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) v[i] = buffer_load16(r, (uint32_t)(part * kWave + lane + i * stride) * 16u);
  };
  // (branch-free: a load under a condition is waited for where it ends)
  float token_scale = 0.0f;
  if constexpr (kCodes) token_scale = sx[min(tid, M - 1)];
  else load_x(wave / P);
  const int64_t n_first = scale_row(0);
  const float first_scale = sw[n_first];
  auto share_id = [&](int i) { return kLow ? low.ids[i / kRows % M] : 0; };
  [[maybe_unused]] int first_id = 0;
  if constexpr (kLow) first_id = share_id(min(tid, mine * M * kRows - 1));
  const uint16_t* const bias_or = bias != nullptr ? bias : reinterpret_cast<const uint16_t*>(sw);
  const uint32_t first_bias = bias_or[n_first];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int s = 0; s + 1 < S; ++s) request(s);
  __builtin_amdgcn_sched_barrier(0);
  lds_write(lds_address(s_lds + tid), __float_as_uint(first_scale));
  lds_write(lds_address(b_lds + tid), bias != nullptr ? first_bias << 16 : 0u);
  if constexpr (kCodes) lds_write(lds_address(sx_lds + tid), __float_as_uint(token_scale));

  // Adapters' shares: a thread for a token and a channel of one of this
  // workgroup's groups (neighbouring threads: neighbouring rows of b).  The
  // first one's rows are on the way while the codes and t are made.
  constexpr int kSharePieces = kLow ? 2 : 1;   // of 8 ranks at a time
  [[maybe_unused]] const int low_all = kLow ? mine * M * kRows : 0;
  [[maybe_unused]] const uint16_t *share_b = nullptr, *share_row = nullptr;
  [[maybe_unused]] u32x4 share_w[kSharePieces], share_t[kSharePieces];
  [[maybe_unused]] bool share_on = false;
  auto load_ranks_of_share = [&](int r) __attribute__((always_inline)) {
    // (branch-free: ranks past the last are not used)
#pragma unroll
    for (int p = 0; p < kSharePieces; ++p) {
      const int at = min(r + 8 * p, (int)low.R - 8);
      share_w[p] = *reinterpret_cast<const u32x4*>(share_b + at);
      if constexpr (kCodes) share_t[p] = *reinterpret_cast<const u32x4*>(share_row + at);
    }
  };
  auto load_share = [&](int i, int id) __attribute__((always_inline)) {
    const int64_t n = min(((int64_t)blockIdx.x + (int64_t)(i / kRows / M) * gridDim.x) * kRows + i % kRows, N - 1);
    share_on = id >= 0 && id < low.count;
    share_b = low.b + ((share_on ? id : 0) * N + n) * low.R;
    if constexpr (kCodes) share_row = low.t + i / kRows % M * low.ldt;
    load_ranks_of_share(0);
  };
  if constexpr (kLow) load_share(min(tid, low_all - 1), first_id);

  // Adapters from bf16 activations: a wavefront takes a token and two ranks at a
  // time, as the first product's own kernel does; its first pieces are on the
  // way while the codes are made.
  [[maybe_unused]] RankPieces ranks;
  [[maybe_unused]] RankRows rank_rows(nullptr, 0, 0, false);
  [[maybe_unused]] int rank_id = -1;
  [[maybe_unused]] const int pairs = kLow && !kCodes ? (int)low.R / 2 : 1, eighths = K / 8;
  auto start_pair = [&](int i) __attribute__((always_inline)) {
    rank_id = low.ids[i / pairs];
    if (rank_id >= low.count) rank_id = -1;
    rank_rows = RankRows(low.a + ((int64_t)max(rank_id, 0) * low.R + i % pairs * 2) * K, K, eighths, rank_id >= 0);
    rank_rows.load(lane, ranks);
  };
  if constexpr (kLow && !kCodes) start_pair(min(wave, M * pairs - 1));

  if constexpr (!kCodes) {
    // ---- the tokens' codes ----
    const int64_t row_bytes = code_row(K);
    for (int m = wave / P; m < M; m += kWaves / P) {
      const u32x4* xr = reinterpret_cast<const u32x4*>(x + (int64_t)m * K);
      uint32_t mx = 0;
      if (m >= kWaves / P) load_x(m);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = absmax_bits(mx, v[i][e]);
      for (int c = part * kWave + lane + kKeep * stride; c < nchunk; c += stride) {
        const u32x4 z = xr[c];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = absmax_bits(mx, z[e]);
      }
      mx = wave_max_dpp(max(mx & 0xffffu, mx >> 16));
      if (P > 1) {
        // every wavefront comes here exactly once (those of a fourth token
        // slot with three tokens below)
        if (lane == 0) lds_write(lds_address(amax_lds + wave), mx);
        barrier();
        v4i all[2];
        lds_read16x2(lds_address(amax_lds), lds_address(amax_lds + 4), all);
#pragma unroll
        for (int q = 0; q < kWaves; ++q)
          if (q / P == wave / P) mx = max(mx, (uint32_t)all[q / 4][q % 4]);
      }
      const RowScale rs = row_scale<false>(mx);
      const uint32_t row = lds_address(codes) + (uint32_t)(m * row_bytes);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int c = part * kWave + lane + i * stride;
        if (c < nchunk) lds_write(row + c * 8, mx ? quant_chunk<false>(v[i], rs.xs, rs.ss, rs.r) : u32x2{0, 0});
      }
      for (int c = part * kWave + lane + kKeep * stride; c < nchunk; c += stride)
        lds_write(row + c * 8, mx ? quant_chunk<false>(xr[c], rs.xs, rs.ss, rs.r) : u32x2{0, 0});
      const int c = nchunk + lane;   // zeros up to whole pieces
      if (part == 0 && c * 8 < pieces * kPiece) lds_write(row + c * 8, u32x2{0, 0});
      if (part == 0 && lane == 0) lds_write(lds_address(sx_lds + m), __float_as_uint(mx ? rs.s : 0.0f));
    }
    if (P > 1 && wave / P >= M) barrier();
  }
  if constexpr (kLow && !kCodes) {
    barrier();   // the codes and scales are there
    for (int i = wave; i < M * pairs; i += kWaves) {
      if (i > wave) start_pair(i);
      const int m = i / pairs;
      float sum[2] = {0.0f, 0.0f};
      if (rank_id >= 0) {
        const uint32_t row = lds_address(codes) + (uint32_t)(m * code_row(K));
        for (int c0 = lane; c0 < eighths; c0 += kSumSteps * kWave) {
          if (c0 > lane) rank_rows.load(c0, ranks);
          float v[kSumSteps][8];
#pragma unroll
          for (int s = 0; s < kSumSteps; ++s) {
            const int c = c0 + s * kWave;
            const u32x2 q = lds_read8(row + (uint32_t)min(c, eighths - 1) * 8);   // (past the row: times zeros)
            codes4(q[0], v[s]);
            codes4(q[1], v[s] + 4);
          }
          add_ranks(ranks, v, sum);
        }
        const float sa = __uint_as_float(lds_read_word(lds_address(sx_lds + m))), f = low.scaling[rank_id];
#pragma unroll
        for (int k = 0; k < 2; ++k) sum[k] = sum_lanes(sum[k]) * sa * f;
      }
      if (lane == 0)
        lds_write(lds_address(t_lds + m * kFewRank + i % pairs * 2),
                  __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{sum[0], sum[1]}), bf16x2)));
    }
    barrier();
  }
  if constexpr (kLow) {
    for (int i = tid; i < low_all; i += kThreads) {
      if (i > tid) load_share(i, share_id(i));
      float v = 0.0f;
      if (share_on) {
        for (int r = 0; r < (int)low.R; r += 8 * kSharePieces) {
          if (r > 0) load_ranks_of_share(r);
#pragma unroll
          for (int p = 0; p < kSharePieces; ++p) {
            if (r + 8 * p >= (int)low.R) continue;
            u32x4 tv;
            if constexpr (kCodes) tv = share_t[p];
            else tv = __builtin_bit_cast(u32x4, lds_read16(lds_address(t_lds + i / kRows % M * kFewRank + r + 8 * p)));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v = fmaf(__uint_as_float(tv[e] << 16), __uint_as_float(share_w[p][e] << 16), v);
              v = fmaf(__uint_as_float(tv[e] & 0xffff0000u), __uint_as_float(share_w[p][e] & 0xffff0000u), v);
            }
          }
        }
      }
      lds_write(lds_address(low_lds + (i / kRows / M * MT * 16 + i / kRows % M) * kRows + i % kRows), __float_as_uint(v));
    }
  }
  barrier();

  v4i acc[NW][MT];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[i][t] = v4i{0, 0, 0, 0};
  };
  clear();

  // The last piece of this workgroup's group gi is done: join the sums, each
  // wavefront's in its part of the slot just read (free until the next
  // request); one wavefront per 16 tokens writes them, in turn.
  int turn = 0;
  auto finish = [&](int gi, int slot) {
    const int64_t g = (int64_t)blockIdx.x + (int64_t)gi * gridDim.x;
    if (gi > 0 && gi % F::kAhead == 0) load_scales(gi);
    const uint32_t sums = lds_address(ring) + (uint32_t)(slot * F::kSlotBytes + lane * 16);
    constexpr uint32_t kPart = F::kTiles * kPieceBytes;
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t) lds_write(sums + (uint32_t)wave * kPart + (i * MT + t) * kWave * 16, acc[i][t]);
    barrier();
    const int mine_t = (wave - turn) & (kWaves - 1);
    turn += MT;
    const int tok = mine_t * 16 + l16;
    v4i sum[NW];
    f32x4 swv[NW], bv[NW];
    [[maybe_unused]] f32x4 lowv;
    float sa = 0.0f;
    if (mine_t < MT) {
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint32_t a = sums + (uint32_t)(i * MT + mine_t) * kWave * 16;
        v4i r[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; w += 4)
          lds_read16x4(a + w * kPart, a + (w + 1) * kPart, a + (w + 2) * kPart, a + (w + 3) * kPart, r + w);
        sum[i] = r[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum[i] += r[w];
        const int e0 = (gi % F::kAhead * NW + i) * kRows + 4 * h;
        swv[i] = __builtin_bit_cast(f32x4, lds_read16(lds_address(s_lds + e0)));
        bv[i] = __builtin_bit_cast(f32x4, lds_read16(lds_address(b_lds + e0)));
      }
      sa = __uint_as_float(lds_read_word(lds_address(sx_lds + tok)));
      if constexpr (kLow)
        lowv = __builtin_bit_cast(f32x4, lds_read16(lds_address(low_lds + (gi * MT * 16 + tok) * kRows + 4 * h)));
    }
    barrier();   // read: the slot may be requested again, the scales replaced
    if (mine_t < MT) {
      const int64_t n0 = g * kRows + 4 * h;   // this lane's channels
      if (tok < M) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = dequant((float)sum[0][e], sa, swv[0][e], bv[0][e]);
          if constexpr (kLow) v += lowv[e];
          if constexpr (ACT == FewAct::kGelu) v = gelu(v);
          if constexpr (F::kGate) {
            const float up = dequant((float)sum[NW - 1][e], sa, swv[NW - 1][e], bv[NW - 1][e]);
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
    clear();
  };

  int left = per;      // pieces of the current group still to come
  int gi = 0, slot = 0;
  uint32_t chunk[2];   // this lane's fragments of a 16-row tile
#pragma unroll
  for (int k = 0; k < 2; ++k) chunk[k] = lds_address(my_ring) + (uint32_t)(l16 * kPiece + swizzled(l16, 4 * k + h) * 16);
  for (int t = 0; t < items; ++t) {
    // the slot read one item ago takes the piece S - 1 items ahead (past the
    // end: zeros, which keeps the count below)
    request(slot == 0 ? S - 1 : slot - 1);
    wait_vmcnt<(S - 1) * F::kDma>();   // item t has landed
    const uint32_t base = (uint32_t)(slot * F::kSlotBytes);
    auto read = [&](int tile, v4i* f) {
      const uint32_t o = base + (uint32_t)(tile * kPieceBytes);
      lds_read16x2(chunk[0] + o, chunk[1] + o, f);
    };
    v4i w[NW][2], c[MT][2];
#pragma unroll
    for (int i = 0; i < NW; ++i) read(i, w[i]);
    if constexpr (kCodes) {
#pragma unroll
      for (int m = 0; m < MT; ++m) read(NW + m, c[m]);
    } else {
      const int at = min(wave + kWaves * (per - left), pieces - 1) * kPiece;
      const uint32_t a = lds_address(codes) + (uint32_t)(min(l16, M - 1) * (int)code_row(K) + at + h * 16);
      lds_read16x2(a, a + 64, c[0]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NW; ++i) acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i][k], c[m][k], acc[i][m], 0, 0, 0);
    if (--left == 0) {
      finish(gi++, slot);
      left = per;
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  wait_vmcnt<0>();   // no request may write LDS after the workgroup ends
}

template <int MT, FewAct ACT, bool kCodes, bool kLow = false>
hipError_t launch(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                  const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t stream,
                  const Low& low = Low{}) {
  const int64_t groups = (N + kRows - 1) / kRows;
  const int64_t grid = std::min<int64_t>(groups, 256);   // one workgroup per compute unit
  hipLaunchKernelGGL((few_tokens_kernel<MT, ACT, kCodes, kLow>), dim3((unsigned)grid),
                     dim3(Few<MT, ACT, kCodes, kLow>::kThreads), 0, stream, x, xq, sx, wq, sw, bias, y, (int)M, N, (int)K,
                     (int)groups, low);
  return hipGetLastError();
}

template <FewAct ACT>
hipError_t launch_act(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                      const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (xq == nullptr) return launch<1, ACT, false>(x, xq, sx, wq, sw, bias, y, M, N, K, s);
  return M <= 16 ? launch<1, ACT, true>(x, xq, sx, wq, sw, bias, y, M, N, K, s)
                 : launch<2, ACT, true>(x, xq, sx, wq, sw, bias, y, M, N, K, s);
}

}  // namespace

// Where every workgroup makes the first products for itself: the codes fit LDS,
// and the adapters' rows that each has to read, two at a time by a wavefront, take
// less than a launch.  Cold weights, us so / in two launches, 2048 channels: 1 token
// of K = 2048, rank 16 8.5 / 10.1, rank 32 9.4 / 10.2, rank 64 12.4 / 9.8; K = 4096,
// rank 16 10.1 / 10.7, rank 32 11.7 / 10.8; 2 tokens of 2048, rank 16 9.7 / 10.7; 4,
// rank 8 9.2 / 10.3; 4 of 1024, rank 16 11.8 / 9.7.  8192 channels: 1 token, rank 16,
// K = 1024 9.0 / 10.5, 2048 10.8 / 10.4, 4096 14.4 / 14.7; 2 tokens of 2048 11.4 /
// 10.7; 4, rank 8 11.9 / 10.3.
bool few_tokens_low_from_x(int64_t M, int64_t N, int64_t K, int64_t R) {
  return few_tokens_in_lds(M, K) && M * R <= (N <= 4096 ? kFewRank : kFewRank / 2) && M * R * K <= 65536 &&
         few_tokens_low_fit(M, N);
}

hipError_t launch_few_tokens_low_from_x(const uint16_t* x, const int8_t* wq, const float* sw, const uint16_t* bias,
                                        const Low& low, uint16_t* y, int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (M < 1 || !few_tokens_low_from_x(M, N, K, low.R)) return hipErrorInvalidValue;
  return launch<1, FewAct::kNone, false, true>(x, nullptr, nullptr, wq, sw, bias, y, M, N, K, s, low);
}

bool few_tokens_low_fit(int64_t M, int64_t N) {
  const int64_t groups = (N + kRows - 1) / kRows, per = (groups + 255) / 256;
  return per <= (M <= 16 ? Few<1, FewAct::kNone, true, true>::kLowGroups : Few<2, FewAct::kNone, true, true>::kLowGroups);
}

hipError_t launch_few_tokens_low(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                 const uint16_t* bias, const Low& low, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                 hipStream_t s) {
  if (M < 1 || M > kFewTokens || !few_tokens_low_fit(M, N)) return hipErrorInvalidValue;
  return M <= 16 ? launch<1, FewAct::kNone, true, true>(nullptr, xq, sx, wq, sw, bias, y, M, N, K, s, low)
                 : launch<2, FewAct::kNone, true, true>(nullptr, xq, sx, wq, sw, bias, y, M, N, K, s, low);
}

bool few_tokens_in_lds(int64_t M, int64_t K) { return M <= 16 && M * code_row(K) <= kCodeBytes; }

hipError_t launch_few_tokens(const uint16_t* x, const int8_t* xq, const float* sx, const int8_t* wq,
                             const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                             int64_t K, int act, bool gated, hipStream_t stream) {
  if (M < 1 || M > kFewTokens || (xq == nullptr && !few_tokens_in_lds(M, K))) return hipErrorInvalidValue;
  if (gated)
    return act == static_cast<int>(GateAct::kGelu)
               ? launch_act<FewAct::kGeluGate>(x, xq, sx, wq, sw, bias, y, M, N, K, stream)
               : launch_act<FewAct::kSiluGate>(x, xq, sx, wq, sw, bias, y, M, N, K, stream);
  return act ? launch_act<FewAct::kGelu>(x, xq, sx, wq, sw, bias, y, M, N, K, stream)
             : launch_act<FewAct::kNone>(x, xq, sx, wq, sw, bias, y, M, N, K, stream);
}

}  // namespace w8a8
