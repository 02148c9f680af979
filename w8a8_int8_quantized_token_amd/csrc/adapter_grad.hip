// Gradients of the low-rank adapters' two matrices: for each adapter i, over its
// rows m (tokens),
//   out[i][r, c] = sum_m v[m, r] x[m, c],
// v [M, ldt] (t or u, which have the scalings), x the activations' codes (v then
// has their scales too) or the output's gradient in bf16.  fp32 sums on the bf16
// matrix cores.
//
// x is exact in bf16; v comes in two bf16 parts, each multiplied by the same
// fragment of x.  Rounded to one part, v would be off by up to 2^-8 in each term,
// and that error grows with the sum as the sum itself does, so that a gradient
// of any number of rows had 1.4 times the error of its own rounding (relative
// error 2.4e-3 and not 1.7e-3).  The second part costs nothing up to rank 32
// and 13 us of 131 at 8192 rows of 4096 and 8192, rank 64.
//
// The rows of an adapter come as a list (`lists`, made beside the operands'
// layout), so ids may be in any order; a row's values lie together, and only
// the row's address is looked up.
//
// Bound by reading x once.  A wavefront takes 32 rows of the list at a time and
// 16 * KB columns: a lane loads KB columns of each of 8 rows, and value j of
// those 8 rows is its fragment of column KB * (lane % 16) + j for
// v_mfma_f32_16x16x32_bf16; v's ranks are dealt to the lanes the same way.  No
// transposition goes through LDS.  The list is cut into parts where columns and
// adapters leave compute units idle; the wavefronts' sums are joined through
// LDS and the parts' go to slices for launch_finish, each in a fixed order; of one
// part the result is written at once.
//
// Measured, both matrices: 4096 rows of 4096 codes and 4096 values, rank 16, 16.4
// us (50 MB); 8192 rows of 4096 and 8192, four adapters of rank 64, 79 (168 MB of x;
// 58 with v in one part, whose registers allowed a lane twice the columns).
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWave = 64, kWaves = 8, kThreads = kWave * kWaves;
constexpr int kRows = 32;    // rows of the list of a step

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
// The 16-bit values j of two rows' words.
__device__ __forceinline__ uint32_t pair(uint32_t first, uint32_t second, int j) {
  return __builtin_amdgcn_perm(second, first, j % 2 ? 0x07060302u : 0x05040100u);
}

// Rows of the list that are in LDS at once: looked up in memory, each would
// wait for the loads of x that were sent before it.
constexpr int kListed = 8 * kWaves * kRows;

struct Lds {
  f32x4 part[kWaves][kWaves][kWave];   // of each wavefront, as many of its sums
  __attribute__((aligned(16))) int32_t list[kListed];
};

// KR ranks to a lane (16 KR of a workgroup), KB columns.
template <int KR, int KB, bool kCodes>
__device__ __forceinline__ void adapter_grad(const AdapterGrad& a, unsigned block, Lds& lds) {
  constexpr int kWords = kCodes ? KB / 4 : KB / 2;   // of a lane's columns in a row
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int l16 = lane % 16, h = lane / 16;
  const int cb = (int)(block % (unsigned)a.col_blocks);
  block /= (unsigned)a.col_blocks;
  const int rb = (int)(block % (unsigned)a.rank_blocks);
  block /= (unsigned)a.rank_blocks;
  const int slice = (int)(block % (unsigned)a.parts), id = (int)(block / (unsigned)a.parts);
  // Where columns end inside a lane's, it takes the last KB (its neighbour has
  // some of them too, with the same sums): no load needs a check.
  int64_t col = (int64_t)cb * 16 * KB + l16 * KB;
  const bool narrow = a.C < KB;
  if (!narrow) col = min(col, a.C - KB);
  const int rank = rb * 16 * KR + l16 * KR;
  // this part's rows of the adapter's list
  const int from = a.starts[id], to = a.starts[id + 1];
  const int per = (to - from + a.parts - 1) / a.parts;
  const int first = min(from + slice * per, to), last = min(first + per, to);

  f32x4 acc[KR][KB];
#pragma unroll
  for (int r = 0; r < KR; ++r)
#pragma unroll
    for (int j = 0; j < KB; ++j) acc[r][j] = f32x4{0, 0, 0, 0};

  struct Step {
    uint32_t x[8][kWords];
    uint32_t v[8][KR];
  };
  // The step at place p0 of the listed rows (the list goes on with its last row).
  auto load = [&](int p0, Step& s, auto whole) __attribute__((always_inline)) {
    int32_t rows[8];
    __builtin_memcpy(rows, __builtin_assume_aligned(lds.list + p0 + 8 * h, 16), 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t m = rows[i];
      if constexpr (kCodes) {
        __builtin_memcpy(s.x[i], __builtin_assume_aligned(static_cast<const int8_t*>(a.x) + m * a.C + col, KB), KB);
      } else {
        const uint16_t* row = static_cast<const uint16_t*>(a.x) + m * a.C;
        if constexpr (decltype(whole)::value) {
          __builtin_memcpy(s.x[i], row + col, 2 * KB);
        } else {
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const uint32_t lo = col + 2 * w < a.C ? row[col + 2 * w] : 0;
            const uint32_t hi = col + 2 * w + 1 < a.C ? row[col + 2 * w + 1] : 0;
            s.x[i][w] = lo | hi << 16;
          }
        }
      }
      __builtin_memcpy(s.v[i], __builtin_assume_aligned(a.v + m * a.ldt + min(rank, a.ldt - KR), KR == 3 ? 4 : 4 * KR), 4 * KR);
    }
    __builtin_amdgcn_sched_barrier(0);   // (moved loads would be waited for sooner)
  };
  auto multiply = [&](Step& s) __attribute__((always_inline)) {
    u32x4 fv[2][KR];   // both parts
#pragma unroll
    for (int r = 0; r < KR; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int half = 0; half < 2; ++half) fv[half][r][q] = pair(s.v[2 * q][r], s.v[2 * q + 1][r], half);
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      u32x4 fx;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (kCodes)
          fx[q] = pack2((float)(int8_t)(s.x[2 * q][j / 4] >> (8 * (j % 4))),
                        (float)(int8_t)(s.x[2 * q + 1][j / 4] >> (8 * (j % 4))));
        else fx[q] = pair(s.x[2 * q][j / 2], s.x[2 * q + 1][j / 2], j);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int r = 0; r < KR; ++r)
          acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fv[half][r]),
                                                              __builtin_bit_cast(bf16x8, fx), acc[r][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // This wavefront's steps of the n listed rows, the next step's loads on their
  // way (past the end the last step's again).  The rows that make no whole step
  // are one wavefront's.
  auto run = [&](int n) __attribute__((always_inline)) {
    const int whole = narrow ? 0 : n / kRows, count = (whole - wave + kWaves - 1) / kWaves;
    auto at = [&](int i) { return (wave + min(i, count - 1) * kWaves) * kRows; };
    if (count > 0) {
      Step even, odd;
      load(at(0), even, std::true_type{});
      int i = 0;
      for (; i + 2 <= count; i += 2) {
        load(at(i + 1), odd, std::true_type{});
        multiply(even);
        load(at(i + 2), even, std::true_type{});
        multiply(odd);
      }
      if (i < count) multiply(even);
    }
    for (int p = (whole + (wave - whole % kWaves + kWaves) % kWaves) * kRows; p < n; p += kWaves * kRows) {
      Step s;
      load(p, s, std::false_type{});
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = p + 8 * h + i < n;
#pragma unroll
        for (int w = 0; w < kWords; ++w) s.x[i][w] = in ? s.x[i][w] : 0;
#pragma unroll
        for (int w = 0; w < KR; ++w) s.v[i][w] = in ? s.v[i][w] : 0;
      }
      multiply(s);
    }
  };
  for (int base = first; base < last; base += kListed) {
    const int n = min(kListed, last - base);
    if (base > first) __syncthreads();
    for (int i = threadIdx.x; i < (n + kRows - 1) / kRows * kRows; i += kThreads) lds.list[i] = a.list[base + min(i, n - 1)];
    __syncthreads();
    run(n);
  }
  // The sums of the wavefronts that had rows, in order: eight at a time through
  // LDS, one to each wavefront to add up and store.  (The first wavefront alone:
  // 76 tokens, rank 40 20.3 us and not 12.6; 8192 tokens, rank 64 68 and not 58.)
  const int active = min(kWaves, (last - first + kRows - 1) / kRows);
  const int64_t matrix = (int64_t)a.R * a.C;
  float* const part = a.slices + ((int64_t)slice * a.count + id) * matrix;
#pragma unroll
  for (int c = 0; c < KR * KB; c += kWaves) {
    if (c > 0) __syncthreads();
    if (wave < active) {
#pragma unroll
      for (int k = 0; k < kWaves; ++k) lds.part[wave][k][lane] = acc[(c + k) / KB][(c + k) % KB];
    }
    __syncthreads();
    f32x4 sum = {0, 0, 0, 0};
    for (int w = 0; w < active; ++w) sum += lds.part[w][wave][lane];
    // lane: column col + j, ranks KR (4h + e) + r of the block's
    constexpr bool kOneRank = KB % kWaves == 0;   // of the eight sums
    const int r = kOneRank ? c / KB : (c + wave) / KB, j = kOneRank ? c % KB + wave : (c + wave) % KB;
    if (col + j >= a.C) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int rank = rb * 16 * KR + KR * (4 * h + e) + r;
      if (rank >= a.R) continue;
      const int64_t at = kCodes ? rank * a.C + col + j : (col + j) * a.R + rank;
      if (a.parts > 1) part[at] = sum[e];
      else a.out[id * matrix + at] = __builtin_bit_cast(uint16_t, (__bf16)sum[e]);
    }
  }
}

// The gradients of both matrices in one launch: b's workgroups, whose rows are
// longer, before a's.  (The grid's rows are for more workgroups than one dimension
// of it may have threads.)
template <int KR, int KA, int KB>
__global__ __launch_bounds__(kThreads) void adapter_grad_kernel(AdapterGrad ga, AdapterGrad gb, unsigned blocks_b,
                                                                unsigned blocks) {
  __shared__ Lds lds;
  const unsigned block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block < blocks_b) adapter_grad<KR, KB, false>(gb, block, lds);
  else if (block < blocks) adapter_grad<KR, KA, true>(ga, block - blocks_b, lds);
}

// Ranks of a lane, and columns: as many sums as registers allow.  Us of both
// gradients without the input's, by ranks and columns (codes, values) of a lane:
// 4096 rows of 4096 and 4096, rank 32: 2 16 8 46.4, 2 8 8 44.6, 3 8 8 46.8, 4 4 4 42.9;
// 217 of 2048: 22.0, 21.8, 22.2, 19.8; rank 40, 2048 of 4096: 62, 58.3, 55.1, 56.8; 64
// of 2592 and 2776: 34.6, 32.8, 27.0, 29.4; rank 48, 4096 of 2048 and 5136: 72, 67, 61,
// 62; rank 64, 8192 of 4096 and 8192: 146, 142, 161, 142; 2048 of 4096: 44.4, 42.5,
// 46.1, 43.3; 300 of 1024: 27.5, 26.4, 27.4, 25.8; rank 128, 1024 of 4096: 45, 40.8,
// 44.5, 40.4.
int ranks_of(int R) { return R <= 16 ? 1 : R > 32 && R <= 48 ? 3 : 4; }
int columns_of(int R, bool codes) { return ranks_of(R) == 4 ? 4 : ranks_of(R) == 1 && codes ? 16 : 8; }

int64_t col_blocks_of(int64_t C, int R, bool codes) { return (C + 16 * columns_of(R, codes) - 1) / (16 * columns_of(R, codes)); }
int64_t rank_blocks_of(int R) { return (R + 16 * ranks_of(R) - 1) / (16 * ranks_of(R)); }

// Parts of the lists: about one workgroup per compute unit for both gradients
// (b's has twice the bytes), each wavefront a step or more.
int parts_of(int64_t M, int64_t C, int R, int count, bool codes) {
  const int64_t blocks = col_blocks_of(C, R, codes) * rank_blocks_of(R) * count, want = codes ? 96 : 160;
  return (int)std::max<int64_t>(1, std::min(want / blocks, (M + kWaves * kRows - 1) / (kWaves * kRows)));
}

// A row of the grid, and all of it.
constexpr int64_t kGridRow = int64_t(1) << 20, kMaxBlocks = int64_t(1) << 31;

// Workgroups of one of the gradients (none: 0).
int64_t set_blocks(AdapterGrad& g, bool codes) {
  if (g.out == nullptr) return 0;
  g.col_blocks = (int)col_blocks_of(g.C, g.R, codes);
  g.rank_blocks = (int)rank_blocks_of(g.R);
  return (int64_t)g.col_blocks * g.rank_blocks * g.parts * g.count;
}

// ---- the adapters' share of few rows' input gradient ----

// out fp32 [M, C] = sum_r u[m, r] p[id][r, c]: a thread for 8 columns of a row.
constexpr int kUpThreads = 256;
__global__ __launch_bounds__(kUpThreads) void adapter_up_kernel(const uint16_t* __restrict__ u, int ldt,
                                                                const uint16_t* __restrict__ p,
                                                                const int32_t* __restrict__ ids, int count, int R,
                                                                int64_t C, float* __restrict__ out) {
  const int64_t m = blockIdx.y, c = ((int64_t)blockIdx.x * kUpThreads + threadIdx.x) * 8;
  if (c >= C) return;
  const int id = ids[m];
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  if (id >= 0 && id < count) {
    const uint16_t* row = p + (int64_t)id * R * C + c;
#pragma unroll 8
    for (int r = 0; r < R; ++r) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(row + r * C);
      const float f = __uint_as_float((uint32_t)u[m * ldt + r] << 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[2 * e] = fmaf(f, __uint_as_float(w[e] << 16), s[2 * e]);
        s[2 * e + 1] = fmaf(f, __uint_as_float(w[e] & 0xffff0000u), s[2 * e + 1]);
      }
    }
  }
  f32x4* o = reinterpret_cast<f32x4*>(out + m * C + c);
  o[0] = f32x4{s[0], s[1], s[2], s[3]};
  o[1] = f32x4{s[4], s[5], s[6], s[7]};
}

}  // namespace

int adapter_grad_parts(int64_t M, int64_t C, int64_t R, int64_t count, bool codes) {
  return parts_of(M, C, (int)R, (int)count, codes);
}

bool adapter_grads_fit(int64_t M, int64_t N, int64_t K, int64_t R, int64_t count) {
  int64_t blocks = 0;
  for (const bool codes : {true, false}) {
    const int64_t C = codes ? K : N;
    blocks += col_blocks_of(C, (int)R, codes) * rank_blocks_of((int)R) * count * parts_of(M, C, (int)R, (int)count, codes);
  }
  return blocks <= kMaxBlocks;
}

hipError_t launch_adapter_grads(AdapterGrad ga, AdapterGrad gb, hipStream_t s) {
  const int64_t na = set_blocks(ga, true), nb = set_blocks(gb, false);
  if (na + nb == 0) return hipSuccess;
  if (na + nb > kMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid((unsigned)std::min(na + nb, kGridRow), (unsigned)((na + nb + kGridRow - 1) / kGridRow)), block(kThreads);
  const unsigned first = (unsigned)nb, all = (unsigned)(na + nb);
  switch (ranks_of(na ? ga.R : gb.R)) {
    case 1: hipLaunchKernelGGL((adapter_grad_kernel<1, 16, 8>), grid, block, 0, s, ga, gb, first, all); break;
    case 3: hipLaunchKernelGGL((adapter_grad_kernel<3, 8, 8>), grid, block, 0, s, ga, gb, first, all); break;
    default: hipLaunchKernelGGL((adapter_grad_kernel<4, 4, 4>), grid, block, 0, s, ga, gb, first, all); break;
  }
  return hipGetLastError();
}

hipError_t launch_adapter_up(const uint16_t* u, int64_t ldt, const uint16_t* p, const int32_t* ids, int64_t count,
                             int64_t R, int64_t M, int64_t C, float* out, hipStream_t s) {
  const dim3 grid((unsigned)((C / 8 + kUpThreads - 1) / kUpThreads), (unsigned)M);
  hipLaunchKernelGGL(adapter_up_kernel, grid, dim3(kUpThreads), 0, s, u, (int)ldt, p, ids, (int)count, (int)R, C, out);
  return hipGetLastError();
}

}  // namespace w8a8
