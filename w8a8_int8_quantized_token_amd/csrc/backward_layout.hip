// Operand layout of the backward products, and the joins after them.  The
// product kernel wants both operands contiguous along the summed index, but
// the input's gradient sums over output channels (rows of the weight) and the
// weight's gradient over tokens (rows of the activations).  Before the
// products, one launch of up to six jobs (`prepare`):
//   turn_codes:  int8 [R,C] (times scale[r]) -> bf16 [C, ld], zeros past
//     column R; or, `paired`, the R = 2N rows of a stacked [gate; up] weight
//     with 16 gate columns, the 16 up columns of the same channels, and so on
//     (the order of the gated gradient's columns; zeros for channels past N);
//   turn_values: bf16 [R,C] -> bf16 [C, ld] (zeros past column R), and the
//     fp32 sums of each column over blocks of rows;
//   pad_rows:    bf16 [R,C] -> bf16 [R, ld], zeros past column C;
//   turn_each:   as turn_values without sums, for several matrices;
//   lists:       the rows of each id, in order (low-rank adapters);
// after them one launch of up to three (`finish`):
//   join_slices: the fp32 slices of a product split along its sum -> bf16;
//   sum_rows:    fp32 [P,C] -> bf16 [C], summed over P in a fixed order.
// Codes are small integers and exact in bf16; with a scale each value
// q * scale is rounded to bf16 once.  The scale belongs to the summed index, so
// one of a product's operands has to take it, and bf16 MFMAs take no more bits: a
// second, lower part of that operand would double the product.  The rounding
// is one of half a step (2^-8) per term, of either sign; a gradient's rms error is
// 2.3e-3 of its own, of which its rounding to bf16 alone is 1.7e-3.
//
// Bound by memory (R*C*(1+2) and R*C*(2+2) bytes) where they are large, and by
// their launch where they are small, which is why they share one: a gradient
// of a 300 x 600 linear has five of them at 4 us each.
#include "kernels.h"

#include <algorithm>

namespace w8a8 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t __attribute__((may_alias)) word;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kT = 64;          // tile edge
constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / kThreads - 1;   // a launch has under 2^32 threads

union Lds {
  struct { uint32_t tile[64][33]; float scale[64]; } codes;
  struct { uint16_t tile[kT][kT + 2]; float part[kThreads / 8][kT]; } values;
};

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

// 64 rows by 128 columns (C % 16 == 0, ld % 8 == 0).  A thread turns 8 rows of
// 4 columns, read as 8 words (LDS rows of 33 words: the 64 lanes' words lie in
// 64 banks) and written as four 16-byte pieces of 128-byte runs.  4096 x 4096:
// 10.6 us, 4.7 TB/s.
constexpr int kCodeRows = 64, kCodeCols = 128;
template <bool kPaired>
__device__ void turn_codes(const LayoutJob& j, int64_t block, Lds& lds) {
  const int tid = threadIdx.x;
  const int64_t nx = (j.C + kCodeCols - 1) / kCodeCols;
  const int64_t c0 = block % nx * kCodeCols, r0 = block / nx * kCodeRows;
  const int8_t* q = static_cast<const int8_t*>(j.in);
  const int r = tid / 8, c = (tid % 8) * 16;
  u32x4 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t from = source_row(r0 + i * 32 + r, j.R, kPaired);
    v[i] = from >= 0 && c0 + c < j.C ? *reinterpret_cast<const u32x4*>(q + from * j.C + c0 + c) : u32x4{0, 0, 0, 0};
  }
  if (j.scale != nullptr && tid < kCodeRows) {
    const int64_t at = source_row(r0 + tid, j.R, kPaired);
    lds.codes.scale[tid] = at >= 0 ? j.scale[at] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) lds.codes.tile[i * 32 + r][c / 4 + e] = v[i][e];
  __syncthreads();
  const int tr = (tid % 8) * 8, tc = tid / 8;   // this thread's rows and word column when writing
  if (c0 + tc * 4 < j.C && r0 + tr < j.ld) {
    uint32_t w[8];
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = lds.codes.tile[tr + k][tc];
      s[k] = j.scale != nullptr ? lds.codes.scale[tr + k] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack2((float)(int8_t)(w[2 * e] >> (8 * i)) * s[2 * e],
                     (float)(int8_t)(w[2 * e + 1] >> (8 * i)) * s[2 * e + 1]);
      *reinterpret_cast<u32x4*>(j.out + (c0 + tc * 4 + i) * j.ld + r0 + tr) = o;
    }
  }
}

// 64 columns, `span` rows (a multiple of 64).  out may be null (sums only),
// sums may be null.
__device__ void turn_values(const LayoutJob& j, int64_t block, Lds& lds) {
  const int tid = threadIdx.x;
  const int64_t nx = (j.C + kT - 1) / kT, by = block / nx;
  const int64_t c0 = block % nx * kT;
  const uint16_t* x = static_cast<const uint16_t*>(j.in);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  const int64_t first = by * j.span, last = first + j.span < j.ld ? first + j.span : j.ld;
  for (int64_t r0 = first; r0 < last; r0 += kT) {
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int r = it * 32 + tid / 8, c = (tid % 8) * 8;
      u32x4 v = u32x4{0, 0, 0, 0};
      if (r0 + r < j.R) v = load8(x + (r0 + r) * j.C, c0 + c, j.C);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[2 * e] += bf(v[e] & 0xffffu);
        acc[2 * e + 1] += bf(v[e] >> 16);
        *reinterpret_cast<word*>(&lds.values.tile[r][c + 2 * e]) = v[e];
      }
    }
    __syncthreads();
    if (j.out != nullptr) {
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const int id = it * kThreads + tid, c = id / 8, r = (id % 8) * 8;
        if (c0 + c < j.C && r0 + r < j.ld) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = (uint32_t)lds.values.tile[r + 2 * e][c] | (uint32_t)lds.values.tile[r + 2 * e + 1][c] << 16;
          *reinterpret_cast<u32x4*>(j.out + (c0 + c) * j.ld + r0 + r) = w;
        }
      }
    }
    __syncthreads();
  }
  if (j.sums != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) lds.values.part[tid / 8][(tid % 8) * 8 + e] = acc[e];
    __syncthreads();
    if (tid < kT && c0 + tid < j.C) {
      float s = 0.0f;
      for (int g = 0; g < kThreads / 8; ++g) s += lds.values.part[g][tid];
      j.sums[by * j.C + c0 + tid] = s;
    }
  }
}

// Eight values per thread, kPadBlock of them per workgroup.
constexpr int64_t kPadBlock = 4 * kThreads;
__device__ void pad_rows(const LayoutJob& j, int64_t block) {
  const uint16_t* x = static_cast<const uint16_t*>(j.in);
  const int64_t per_row = j.ld / 8, n = j.R * per_row;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = block * kPadBlock + k * kThreads + threadIdx.x;
    if (i < n) {
      const int64_t r = i / per_row, c = (i - r * per_row) * 8;
      *reinterpret_cast<u32x4*>(j.out + r * j.ld + c) = load8(x + r * j.C, c, j.C);
    }
  }
}

// A workgroup for an id: where its list starts (the rows with smaller ids), then
// its rows in order, each wavefront a quarter of them.  Two passes over the
// ids with sixteen loads in flight (one wavefront with four: 25 us for 4096 ids,
// the longest part of the launch).
__device__ void make_lists(const LayoutJob& j, int64_t block, Lds& lds) {
  constexpr int kLoads = 16, kWaves = kThreads / 64;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int id = (int)block, count = (int)j.C, M = (int)j.R;
  const int32_t* ids = static_cast<const int32_t*>(j.in);
  const int per = (M + kWaves * 64 - 1) / (kWaves * 64) * 64;   // rows of a wavefront
  const int first = wave * per, last = min(first + per, M);
  auto load = [&](int m0, int (&v)[kLoads]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int m = m0 + i * 64 + lane;
      v[i] = m < last ? ids[m] : -1;
    }
  };
  int before = 0, own = 0;
  for (int m0 = first; m0 < last; m0 += 64 * kLoads) {
    int v[kLoads];
    load(m0, v);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      before += __popcll(__builtin_amdgcn_ballot_w64(v[i] >= 0 && v[i] < id));
      own += __popcll(__builtin_amdgcn_ballot_w64(v[i] == id));
    }
  }
  int (*const counts)[2] = reinterpret_cast<int (*)[2]>(&lds);
  if (lane == 0) counts[wave][0] = before, counts[wave][1] = own;
  __syncthreads();
  int start = 0, at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    start += counts[w][0];
    if (w < wave) at += counts[w][1];
    all += counts[w][1];
  }
  if (threadIdx.x == 0) {
    j.starts[id] = start;
    if (id == count - 1) j.starts[count] = start + all;
  }
  at += start;
  if (own == 0) return;
  for (int m0 = first; m0 < last; m0 += 64 * kLoads) {
    int v[kLoads];
    load(m0, v);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint64_t hits = __builtin_amdgcn_ballot_w64(v[i] == id);
      if (v[i] == id) j.list[at + __popcll(hits & ((uint64_t(1) << lane) - 1))] = m0 + i * 64 + lane;
      at += __popcll(hits);
    }
  }
}

// One of `batch` matrices, each as turn_values without sums.
__device__ void turn_each(const LayoutJob& j, int64_t block, Lds& lds) {
  const int64_t per = (j.C + kT - 1) / kT * ((j.ld + j.span - 1) / j.span), k = block / per;
  LayoutJob one = j;
  one.in = static_cast<const uint16_t*>(j.in) + k * j.R * j.C;
  one.out = j.out + k * j.C * j.ld;
  one.sums = nullptr;
  turn_values(one, block - k * per, lds);
}

struct Prepare {
  LayoutJob job[kMaxJobs];
  int64_t end[kMaxJobs];   // workgroups up to and with each job
};
__global__ __launch_bounds__(kThreads) void prepare_kernel(Prepare p) {
  __shared__ __attribute__((aligned(16))) Lds lds;
  int64_t block = blockIdx.x;
  int k = 0;
  while (block >= p.end[k]) ++k;
  if (k > 0) block -= p.end[k - 1];
  const LayoutJob& j = p.job[k];
  switch (j.kind) {
    case LayoutJob::kTurnCodes: turn_codes<false>(j, block, lds); break;
    case LayoutJob::kTurnPaired: turn_codes<true>(j, block, lds); break;
    case LayoutJob::kTurnValues: turn_values(j, block, lds); break;
    case LayoutJob::kTurnEach: turn_each(j, block, lds); break;
    case LayoutJob::kLists: make_lists(j, block, lds); break;
    default: pad_rows(j, block); break;
  }
}

// Eight outputs per thread and step (n % 8 == 0).  Up to eight slices' loads are
// in flight: with one at a time the join of few outputs takes a memory latency
// for each of its slices (46 of 1 x 512 values: 15 us).  Only slices that are
// there are read (two of 4096 x 2048 values: 17 us, and 36 when eight are always
// read).
template <int kSlices>
__device__ __forceinline__ void add_slices(const f32x4* p, int64_t stride, f32x4& lo, f32x4& hi) {
  f32x4 v[kSlices][2];
#pragma unroll
  for (int i = 0; i < kSlices; ++i) {
    v[i][0] = __builtin_nontemporal_load(p + i * stride);
    v[i][1] = __builtin_nontemporal_load(p + i * stride + 1);
  }
#pragma unroll
  for (int i = 0; i < kSlices; ++i) lo += v[i][0], hi += v[i][1];
}
__device__ void join_slices(const JoinJob& j, int64_t block) {
  const int64_t groups = j.n / 8, stride = j.n / 4;
  const f32x4* part = reinterpret_cast<const f32x4*>(j.part);
  for (int64_t g = block * kThreads + threadIdx.x; g < groups; g += j.blocks * kThreads) {
    f32x4 lo = f32x4{0, 0, 0, 0}, hi = lo;
    const f32x4* p = part + g * 2;
    int64_t left = j.P;
    for (; left >= 8; left -= 8, p += 8 * stride) add_slices<8>(p, stride, lo, hi);
    if (left & 4) add_slices<4>(p, stride, lo, hi), p += 4 * stride;
    if (left & 2) add_slices<2>(p, stride, lo, hi), p += 2 * stride;
    if (left & 1) add_slices<1>(p, stride, lo, hi);
    *reinterpret_cast<u32x4*>(j.out + g * 8) = u32x4{pack2(lo[0], lo[1]), pack2(lo[2], lo[3]), pack2(hi[0], hi[1]), pack2(hi[2], hi[3])};
  }
}

// 32 columns per workgroup, 8 groups of rows with eight loads in flight each.
__device__ void sum_rows(const JoinJob& j, int64_t block, float (*lds)[33]) {
  constexpr int kGroups = kThreads / 32;
  const int g = threadIdx.x / 32, l = threadIdx.x % 32;
  const int64_t c = block * 32 + l;
  float s = 0.0f;
  if (c < j.n)
    for (int64_t p = g; p < j.P; p += 8 * kGroups) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p + i * kGroups < j.P ? j.part[(p + i * kGroups) * j.n + c] : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  lds[g][l] = s;
  __syncthreads();
  if (g == 0 && c < j.n) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t += lds[i][l];
    j.out[c] = __builtin_bit_cast(uint16_t, (__bf16)t);
  }
}

struct Finish {
  JoinJob job[kMaxJobs];
  int64_t end[kMaxJobs];
};
__global__ __launch_bounds__(kThreads) void finish_kernel(Finish p) {
  __shared__ float lds[kThreads / 32][33];
  int64_t block = blockIdx.x;
  int k = 0;
  while (block >= p.end[k]) ++k;
  if (k > 0) block -= p.end[k - 1];
  if (p.job[k].slices) join_slices(p.job[k], block);
  else sum_rows(p.job[k], block, lds);
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

// Rows of one workgroup's sums: as many as leave at least about 8 workgroups
// per compute unit, 64 to 1024.
int64_t transpose_sum_span(int64_t R, int64_t C) {
  const int64_t tiles = (C + kT - 1) / kT;
  int64_t span = 64;
  while (span < 1024 && tiles * ((R + 2 * span - 1) / (2 * span)) >= 2048) span *= 2;
  return span;
}

namespace {
// Workgroups of a job.
int64_t blocks_of(const LayoutJob& j) {
  const auto tiles = [](int64_t v, int64_t t) { return (v + t - 1) / t; };
  return j.kind == LayoutJob::kPadRows      ? tiles(j.R * (j.ld / 8), kPadBlock)
         : j.kind == LayoutJob::kTurnValues ? tiles(j.C, kT) * tiles(j.R, j.span)
         : j.kind == LayoutJob::kTurnEach   ? tiles(j.C, kT) * tiles(j.ld, j.span) * j.batch
         : j.kind == LayoutJob::kLists      ? j.C
                                            : tiles(j.C, kCodeCols) * tiles(j.ld, kCodeRows);
}
}  // namespace

bool prepare_fits(const LayoutJob* jobs, int n) {
  int64_t blocks = 0;
  for (int k = 0; k < n; ++k) blocks += blocks_of(jobs[k]);
  return blocks <= kMaxBlocks;
}

hipError_t launch_prepare(const LayoutJob* jobs, int n, hipStream_t stream) {
  if (!prepare_fits(jobs, n)) return hipErrorInvalidValue;
  Prepare p;
  int64_t end = 0;
  for (int k = 0; k < kMaxJobs; ++k) {
    if (k < n) end += blocks_of(p.job[k] = jobs[k]);
    p.end[k] = end;
  }
  hipLaunchKernelGGL(prepare_kernel, dim3((unsigned)end), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_finish(const JoinJob* jobs, int n, hipStream_t stream) {
  Finish p;
  int64_t end = 0;
  for (int k = 0; k < kMaxJobs; ++k) {
    if (k < n) {
      JoinJob& j = p.job[k] = jobs[k];
      j.blocks = j.slices ? std::min<int64_t>((j.n / 8 + kThreads - 1) / kThreads, 256 * 16) : (j.n + 31) / 32;
      end += j.blocks;
    }
    p.end[k] = end;
  }
  if (end > kMaxBlocks) return hipErrorInvalidValue;
  hipLaunchKernelGGL(finish_kernel, dim3((unsigned)end), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace w8a8
