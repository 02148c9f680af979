// C ABI of the operators around the linear (few-token forms, gated product,
// backward passes, norm and rotation of queries and keys): argument checks,
// workspace layout and launches.  Semantics are documented in include/w8a8.h;
// checks always complete before anything is launched.
#include "../../include/w8a8.h"
#include "kernels.h"

#include <algorithm>

namespace {

using w8a8::GateAct;

constexpr int64_t kMaxRows = int64_t(1) << 26;
// Longest summed index of a backward product: a tile's 256 rows of bf16 stay
// within the 31-bit offsets of its buffer ranges.
constexpr int64_t kMaxSummed = int64_t(1) << 21;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
w8a8_status launched(hipError_t e) { return e == hipSuccess ? W8A8_OK : W8A8_ERR_LAUNCH; }

// N output channels from `per` weight rows each.
bool shape_ok(int64_t M, int64_t N, int64_t K, int per) {
  return M >= 0 && M <= kMaxRows && N >= 1 && N <= kMaxRows / per && K >= 16 && K % 16 == 0 && K <= W8A8_MAX_K;
}

// Consecutive 256-byte aligned pieces of a workspace.
struct Pieces {
  int64_t bytes = 0;
  int64_t add(int64_t n) {
    const int64_t at = bytes;
    bytes += (n + 255) / 256 * 256;
    return at;
  }
};
template <class T>
T* at(void* ws, int64_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

// ---- few tokens / quantize on the way ----

struct DynamicPlan {
  bool few, codes;     // one of the few-token launches; codes made beforehand
  int splits, tile;    // otherwise the linear's plan (gated: tile -1, no split)
  int64_t xq, xs, slices;
  int64_t bytes;
};
// Where the few-token kernel is the faster one.  It walks 16 channels at a time,
// one group to a compute unit up to 4096 channels, and a group takes 0.8 us (1.2
// beyond 16 tokens) however short K is, so many channels of a short K go to the
// tiled kernel; beyond 16 tokens short rows do too, as the codes are a launch of
// their own there.  Cold weights, us (quantize + tiled / few tokens):
//   1 and 16 tokens, K = 64: 8192 channels 5.8 / 5.7 and 6.4 / 6.3, 12288 6.0 / 6.3
//   and 6.5 / 7.1, 65536 11.7 / 16.4 and 12.2 / 17.4; K = 256: 12288 6.7 / 6.5 and
//   7.0 / 7.2, 16384 6.7 / 7.2 and 7.1 / 8.0; K = 512: 16384 8.2 / 8.2 and 8.7 / 9.0,
//   32768 10.4 / 11.5 and 10.8 / 12.4; K = 768: 32768 11.9 / 11.8 and 12.4 / 13.1,
//   65536 18.7 / 18.8 and 19.4 / 20.5;
//   12 and 16 tokens whose codes come from memory, K = 4096: 32768 37 / 31 and 37 /
//   32, 40960 73 / 36 and 73 / 37, 65536 57 / 53 and 57 / 56; K = 5120: 50000 52 / 53
//   and 52 / 57, 65536 62 / 64 and 62 / 70; K = 8192: 65536 114 / 92 and 115 / 98
//   (8 tokens, K = 5120: 65536 61 / 61);
//   17 and 32 tokens, K = 64: 512 channels 5.8 / 6.2 and 5.6 / 6.2; K = 256: 2048
//   6.8 / 6.7 and 6.9 / 6.8, 6144 6.9 / 8.0 and 7.0 / 7.9; K = 1024: 8192 11.3 / 9.4
//   and 11.5 / 9.6, 16384 11.8 / 11.9 and 12.0 / 12.4 (warm 9.3 / 10.9 and 9.5 / 11.3);
//   K = 2048: 16384 17.9 / 15.7 and 18.0 / 16.6, 32768 22.3 / 23.8 and 22.9 / 26.1; K =
//   8192: 16384 54 / 34 and 54 / 38, 32768 59 / 59 and 61 / 67;
//   gated, where long rows go on paying: 12 and 16 tokens, K = 2048: 65536 channels
//   54 / 47 and 54 / 49, K = 4096: 65536 119 / 95 and 118 / 97; 17 and 32 tokens, K =
//   2048: 16384 22.1 / 21.7 and 22.8 / 22.7, 65536 55 / 59 and 55 / 62, K = 4096: 24576
//   47 / 41 and 50 / 44, 65536 118 / 104 and 120 / 112, K = 8192: 32768 111 / 94 and 112 /
//   105.
bool few_tokens_pay(int64_t M, int64_t N, int64_t K, bool gated, bool in_lds) {
  if (M > 16) return K >= 256 && (N <= 8 * std::min<int64_t>(K, 2048) || (gated && K >= 4096));
  if (!gated && M > 8 && !in_lds && N > 40960 && K < 8192) return false;
  return K >= 768 || N <= 8192 + 16 * K;
}

// More tokens: K ranges where the linear is hardly ever faster whole, be the weight
// cold or warm (us whole / in ranges, cold; warm): 256 x 2048 x 6144 38.9 / 28.5; 27.9 /
// 27.7, 64 x 2048 x 4096 27.8 / 20.6; 19.1 / 18.9, but 512 x 2048 x 4096 27.8 / 29.3;
// 21.6 / 27.9, 256 x 512 x 4096 20.7 / 23.7; 20.1 / 22.1, 192 x 2048 x 5120 33.6 /
// 28.8; 23.8 / 27.6.  (At the worst of it, 1024 x 1024 x 6144, 40.3 / 35.5; 30.9 / 35.7.)
bool ranges_pay(int64_t M, int64_t K) { return K >= 6144 || M <= 64; }

// `room`: there is a workspace; without one the few-token kernel takes what
// needs none.
DynamicPlan dynamic_plan(int64_t M, int64_t N, int64_t K, bool gated, bool room) {
  DynamicPlan p{};
  const bool in_lds = w8a8::few_tokens_in_lds(M, K);
  p.few = M <= w8a8::kFewTokens && (few_tokens_pay(M, N, K, gated, in_lds) || (in_lds && !room));
  p.codes = !p.few || !in_lds;
  p.splits = 1;
  p.tile = -1;
  Pieces w;
  if (p.codes) {
    p.xq = w.add(M * K);
    p.xs = w.add(4 * M);
  }
  if (!p.few && !gated && ranges_pay(M, K)) {
    p.splits = w8a8::select_splitk(M, N, K, &p.tile);
    if (p.splits > 1) p.slices = w.add((int64_t)w8a8_linear_splitk_workspace(M, N, p.splits));
  }
  p.bytes = w.bytes;
  return p;
}

w8a8_status dynamic(const uint16_t* x, const int8_t* wq, const float* w_scale, const uint16_t* bias, uint16_t* y,
                    int64_t M, int64_t N, int64_t K, int act, bool gated, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  if (!shape_ok(M, N, K, gated ? 2 : 1)) return W8A8_ERR_SHAPE;
  if (act < 0 || act > 1) return W8A8_ERR_ARG;
  if (M == 0) return W8A8_OK;
  DynamicPlan p = dynamic_plan(M, N, K, gated, true);
  if (!ws || !aligned(ws, 16) || ws_bytes < (size_t)p.bytes) p = dynamic_plan(M, N, K, gated, false);
  if (!x || !wq || !w_scale || !y || (p.bytes && !ws)) return W8A8_ERR_NULL;
  if (!aligned(x, 16) || !aligned(wq, 16) || !aligned(w_scale, 4) || !aligned(y, 2) || (bias && !aligned(bias, 2)) ||
      (p.bytes && !aligned(ws, 16)))
    return W8A8_ERR_ALIGN;
  if (ws_bytes < (size_t)p.bytes) return W8A8_ERR_ARG;
  int8_t* xq = nullptr;
  float* xs = nullptr;
  if (p.codes) {
    xq = at<int8_t>(ws, p.xq);
    xs = at<float>(ws, p.xs);
    if (w8a8::launch_quantize_rows(x, xq, xs, M, K, stream) != hipSuccess) return W8A8_ERR_LAUNCH;
  }
  if (p.few)
    return launched(w8a8::launch_few_tokens(x, xq, xs, wq, w_scale, bias, y, M, N, K, act, gated, stream));
  if (gated)
    return launched(w8a8::launch_gated(-1, static_cast<GateAct>(act), xq, xs, wq, w_scale, bias, y, M, N, K, stream));
  if (p.splits > 1 && aligned(y, 16))   // its second pass writes 16 bytes at a time
    return w8a8_linear_splitk(xq, xs, wq, w_scale, bias, y, M, N, K, p.splits, p.tile, act, at<void>(ws, p.slices),
                              (size_t)(p.bytes - p.slices), stream);
  return act ? w8a8_linear_gelu(xq, xs, wq, w_scale, bias, y, M, N, K, stream)
             : w8a8_linear(xq, xs, wq, w_scale, bias, y, M, N, K, stream);
}

// ---- backward products ----

// Workspace of a backward pass: the padded copy of dy where it is needed, the
// sums for the bias, and for the input's and the weight's gradient their first
// operands (where not dy itself), their second ones, and the slices of a
// product that is split along its sum.
struct BackPlan {
  int64_t ldy;                // row length of the copy of dy
  int64_t ld, mp;             // summed lengths of the two products, padded
  int64_t copy, sums, sum_rows;
  int64_t first, wt, slices_x;
  int64_t second, xt, slices_w;
  int ranges_x, ranges_w;
  bool few;                   // dx straight from the codes (few_grad.hip): no wt
  int64_t bytes;
};
// Rows of an operand laid out here are whole 128-byte lines, zeros past their
// end: rows that start inside a line cost the product a quarter of its time
// (2000 x 2000 x 5000: 53 us with rows of 5000 values, 41 with 5056; 333 x
// 2064 x 3000: 18.1 and 13.6).
constexpr int64_t kLine = 64;
// Few tokens' dx comes from the codes as they are (its join writes 16 bytes at
// a time) where turning them costs more than its slices do: from 6 million
// codes on (us turned and as they are: 29 tokens, 2776 x 2592 20.2 and 15.9,
// 12000 x 5408 75 and 30; gated, 26 tokens, 2 x 2749 x 1872 32.1 and 31.4; but
// 600 x 5440 11.9 and 13.4, gated 2 x 722 x 2176 22.8 and 26.7).
bool few_rows(int64_t M, int64_t rows, int64_t K) { return M <= w8a8::kFewGradTokens && rows * K >= 6000000; }
// Rows of dy that start inside a line are copied too where the product is long
// enough (dx alone, us without and with the copy; M x N x K): 4096 x 5000 x 512
// 45 and 42, 777 x 5000 x 2048 51 and 37; but 4096 x 5000 x 256 31 and 37, 4096
// x 1000 x 1024 20 and 22, 100 x 5000 x 1024 16 and 22.
bool copy_lines(int64_t M, int64_t N, int64_t K) {
  return N % kLine != 0 && M >= 256 && N >= 2048 && K >= 512;
}

BackPlan back_plan(int64_t M, int64_t N, int64_t K, bool gated, bool dx, bool dw, bool db, bool copy_dy, bool few) {
  BackPlan p{};
  p.few = dx && few;
  const int64_t cols = (gated ? 2 : 1) * N;
  p.ldy = gated ? up(N, 8) : copy_dy ? up(N, kLine) : N;
  p.ld = gated ? up(2 * N, kLine) : p.ldy;
  p.mp = up(M, kLine);
  Pieces w;
  if (db) {
    p.sum_rows = gated ? w8a8::gated_grad_sum_rows(M, N, K)
                       : (M + w8a8::transpose_sum_span(M, N) - 1) / w8a8::transpose_sum_span(M, N);
    p.sums = w.add(4 * p.sum_rows * cols);
  }
  if (copy_dy && (gated || (dx && !few))) p.copy = w.add(2 * M * p.ldy);
  if (dx) {
    if (gated) p.first = w.add(2 * M * p.ld);
    if (!few) p.wt = w.add(2 * K * p.ld);
    p.ranges_x = few ? w8a8::few_grad_slices(M, N, K, gated) : w8a8::gemm_bf16_slices(M, K, p.ld);
    if (few || p.ranges_x > 1) p.slices_x = w.add(4 * M * K * p.ranges_x);
  }
  if (dw) {
    p.second = w.add(2 * cols * p.mp);
    p.xt = w.add(2 * K * p.mp);
    p.ranges_w = w8a8::gemm_bf16_slices(cols, K, p.mp);
    if (p.ranges_w > 1) p.slices_w = w.add(4 * cols * K * p.ranges_w);
  }
  p.bytes = w.bytes;
  return p;
}

// The largest of the plans that calls of these sizes may take, as their
// addresses are (without the copy of dy a plan is smaller unless its rows, and
// with them its ranges, are others).
size_t back_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool dx, bool dw, bool db) {
  int64_t most = 0;
  for (const bool copy : {true, false})
    for (const bool few : {false, true})
      if ((copy || (!gated && N % 8 == 0 && N % kLine != 0)) && (!few || few_rows(M, gated ? 2 * N : N, K)))
        most = std::max(most, back_plan(M, N, K, gated, dx, dw, db, copy, few).bytes);
  return (size_t)most;
}

// The products of a backward pass and what comes after them: dx [M,K] from
// first [M,ld] and wt [K,ld] (few tokens: the codes and scales), dw [cols,K] from second [cols,mp] and xt [K,mp],
// dbias [cols] from the sums.
hipError_t products(const BackPlan& p, void* ws, const uint16_t* first, const int8_t* wq, const float* w_scale,
                    bool gated, uint16_t* dx, uint16_t* dw, uint16_t* dbias, int64_t M, int64_t cols, int64_t K,
                    hipStream_t stream) {
  w8a8::JoinJob jobs[w8a8::kMaxJobs];
  int n = 0;
  hipError_t e = hipSuccess;
  if (dx) {
    // the join writes 16 bytes at a time
    float* slices = p.few || (p.ranges_x > 1 && aligned(dx, 16)) ? at<float>(ws, p.slices_x) : nullptr;
    if (p.few)
      e = gated ? w8a8::launch_few_grad(first, p.ld, wq, nullptr, slices, M, cols / 2, K, true, stream)
                : w8a8::launch_few_grad(first, cols, wq, w_scale, slices, M, cols, K, false, stream);
    else e = w8a8::launch_gemm_bf16(first, at<uint16_t>(ws, p.wt), dx, slices, M, K, p.ld, stream);
    if (slices) jobs[n++] = {slices, dx, p.ranges_x, M * K, true, 0};
  }
  if (dw && e == hipSuccess) {
    float* slices = p.ranges_w > 1 && aligned(dw, 16) ? at<float>(ws, p.slices_w) : nullptr;
    e = w8a8::launch_gemm_bf16(at<uint16_t>(ws, p.second), at<uint16_t>(ws, p.xt), dw, slices, cols, K, p.mp, stream);
    if (slices) jobs[n++] = {slices, dw, p.ranges_w, cols * K, true, 0};
  }
  if (dbias) jobs[n++] = {at<float>(ws, p.sums), dbias, p.sum_rows, cols, false, 0};
  return e == hipSuccess && n > 0 ? w8a8::launch_finish(jobs, n, stream) : e;
}

// dw and dbias of no tokens are zeros.
w8a8_status no_tokens(uint16_t* dw, uint16_t* dbias, int64_t cols, int64_t K, hipStream_t stream) {
  if (dw && w8a8::launch_zero(dw, cols * K, stream) != hipSuccess) return W8A8_ERR_LAUNCH;
  if (dbias && w8a8::launch_zero(dbias, cols, stream) != hipSuccess) return W8A8_ERR_LAUNCH;
  return W8A8_OK;
}

w8a8_status check_back(const uint16_t* dy, const int8_t* xq, const float* x_scale, const int8_t* wq,
                       const float* w_scale, const uint16_t* bias, const uint16_t* dx, const uint16_t* dw,
                       const uint16_t* dbias, int64_t M, int64_t N, int64_t K, bool gated) {
  if (!shape_ok(M, N, K, gated ? 2 : 1)) return W8A8_ERR_SHAPE;
  // (a gated gradient's epilogue addresses a tile's rows of dy the same way)
  if (((dx || gated) && (gated ? up(2 * N, kLine) : up(N, kLine)) > kMaxSummed) || (dw && up(M, kLine) > kMaxSummed))
    return W8A8_ERR_SHAPE;
  const bool codes = dw || (gated && (dx || dbias)), weight = dx || (gated && (dw || dbias));
  if (M > 0) {
    if ((dx || dw || dbias) && !dy) return W8A8_ERR_NULL;
    if ((codes && (!xq || !x_scale)) || (weight && (!wq || !w_scale))) return W8A8_ERR_NULL;
  }
  if (!aligned(dy, 2) || !aligned(dx, 2) || !aligned(dw, 2) || !aligned(dbias, 2) || !aligned(bias, 2))
    return W8A8_ERR_ALIGN;
  if (M > 0 && ((codes && (!aligned(xq, 16) || !aligned(x_scale, 4))) ||
                (weight && (!aligned(wq, 16) || !aligned(w_scale, 4)))))
    return W8A8_ERR_ALIGN;
  return W8A8_OK;
}

w8a8_status check_workspace(const void* ws, size_t have, int64_t need) {
  if (need == 0) return W8A8_OK;
  if (!ws) return W8A8_ERR_NULL;
  if (!aligned(ws, 16)) return W8A8_ERR_ALIGN;
  return have < (size_t)need ? W8A8_ERR_ARG : W8A8_OK;
}

#define TRY(call) \
  if ((call) != hipSuccess) return W8A8_ERR_LAUNCH

// ---- norm and rotation ----

// Without a rotation positions still say which rows are padding; without
// positions either, every row is at some position of any table.
bool positions_matter(int64_t rot, const int32_t* positions) { return rot > 0 || positions != nullptr; }

w8a8_status check_rope(const w8a8::RopeArgs& a, int64_t Hq, int64_t Hk, int64_t D, int64_t rot) {
  if (a.M < 0 || a.M > kMaxRows || Hq < 0 || Hk < 0 || Hq + Hk < 1 || Hq + Hk > 65536 || D < 16 || D > 1024 ||
      D % 16 != 0 || rot < 0 || rot > D || rot % 16 != 0 || a.P < 1 || a.P > INT32_MAX)
    return W8A8_ERR_SHAPE;
  int64_t lanes = 1;
  while (lanes * 16 < D) lanes *= 2;
  if (a.M * (Hq + Hk) * lanes > (int64_t(1) << 31)) return W8A8_ERR_SHAPE;
  if (!(a.eps >= 0.0f)) return W8A8_ERR_ARG;
  return W8A8_OK;
}
w8a8_status check_view(const w8a8::RopeView& v, int64_t heads) {
  if (heads == 0) return W8A8_OK;
  if (!v.p) return W8A8_ERR_NULL;
  return !aligned(v.p, 16) || v.row % 8 != 0 || v.head % 8 != 0 ? W8A8_ERR_ALIGN : W8A8_OK;
}
w8a8_status check_rope_ptrs(const w8a8::RopeArgs& a) {
  for (const auto& c : {check_view(a.q, a.Hq), check_view(a.k, a.Hk), check_view(a.qo, a.Hq), check_view(a.ko, a.Hk)})
    if (c != W8A8_OK) return c;
  if (a.rot > 0 && (!a.cos || !a.sin)) return W8A8_ERR_NULL;
  if (!aligned(a.cos, 16) || !aligned(a.sin, 16) || !aligned(a.qw, 16) || !aligned(a.kw, 16) ||
      !aligned(a.positions, 4))
    return W8A8_ERR_ALIGN;
  return W8A8_OK;
}

w8a8::RopeView view(const uint16_t* p, int64_t row, int64_t head) { return {const_cast<uint16_t*>(p), row, head}; }

}  // namespace

extern "C" {

size_t w8a8_linear_dynamic_workspace(int64_t M, int64_t N, int64_t K) {
  return shape_ok(M, N, K, 1) ? (size_t)dynamic_plan(M, N, K, false, true).bytes : 0;
}

w8a8_status w8a8_linear_dynamic(const uint16_t* x, const int8_t* wq, const float* w_scale, const uint16_t* bias,
                                uint16_t* y, int64_t M, int64_t N, int64_t K, int gelu, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  return dynamic(x, wq, w_scale, bias, y, M, N, K, gelu ? 1 : 0, false, workspace, workspace_bytes, stream);
}

w8a8_status w8a8_gated_linear_tile(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                                   const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int act,
                                   int tile, hipStream_t stream) {
  if (!shape_ok(M, N, K, 2)) return W8A8_ERR_SHAPE;
  if (act < 0 || act > 1 || tile >= w8a8::num_tiles()) return W8A8_ERR_ARG;
  if (M == 0) return W8A8_OK;
  if (!xq || !x_scale || !wq || !w_scale || !y) return W8A8_ERR_NULL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y, 2) ||
      !aligned(bias, 2))
    return W8A8_ERR_ALIGN;
  return launched(w8a8::launch_gated(tile, static_cast<GateAct>(act), xq, x_scale, wq, w_scale, bias, y, M, N, K,
                                     stream));
}

w8a8_status w8a8_gated_linear(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                              const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int act,
                              hipStream_t stream) {
  return w8a8_gated_linear_tile(xq, x_scale, wq, w_scale, bias, y, M, N, K, act, -1, stream);
}

size_t w8a8_gated_linear_dynamic_workspace(int64_t M, int64_t N, int64_t K) {
  return shape_ok(M, N, K, 2) ? (size_t)dynamic_plan(M, N, K, true, true).bytes : 0;
}

w8a8_status w8a8_gated_linear_dynamic(const uint16_t* x, const int8_t* wq, const float* w_scale,
                                      const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int act,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return dynamic(x, wq, w_scale, bias, y, M, N, K, act, true, workspace, workspace_bytes, stream);
}

// Both sizes allow for the copy of dy that an odd N or address needs.
size_t w8a8_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int dx, int dw, int dbias) {
  if (!shape_ok(M, N, K, 1) || M == 0) return 0;
  return back_workspace(M, N, K, false, dx, dw, dbias);
}

w8a8_status w8a8_linear_backward(const uint16_t* dy, const int8_t* xq, const float* x_scale, const int8_t* wq,
                                 const float* w_scale, uint16_t* dx, uint16_t* dw, uint16_t* dbias, int64_t M,
                                 int64_t N, int64_t K, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_back(dy, xq, x_scale, wq, w_scale, nullptr, dx, dw, dbias, M, N, K, false);
  if (st != W8A8_OK) return st;
  if (M == 0) return no_tokens(dw, dbias, N, K, stream);
  const bool few = dx && few_rows(M, N, K) && aligned(dx, 16);
  const bool copy = N % 8 != 0 || !aligned(dy, 16) || (dx && copy_lines(M, N, K));
  const BackPlan p = back_plan(M, N, K, false, dx, dw, dbias, copy, few);
  st = check_workspace(workspace, workspace_bytes, p.bytes);
  if (st != W8A8_OK) return st;
  if (!dx && !dw && !dbias) return W8A8_OK;
  using Job = w8a8::LayoutJob;
  Job jobs[w8a8::kMaxJobs];
  int n = 0;
  const uint16_t* first = dy;
  if (dx && !few) {
    if (copy) {
      jobs[n++] = {Job::kPadRows, dy, nullptr, at<uint16_t>(workspace, p.copy), nullptr, M, N, p.ldy, 0};
      first = at<uint16_t>(workspace, p.copy);
    }
    jobs[n++] = {Job::kTurnCodes, wq, w_scale, at<uint16_t>(workspace, p.wt), nullptr, N, K, p.ld, 0};
  }
  if (dw || dbias)
    jobs[n++] = {Job::kTurnValues, dy, nullptr, dw ? at<uint16_t>(workspace, p.second) : nullptr,
                 dbias ? at<float>(workspace, p.sums) : nullptr, M, N, p.mp, w8a8::transpose_sum_span(M, N)};
  if (dw) jobs[n++] = {Job::kTurnCodes, xq, x_scale, at<uint16_t>(workspace, p.xt), nullptr, M, K, p.mp, 0};
  if (n > 0) TRY(w8a8::launch_prepare(jobs, n, stream));
  return launched(products(p, workspace, first, wq, w_scale, false, dx, dw, dbias, M, N, K, stream));
}

size_t w8a8_gated_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int dx, int dw, int dbias) {
  if (!shape_ok(M, N, K, 2) || M == 0) return 0;
  return back_workspace(M, N, K, true, dx, dw, dbias);
}

w8a8_status w8a8_gated_linear_backward(const uint16_t* dy, const int8_t* xq, const float* x_scale, const int8_t* wq,
                                       const float* w_scale, const uint16_t* bias, uint16_t* dx, uint16_t* dw,
                                       uint16_t* dbias, int64_t M, int64_t N, int64_t K, int act, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_back(dy, xq, x_scale, wq, w_scale, bias, dx, dw, dbias, M, N, K, true);
  if (st != W8A8_OK) return st;
  if (act < 0 || act > 1) return W8A8_ERR_ARG;
  if (M == 0) return no_tokens(dw, dbias, 2 * N, K, stream);
  if (!dx && !dw && !dbias) return W8A8_OK;
  const bool copy = N % 8 != 0 || !aligned(dy, 16);
  const bool few = dx && few_rows(M, 2 * N, K) && aligned(dx, 16);
  const BackPlan p = back_plan(M, N, K, true, dx, dw, dbias, copy, few);
  st = check_workspace(workspace, workspace_bytes, p.bytes);
  if (st != W8A8_OK) return st;
  uint16_t* first = dx ? at<uint16_t>(workspace, p.first) : nullptr;
  uint16_t* second = dw ? at<uint16_t>(workspace, p.second) : nullptr;
  float* sums = dbias ? at<float>(workspace, p.sums) : nullptr;
  using Job = w8a8::LayoutJob;
  Job jobs[w8a8::kMaxJobs];
  int n = 0;
  if (copy) {
    jobs[n++] = {Job::kPadRows, dy, nullptr, at<uint16_t>(workspace, p.copy), nullptr, M, N, p.ldy, 0};
    dy = at<uint16_t>(workspace, p.copy);
  }
  if (dx && !few) jobs[n++] = {Job::kTurnPaired, wq, nullptr, at<uint16_t>(workspace, p.wt), nullptr, 2 * N, K, p.ld, 0};
  if (dw) jobs[n++] = {Job::kTurnCodes, xq, nullptr, at<uint16_t>(workspace, p.xt), nullptr, M, K, p.mp, 0};
  if (n > 0) TRY(w8a8::launch_prepare(jobs, n, stream));
  TRY(w8a8::launch_gated_grad(static_cast<GateAct>(act), dy, p.ldy, xq, x_scale, wq, w_scale, bias, first, p.ld,
                              second, p.mp, sums, M, N, K, stream));
  return launched(products(p, workspace, first, wq, w_scale, true, dx, dw, dbias, M, 2 * N, K, stream));
}

w8a8_status w8a8_qk_norm_rope(const uint16_t* q, int64_t q_row, int64_t q_head, const uint16_t* k, int64_t k_row,
                              int64_t k_head, const uint16_t* q_weight, const uint16_t* k_weight, const float* cos,
                              const float* sin, const int32_t* positions, uint16_t* q_out, int64_t q_out_row,
                              int64_t q_out_head, uint16_t* k_out, int64_t k_out_row, int64_t k_out_head, int64_t M,
                              int64_t P, int64_t Hq, int64_t Hk, int64_t D, int64_t rot, float eps, int interleaved,
                              hipStream_t stream) {
  w8a8::RopeArgs a{view(q, q_row, q_head), view(k, k_row, k_head), view(q_out, q_out_row, q_out_head),
                   view(k_out, k_out_row, k_out_head), q_weight, k_weight, cos, sin, positions,
                   M, positions_matter(rot, positions) ? P : 1, (int)Hq, (int)Hk, (int)D, (int)rot, eps};
  w8a8_status st = check_rope(a, Hq, Hk, D, rot);
  if (st != W8A8_OK || M == 0) return st;
  st = check_rope_ptrs(a);
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_norm_rope(a, interleaved != 0, stream));
}

size_t w8a8_qk_norm_rope_backward_workspace(int64_t M, int64_t Hq, int64_t Hk, int64_t D) {
  if (M < 1 || Hq < 0 || Hk < 0 || D < 16 || D > 1024 || M > kMaxRows || Hq + Hk < 1 || Hq + Hk > 65536) return 0;
  return (size_t)(w8a8::norm_rope_grad_rows(M, Hq, Hk, (int)D) * D * 4);
}

w8a8_status w8a8_qk_norm_rope_backward(
    const uint16_t* dq, int64_t dq_row, int64_t dq_head, const uint16_t* dk, int64_t dk_row, int64_t dk_head,
    const uint16_t* q, int64_t q_row, int64_t q_head, const uint16_t* k, int64_t k_row, int64_t k_head,
    const uint16_t* q_weight, const uint16_t* k_weight, const float* cos, const float* sin, const int32_t* positions,
    uint16_t* dq_in, int64_t dq_in_row, int64_t dq_in_head, uint16_t* dk_in, int64_t dk_in_row, int64_t dk_in_head,
    float* dq_weight, float* dk_weight, int64_t M, int64_t P, int64_t Hq, int64_t Hk, int64_t D, int64_t rot,
    float eps, int interleaved, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  w8a8::RopeArgs a{view(q, q_row, q_head), view(k, k_row, k_head), view(dq, dq_row, dq_head),
                   view(dk, dk_row, dk_head), q_weight, k_weight, cos, sin, positions,
                   M, positions_matter(rot, positions) ? P : 1, (int)Hq, (int)Hk, (int)D, (int)rot, eps};
  w8a8_status st = check_rope(a, Hq, Hk, D, rot);
  if (st != W8A8_OK) return st;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return W8A8_ERR_ALIGN;
  if (M == 0) {
    if (dq_weight) TRY(w8a8::launch_zero(dq_weight, 2 * D, stream));
    if (dk_weight) TRY(w8a8::launch_zero(dk_weight, 2 * D, stream));
    return W8A8_OK;
  }
  const w8a8::RopeView oq = view(dq_in, dq_in_row, dq_in_head), ok = view(dk_in, dk_in_row, dk_in_head);
  st = check_rope_ptrs(a);
  if (st == W8A8_OK) st = check_view(oq, Hq);
  if (st == W8A8_OK) st = check_view(ok, Hk);
  if (st != W8A8_OK) return st;
  const bool sums = dq_weight || dk_weight;
  if (sums) {
    st = check_workspace(workspace, workspace_bytes, (int64_t)w8a8_qk_norm_rope_backward_workspace(M, Hq, Hk, D));
    if (st != W8A8_OK) return st;
  }
  return launched(w8a8::launch_norm_rope_grad(a, oq, ok, interleaved != 0, sums ? static_cast<float*>(workspace) : nullptr,
                                              dq_weight, dk_weight, stream));
}

}  // extern "C"
