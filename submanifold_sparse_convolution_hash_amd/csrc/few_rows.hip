// Forward products of a few rows (at most kFewRows) with a weight matrix: one
// conditioning vector, one timestep, a handful of sites. A product reads its
// whole weight matrix for 2 flops per row and element, so it is bound by the
// weights' way to the compute units and, at the usual sizes, by its latency:
// one launch, no join between workgroups, no LDS tiles.
//
// A workgroup owns a strip of LPR x 8 columns for all rows. Each thread walks
// every (512 / LPR)-th row of W, 16 bytes at a time, straight from memory into
// fp32 products with the rows of x, read beside it; the threads' sums are joined
// by lane exchanges, then through LDS, in one fixed order. The gated block's
// hidden rows pass between its two launches in fp32: nothing here needs them in 16
// bits, and they are a few KB beside the weights.
//
// At 1 x 256 -> 1024 it takes 3.2 us, at 1 x 512 / 2048 (gated) 4.6 + 4.4, or
// 5.2 + 6.6 with weights that no L2 holds. The MFMA tile kernels' rows are mostly
// empty here and a workgroup walks all of k in steps of a memory latency each: 8 rows here
// against 9 there take 6.9 and 6.4 us at 256 -> 1024, 8.4 and 13.0 at 1024 -> 1024.
// At a long k the rows from 9 on pay for it (4096 -> 1024 19 us at 8 rows, 40 at 9):
// their products have no split over k.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "lane_ops.h"

namespace submconv {
namespace {

constexpr int kFewThreads = 512;

struct FewEpi {
  const float* bias;
  const uint16_t* residual;
  int64_t ldr;
  uint16_t* out;   // 16-bit result, or
  float* out32;    // fp32 result (the hidden rows between two products)
  uint16_t* pre;   // or null; GATED: [rows][2 N]
  int act;
};

template <bool BF16, typename X>
__device__ __forceinline__ float few_x(X v) {
  if constexpr (std::is_same_v<X, float>) return v;
  else return to_f32<BF16>(v);
}

// out[m][n] = epilogue(sum_k x[m][k] W[k][n]), m < M; GATED: the gate's N
// columns of W, then the up projection's, out = act(gate) up.
template <bool BF16, typename X, int M, int LPR, bool GATED>
__global__ __launch_bounds__(kFewThreads) void k_few(const X* __restrict__ x, int64_t ldx, int rows,
                                                     const uint16_t* __restrict__ W, int64_t ldw,
                                                     int64_t K, int64_t N, FewEpi e) {
  constexpr int H = GATED ? 2 : 1;
  constexpr int SLICES = kFewThreads / LPR, COLS = LPR * 8, WAVES = kFewThreads / 64;
  __shared__ float sums[WAVES][H][M][COLS];
  const int l = threadIdx.x % LPR, slice = threadIdx.x / LPR;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * COLS, n = n0 + l * 8;
  float acc[H][M][8] = {};
#pragma unroll 4
  for (int64_t k = slice; k < K; k += SLICES) {
    float v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = few_x<BF16>(x[(m < rows ? m : 0) * ldx + k]);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float w[8];
      unpack8<BF16>(load_piece(W + k * ldw + h * N, n, N), w);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[h][m][q] += v[m] * w[q];
    }
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float v = lanes_sum_over<LPR>(acc[h][m][q]);
        if (lane < LPR) sums[wave][h][m][l * 8 + q] = v;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < M * COLS; i += kFewThreads) {
    const int m = i / COLS, c = i % COLS;
    const int64_t col = n0 + c;
    if (m >= rows || col >= N) continue;
    float z[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      z[h] = e.bias ? e.bias[h * N + col] : 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) z[h] += sums[w][h][m][c];
      if (e.pre) e.pre[(m * H + h) * N + col] = to_16<BF16>(z[h]);
    }
    float v = 0.0f;
    with_act(e.act, [&](auto a) { v = act_value<decltype(a)::value>(z[0]); });
    if constexpr (GATED) v *= z[H - 1];
    if (e.residual) v += to_f32<BF16>(e.residual[m * e.ldr + col]);
    if (e.out32) e.out32[m * N + col] = v;
    else e.out[m * N + col] = to_16<BF16>(v);
  }
}

template <bool BF16, typename X, bool GATED>
int launch_few(const X* x, int64_t ldx, int rows, const Mat16& W, int64_t N, const FewEpi& e,
               hipStream_t stream) {
  auto go = [&](auto m, auto lpr) {
    const dim3 grid(static_cast<unsigned>(div_up(N, lpr * 8)));
    k_few<BF16, X, m, lpr, GATED><<<grid, kFewThreads, 0, stream>>>(x, ldx, rows, W.p, W.ld,
                                                                   W.rows, N, e);
  };
  // Strips of 128 bytes take whole memory lines; more rows hold too many sums a
  // thread for them until there are strips for every compute unit, and a narrow
  // matrix has too few strips, the more so the longer each one's walk along k is.
  // With strips of 32 / 64 / 128 bytes, in us:
  // 1 row of 300 -> 77 5.9 / 6.5 / 7.9, 256 -> 1024 3.4 / 3.4 / 3.2, 1024 -> 4096
  // 7.6 / 5.5 / 4.8, 4096 -> 8192 43 / 21 / 12; 8 rows of 1024 -> 1024 8.4 / 8.4
  // / 10.8, 1024 -> 4096 11.2 / 9.3 / 11.1, 512 -> 16384 27 / 15 / 8.7. Long walks:
  // 1 row of 4096 -> 320 8.0 / 8.0 / 9.9, 4096 -> 1024 14.9 / 15.9 / 15.8, 8192 -> 512
  // 25.5 / 29.0 / 28.7, but 2048 -> 2048 9.7 / 9.8 / 9.7, 8192 -> 2048 26.7 / 20.7 /
  // 20.5; 8 rows of 4096 -> 320 13.3 / 16.4 / 26, 4096 -> 1024 19.0 / 21.5 / 27.7.
  // (The gated block's second product, one row, both launches, narrow against not: 512
  // / 4096 22.0 against 24.7, 1024 / 4096 26.3 against 29.0; with all weights in L2 512 /
  // 2048 7.9 against 9.7, but 1024 / 4096 18.4 against 14.5.)
  constexpr std::integral_constant<int, 1> one;
  constexpr std::integral_constant<int, 2> two;
  constexpr std::integral_constant<int, 4> four;
  constexpr std::integral_constant<int, 8> eight;
  static_assert(kFewRows == 8);
  if (N <= 256 || (N <= 1024 && W.rows >= 4 * N)) {
    if (rows <= 1) go(one, two);
    else if (rows <= 2) go(two, two);
    else if (rows <= 4) go(four, two);
    else go(eight, two);
  } else if (rows <= 2 || N >= 8192) {
    if (rows <= 1) go(one, eight);
    else if (rows <= 2) go(two, eight);
    else if (rows <= 4) go(four, eight);
    else go(eight, eight);
  } else {
    if (rows <= 4) go(four, four);
    else go(eight, four);
  }
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

}  // namespace

int few_linear(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16,
               const uint16_t* residual, int64_t ldr, uint16_t* out, uint16_t* pre,
               hipStream_t stream) {
  const FewEpi e{bias, residual, ldr, out, nullptr, pre, act};
  const int rows = static_cast<int>(x.rows);
  return bf16 ? launch_few<true, uint16_t, false>(x.p, x.ld, rows, W, W.cols, e, stream)
              : launch_few<false, uint16_t, false>(x.p, x.ld, rows, W, W.cols, e, stream);
}

int few_gate(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16, float* h,
             uint16_t* pre, hipStream_t stream) {
  const FewEpi e{bias, nullptr, 0, nullptr, h, pre, act};
  const int rows = static_cast<int>(x.rows);
  return bf16 ? launch_few<true, uint16_t, true>(x.p, x.ld, rows, W, W.cols / 2, e, stream)
              : launch_few<false, uint16_t, true>(x.p, x.ld, rows, W, W.cols / 2, e, stream);
}

int few_out(const float* h, int64_t rows, const Mat16& W, const float* bias, bool bf16,
            const uint16_t* residual, int64_t ldr, uint16_t* out, hipStream_t stream) {
  const FewEpi e{bias, residual, ldr, out, nullptr, nullptr, kActNone};
  return bf16 ? launch_few<true, float, false>(h, W.rows, static_cast<int>(rows), W, W.cols, e, stream)
              : launch_few<false, float, false>(h, W.rows, static_cast<int>(rows), W, W.cols, e, stream);
}

}  // namespace submconv
