// Epilogue of a linear layer: act(z + bias) + residual from fp32 rows in LDS.
#pragma once

#include "dense_tile.h"

namespace submconv {
namespace {

struct LinearEpi {
  const float* bias;         // [N] or null
  const uint16_t* residual;  // or null
  int64_t ldr;
  uint16_t* out;
  int64_t ldo;
  uint16_t* pre;  // [M][N] dense, or null
  int act;
  bool vec_r, vec_o, vec_p;
};

template <bool BF16, int ACT, typename R>
__device__ __forceinline__ void linear_epilogue(const LinearEpi& e, int64_t M, int64_t N,
                                                int64_t m0, uint32_t n0, const char* smem) {
  constexpr int BM = R::PH_ROWS;
  const int piece = threadIdx.x % R::PIECES, r0 = threadIdx.x / R::PIECES;
  const uint32_t n = n0 + piece * 8;
  const RowsView out(e.out, e.ldo, m0, M, N, BM, e.vec_o);
  const RowsView pre(e.pre, N, m0, M, N, BM, e.vec_p);
  const RowsView res(e.residual, e.ldr, m0, M, N, BM, e.vec_r);
  float b[8];
  load_bias8(e.bias, N, n, b);
  // four rows' loads of the residual in flight (209715 rows of 128 / 512 in the
  // gated block 130 -> 123 us; linear 128 -> 512 98 -> 95 us)
#pragma unroll 4
  for (int p = 0; p < R::ROW_PASSES; ++p) {
    const int m = r0 + p * R::ROW_STEP;
    float z[8];
    R::read8(smem, m, piece, z);
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] += b[q];
    if (e.pre) pre.store(m, n, pack8<BF16>(z));
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] = act_value<ACT>(z[q]);
    if (e.residual) {
      float v[8];
      unpack8<BF16>(res.load(m, n), v);
#pragma unroll
      for (int q = 0; q < 8; ++q) z[q] += v[q];
    }
    out.store(m, n, pack8<BF16>(z));
  }
}

}  // namespace
}  // namespace submconv
