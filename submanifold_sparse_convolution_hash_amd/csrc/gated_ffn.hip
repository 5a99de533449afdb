// Gated feed-forward block on site features, and its gradients:
//
//   [g | u] = x W_in + b_in      W_in [C][2F]: gate columns, then up columns
//   h = act(g) u                 (elementwise)
//   out = h W_out + b_out + residual
//
//   dh = dout W_out^T,  du = dh act(g),  dg = dh u act'(g)
//   dx = [dg | du] W_in^T,  dW_in = x^T [dg | du],  dW_out = h^T dout
//
// Both projections, the activation and the product are one kernel: a
// workgroup's tile holds the gate and up columns of the same hidden channels,
// a wave both accumulators of each, so h is formed in registers and g and u
// are written only where the gradient will need them. In the gradient, dg, du
// and h are formed in the epilogue of dh, which is never stored. h, dg and du
// are rounded to 16 bits, as operands of the products that follow have to be;
// the bias gradient adds dg and du before that.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"

namespace submconv {
namespace {

// ---- forward: h = act(x W_g + b_g) (x W_u + b_u) ----
//
// Bound by its per-tile work at few channels (209715 x 128 / 512 fp16 155 us
// without pre, 177-207 with it, which writes 644 MB: a tile of 128 rows has two
// steps of k, then exp and reciprocal of 64 columns).

struct GateEpi {
  const float* bias;  // [2F] or null
  uint16_t* h;        // blocked [M][Fq], Fq = F rounded up to 64, the rest zeros
  uint16_t* pre;      // [M][2F] or null
  int64_t F, Fq;
  int act;
  bool vec_p;
};

template <bool BF16, int ACT, typename R, int NT>
__device__ __forceinline__ void gate_epilogue(const GateEpi& e, int64_t M, int64_t m0, uint32_t n0,
                                              const char* smem) {
  constexpr int BM = R::PH_ROWS;
  // a row in LDS: the gate's columns, then the up projection's
  constexpr int HP = R::PIECES / 2, STEP = NT / HP;
  const int piece = threadIdx.x % HP, r0 = threadIdx.x / HP;
  const uint32_t n = n0 + piece * 8;
  const BlockView h(e.h, m0, M, e.Fq);
  const RowsView pg(e.pre, 2 * e.F, m0, M, e.F, BM, e.vec_p);
  const RowsView pu(e.pre ? e.pre + e.F : nullptr, 2 * e.F, m0, M, e.F, BM, e.vec_p);
  float bg[8], bu[8];
  load_bias8(e.bias, e.F, n, bg);
  load_bias8(e.bias ? e.bias + e.F : nullptr, e.F, n, bu);
#pragma unroll 2
  for (int p = 0; p < BM / STEP; ++p) {
    const int m = r0 + p * STEP;
    float g[8], u[8];
    R::read8(smem, m, piece, g);
    R::read8(smem, m, HP + piece, u);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      g[q] += bg[q];
      u[q] += bu[q];
    }
    if (e.pre) {
      pg.store(m, n, pack8<BF16>(g));
      pu.store(m, n, pack8<BF16>(u));
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) g[q] = act_value<ACT>(g[q]) * u[q];
    h.store(m, n, pack8<BF16>(g));
  }
}

template <bool BF16, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * 64, tile_waves(BM, BN, STAGES)) void k_gate(Operand A, Operand B, int64_t K, int64_t half,
                                                      uint32_t m_tiles, uint32_t n_tiles, GateEpi e) {
  using T = Tile<BF16, false, true, true, BM, BN, WM, WN, STAGES>;
  __shared__ __attribute__((aligned(16))) char smem[T::LDS_BYTES];
  const TilePos t = tile_pos(m_tiles, n_tiles, blockIdx.x);
  const int64_t m0 = t.m * BM, n0 = t.n * (BN / 2);
  float4v acc[T::FN][T::FM];
  T::run(A, B, half, m0, n0, 0, K, smem, acc);
#pragma unroll 1
  for (int ph = 0; ph < T::PHASES; ++ph) {
    T::to_rows(smem, ph, acc);
    with_act(e.act, [&](auto a) {
      gate_epilogue<BF16, decltype(a)::value, typename T::Rows, T::NT>(e, A.rows, m0 + ph * T::Rows::PH_ROWS,
                                                 static_cast<uint32_t>(n0), smem);
    });
  }
}

// ---- gradient: dh = dout W_out^T; dg, du, h in its epilogue ----
//
// Memory-bound: 209715 x 256 / 1024 bf16 reads pre and dout once and writes dg,
// du and h, 2.3 GB in 450-470 us (5.0 TB/s).

struct GateGradEpi {
  const uint16_t* pre;  // [M][2F]
  uint16_t* dz;         // blocked [M][2Fq]: dg, zeros up to Fq, du, zeros
  uint16_t* h;          // blocked [M][Fq]
  float* sums;          // [m_tiles][2Fq] column sums of the tile's dg and du, or null
  int64_t F, Fq;
  int act;
  bool vec_p;
};

template <bool BF16, int ACT, typename R>
__device__ __forceinline__ void gate_grad_epilogue(const GateGradEpi& e, int64_t M, int64_t m0,
                                                   uint32_t n0, const char* smem, float (&sg)[8],
                                                   float (&su)[8]) {
  constexpr int BM = R::PH_ROWS;
  const int piece = threadIdx.x % R::PIECES, r0 = threadIdx.x / R::PIECES;
  const uint32_t n = n0 + piece * 8;
  const RowsView pg(e.pre, 2 * e.F, m0, M, e.F, BM, e.vec_p);
  const RowsView pu(e.pre + e.F, 2 * e.F, m0, M, e.F, BM, e.vec_p);
  const BlockView z(e.dz, m0, M, 2 * e.Fq);
  const uint32_t Fq = static_cast<uint32_t>(e.Fq);
  const BlockView h(e.h, m0, M, e.Fq);
#pragma unroll 2
  for (int p = 0; p < R::ROW_PASSES; ++p) {
    const int m = r0 + p * R::ROW_STEP;
    float g[8], u[8], dh[8];
    unpack8<BF16>(pg.load(m, n), g);
    unpack8<BF16>(pu.load(m, n), u);
    R::read8(smem, m, piece, dh);
    float dg[8], du[8], v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float a, d;
      act_both<ACT>(g[q], a, d);
      dg[q] = dh[q] * u[q] * d;
      du[q] = dh[q] * a;
      v[q] = a * u[q];
      sg[q] += dg[q];  // rows past M add zeros: their dout is read as zeros
      su[q] += du[q];
    }
    if (n < Fq) {
      z.store(m, n, pack8<BF16>(dg));
      z.store(m, Fq + n, pack8<BF16>(du));
      h.store(m, n, pack8<BF16>(v));
    }
  }
}

template <bool BF16, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * 64, tile_waves(BM, BN, STAGES)) void k_gate_grad(Operand A, Operand B, int64_t K,
                                                           uint32_t m_tiles, uint32_t n_tiles,
                                                           GateGradEpi e) {
  using T = Tile<BF16, false, false, false, BM, BN, WM, WN, STAGES>;
  __shared__ __attribute__((aligned(16))) char smem[T::LDS_BYTES];
  const TilePos t = tile_pos(m_tiles, n_tiles, blockIdx.x);
  const int64_t m0 = t.m * BM, n0 = t.n * BN;
  float4v acc[T::FN][T::FM];
  T::run(A, B, 0, m0, n0, 0, K, smem, acc);
  float sums[2][8] = {};
#pragma unroll 1
  for (int ph = 0; ph < T::PHASES; ++ph) {
    T::to_rows(smem, ph, acc);
    with_act(e.act, [&](auto a) {
      gate_grad_epilogue<BF16, decltype(a)::value, typename T::Rows>(e, A.rows, m0 + ph * T::Rows::PH_ROWS,
                                                      static_cast<uint32_t>(n0), smem, sums[0], sums[1]);
    });
  }
  if (!e.sums) return;
  // the threads that walked the same columns, in order
  float* red = reinterpret_cast<float*>(smem);  // [ROW_STEP][2][BN]
  const int piece = threadIdx.x % T::Rows::PIECES, r0 = threadIdx.x / T::Rows::PIECES;
  __syncthreads();
#pragma unroll
  for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
    for (int q = 0; q < 8; ++q) red[(r0 * 2 + t2) * BN + piece * 8 + q] = sums[t2][q];
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * BN; c += T::NT) {
    float x = 0.0f;
#pragma unroll
    for (int r = 0; r < T::Rows::ROW_STEP; ++r) x += red[r * 2 * BN + c];
    const int64_t n = n0 + c % BN;
    if (n < e.Fq) e.sums[(t.m * 2 + c / BN) * e.Fq + n] = x;
  }
}

constexpr int kGateTile = 128;

int gate_forward(const Mat16& x, const Mat16& W, int64_t F, const float* bias, int act, bool bf16,
                 uint16_t* h, uint16_t* pre, hipStream_t stream) {
  const int64_t Fp = W.cols / 2, Fq = round64(F);
  const int64_t mt = div_up(x.rows, kGateTile), nt = div_up(Fq, kGateTile / 2);
  if (!launch_fits(mt * nt, 512))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "too many output tiles: %lld", (long long)(mt * nt));
  const GateEpi e{bias, h, pre, F, Fq, act, F % 8 == 0 && aligned16(pre)};
  const Operand A{x.p, x.ld, x.rows, x.cols}, B{W.p, W.ld, Fp, W.rows};
  const dim3 grid(static_cast<unsigned>(mt * nt));
  auto go = [&](auto st) {
    if (bf16) k_gate<true, kGateTile, kGateTile, 2, 4, st><<<grid, 512, 0, stream>>>(A, B, x.cols, Fp, mt, nt, e);
    else k_gate<false, kGateTile, kGateTile, 2, 4, st><<<grid, 512, 0, stream>>>(A, B, x.cols, Fp, mt, nt, e);
  };
  if (mt * nt <= 256) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 2>{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int64_t gate_grad_tiles(int64_t rows) { return std::max<int64_t>(1, div_up(rows, kGateTile)); }

// dy [M][C], W_out [F][C]
int gate_grad(const Mat16& dy, const Mat16& W, int64_t Fq, const uint16_t* pre, int act, bool bf16,
              uint16_t* dz, uint16_t* h, float* sums, hipStream_t stream) {
  const int64_t F = W.rows;
  const int64_t mt = gate_grad_tiles(dy.rows), nt = div_up(Fq, kGateTile);
  if (!launch_fits(mt * nt, 512))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "too many output tiles: %lld", (long long)(mt * nt));
  const GateGradEpi e{pre, dz, h, sums, F, Fq, act, F % 8 == 0 && aligned16(pre)};
  const Operand A{dy.p, dy.ld, dy.rows, dy.cols}, B{W.p, W.ld, F, W.cols};
  const dim3 grid(static_cast<unsigned>(mt * nt));
  auto go = [&](auto st) {
    if (bf16) k_gate_grad<true, kGateTile, kGateTile, 2, 4, st><<<grid, 512, 0, stream>>>(A, B, dy.cols, mt, nt, e);
    else k_gate_grad<false, kGateTile, kGateTile, 2, 4, st><<<grid, 512, 0, stream>>>(A, B, dy.cols, mt, nt, e);
  };
  if (mt * nt <= 256) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 2>{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

struct Ffn {
  int64_t n, C, F, Co;
  Mat16 x, W_in, W_out, dy;  // W_in [C][2F], W_out [F][Co]
  int act;
  bool bf16;
};

// `keeps`: pre is asked for (it may be null while the arena counts).
int ffn_forward(const Ffn& f, bool keeps, const float* b_in, const float* b_out,
                const uint16_t* residual, int64_t ldr, uint16_t* out, uint16_t* pre, Arena& ws,
                hipStream_t stream) {
  if (f.n <= kFewRows) {
    float* h = static_cast<float*>(ws.take(f.n * f.F * 4));
    if (ws.counting || f.n == 0) return SUBMCONV_OK;
    SUBMCONV_TRY(few_gate(f.x, f.W_in, b_in, f.act, f.bf16, h, pre, stream));
    return few_out(h, f.n, f.W_out, b_out, f.bf16, residual, ldr, out, stream);
  }
  const int64_t Fq = round64(f.F);
  PackList packs;
  const Mat16 x = readable(f.x, 1, 8, ws, &packs), wi = readable(f.W_in, 2, 8, ws, &packs);
  const Mat16 wo = readable(f.W_out, 1, 8, ws, &packs);
  if (!keeps && fused_ffn_takes(f.n, f.C, f.F, f.Co)) {
    if (ws.counting) return SUBMCONV_OK;
    SUBMCONV_TRY(run_packs(packs, stream));
    return fused_ffn(x, wi, f.F, b_in, wo, b_out, f.act, f.bf16, residual, ldr, out, f.Co, stream);
  }
  uint16_t* h = static_cast<uint16_t*>(ws.take(blocked_bytes(f.n, Fq)));
  if (ws.counting) return SUBMCONV_OK;
  SUBMCONV_TRY(run_packs(packs, stream));
  SUBMCONV_TRY(gate_forward(x, wi, f.F, b_in, f.act, f.bf16, h, pre, stream));
  return linear_forward(blocked16(h, f.n, Fq), wo, b_out, kActNone, f.bf16, residual, ldr, out, f.Co,
                        nullptr, f.Co, stream);
}

struct FfnGrads {
  uint16_t *x, *W_in, *W_out;
  float *b_in, *b_out;
  bool all;  // count the workspace of every gradient
};

int ffn_backward(const Ffn& f, const uint16_t* pre, const FfnGrads& g, Arena& ws, hipStream_t stream) {
  const int64_t Fq = round64(f.F), Cp = round8(f.C), Op = round8(f.Co);
  const bool need_x = g.all || g.x, need_wi = g.all || g.W_in, need_wo = g.all || g.W_out;
  const bool need_bi = g.all || g.b_in, need_bo = g.all || g.b_out;
  const bool hidden = need_x || need_wi || need_wo || need_bi;
  PackList packs;
  Mat16 dy, x, wi, wo;
  if (hidden) {
    dy = readable(f.dy, 1, 8, ws, &packs);
    wo = readable(f.W_out, 1, 8, ws, &packs);
  }
  if (need_x) wi = readable(f.W_in, 2, 64, ws, &packs);
  if (need_wi) x = readable(f.x, 1, 8, ws, &packs);
  float* dy_sums = need_bo ? static_cast<float*>(ws.take(column_parts(f.n, f.Co) * Op * 4)) : nullptr;
  const int64_t tiles = gate_grad_tiles(f.n);
  uint16_t* h = hidden ? static_cast<uint16_t*>(ws.take(blocked_bytes(f.n, Fq))) : nullptr;
  uint16_t* dz = hidden ? static_cast<uint16_t*>(ws.take(blocked_bytes(f.n, 2 * Fq))) : nullptr;
  float* sums = need_bi ? static_cast<float*>(ws.take(tiles * 2 * Fq * 4)) : nullptr;
  float* part_x = need_x ? static_cast<float*>(ws.take(product_nt_bytes(f.n, 2 * Fq, f.C))) : nullptr;
  float* part_wi = need_wi ? static_cast<float*>(ws.take(product_tn_bytes(f.n, Cp, 2 * Fq))) : nullptr;
  float* part_wo = need_wo ? static_cast<float*>(ws.take(product_tn_bytes(f.n, Fq, Op))) : nullptr;
  if (ws.counting) return SUBMCONV_OK;

  PlaneList planes;
  SumList columns;
  SUBMCONV_TRY(run_packs(packs, stream));
  if (need_bo) SUBMCONV_TRY(column_sums(f.dy, f.bf16, dy_sums, g.b_out, &columns, stream));
  if (hidden) {
    const Mat16 hm = blocked16(h, f.n, Fq), zm = blocked16(dz, f.n, 2 * Fq);
    SUBMCONV_TRY(gate_grad(dy, wo, Fq, pre, f.act, f.bf16, dz, h, sums, stream));
    if (need_bi) columns.job[columns.count++] = SumJob{sums, tiles, 2 * Fq, 2 * f.F, 2, g.b_in};
    if (need_x) SUBMCONV_TRY(product_nt(zm, wi, f.bf16, part_x, g.x, f.C, &planes, stream));
    if (need_wi) SUBMCONV_TRY(product_tn(x, zm, f.bf16, part_wi, g.W_in, f.C, 2 * f.F, 2, &planes, stream));
    if (need_wo) SUBMCONV_TRY(product_tn(hm, dy, f.bf16, part_wo, g.W_out, f.F, f.Co, 1, &planes, stream));
  }
  SUBMCONV_TRY(run_planes(planes, f.bf16, stream));
  return run_sums(columns, stream);
}

int ffn_shape(int64_t n, int32_t cin, int32_t hidden, int32_t cout) {
  SUBMCONV_TRY(check_shape("x", n, cin));
  if (hidden < 1 || hidden > (1 << 19))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "hidden = %d", hidden);
  return check_shape("out", n, cout);
}

int64_t ffn_workspace(int64_t n, int32_t cin, int32_t hidden, int32_t cout, int32_t aligned, bool keeps) {
  clear_error();
  SUBMCONV_TRY(ffn_shape(n, cin, hidden, cout));
  const Ffn f{n, cin, hidden, cout, shape_of(n, cin, aligned), shape_of(cin, 2 * hidden, aligned),
              shape_of(hidden, cout, aligned), {}, kActSilu, false};
  Arena ws;
  SUBMCONV_TRY(ffn_forward(f, keeps, nullptr, nullptr, nullptr, 0, nullptr, nullptr, ws, nullptr));
  return ws.used;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int64_t submconv_gated_ffn_workspace_bytes(int64_t n, int32_t cin, int32_t hidden,
                                                      int32_t cout, int32_t aligned) {
  return ffn_workspace(n, cin, hidden, cout, aligned, true);
}

extern "C" int64_t submconv_gated_ffn_inference_workspace_bytes(int64_t n, int32_t cin,
                                                                int32_t hidden, int32_t cout,
                                                                int32_t aligned) {
  return ffn_workspace(n, cin, hidden, cout, aligned, false);
}

extern "C" int submconv_gated_ffn(const uint16_t* x, int64_t ldx, int64_t n, const uint16_t* W_in,
                                  const float* b_in, const uint16_t* W_out, const float* b_out,
                                  const uint16_t* residual, int64_t ldr, uint16_t* out,
                                  uint16_t* pre, int32_t cin, int32_t hidden, int32_t cout,
                                  int32_t act, int32_t dtype, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_kind(act, dtype));
  SUBMCONV_TRY(ffn_shape(n, cin, hidden, cout));
  SUBMCONV_TRY(check_matrix("x", x, n, cin, ldx));
  SUBMCONV_TRY(check_matrix("W_in", W_in, cin, 2 * int64_t{hidden}, 2 * int64_t{hidden}));
  SUBMCONV_TRY(check_matrix("W_out", W_out, hidden, cout, cout));
  SUBMCONV_TRY(check_matrix("out", out, n, cout, cout));
  if (residual) SUBMCONV_TRY(check_matrix("residual", residual, n, cout, ldr));
  if (pre) SUBMCONV_TRY(check_matrix("pre", pre, n, 2 * int64_t{hidden}, 2 * int64_t{hidden}));
  const Ffn f{n, cin, hidden, cout, Mat16{x, n, cin, n == 1 ? round8(cin) : ldx},
              Mat16{W_in, cin, 2 * int64_t{hidden}, 2 * int64_t{hidden}},
              Mat16{W_out, hidden, cout, cout}, {}, act, dtype == SUBMCONV_DTYPE_BF16};
  const int64_t lr = n == 1 ? round8(cout) : ldr;
  Arena count;
  SUBMCONV_TRY(ffn_forward(f, pre != nullptr, b_in, b_out, residual, lr, out, pre, count, stream));
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, count.used));
  Arena ws{false, static_cast<char*>(workspace)};
  return ffn_forward(f, pre != nullptr, b_in, b_out, residual, lr, out, pre, ws, stream);
}

extern "C" int64_t submconv_gated_ffn_backward_workspace_bytes(int64_t n, int32_t cin,
                                                               int32_t hidden, int32_t cout,
                                                               int32_t aligned) {
  clear_error();
  SUBMCONV_TRY(ffn_shape(n, cin, hidden, cout));
  const Ffn f{n, cin, hidden, cout, shape_of(n, cin, aligned), shape_of(cin, 2 * hidden, aligned),
              shape_of(hidden, cout, aligned), shape_of(n, cout, aligned), kActSilu, false};
  Arena ws;
  SUBMCONV_TRY(ffn_backward(f, nullptr, {nullptr, nullptr, nullptr, nullptr, nullptr, true}, ws, nullptr));
  return ws.used;
}

extern "C" int submconv_gated_ffn_backward(const uint16_t* grad_out, int64_t ldg, int64_t n,
                                           const uint16_t* x, int64_t ldx, const uint16_t* W_in,
                                           const uint16_t* W_out, const uint16_t* pre,
                                           uint16_t* grad_x, uint16_t* grad_w_in, float* grad_b_in,
                                           uint16_t* grad_w_out, float* grad_b_out, int32_t cin,
                                           int32_t hidden, int32_t cout, int32_t act, int32_t dtype,
                                           void* workspace, int64_t workspace_bytes,
                                           hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_kind(act, dtype));
  SUBMCONV_TRY(ffn_shape(n, cin, hidden, cout));
  SUBMCONV_TRY(check_matrix("grad_out", grad_out, n, cout, ldg));
  if (grad_w_in) SUBMCONV_TRY(check_matrix("x", x, n, cin, ldx));
  if (grad_x) SUBMCONV_TRY(check_matrix("W_in", W_in, cin, 2 * int64_t{hidden}, 2 * int64_t{hidden}));
  SUBMCONV_TRY(check_matrix("W_out", W_out, hidden, cout, cout));
  SUBMCONV_TRY(check_matrix("pre", pre, n, 2 * int64_t{hidden}, 2 * int64_t{hidden}));
  const Ffn f{n, cin, hidden, cout, Mat16{x, n, cin, n == 1 ? round8(cin) : ldx},
              Mat16{W_in, cin, 2 * int64_t{hidden}, 2 * int64_t{hidden}},
              Mat16{W_out, hidden, cout, cout},
              Mat16{grad_out, n, cout, n == 1 ? round8(cout) : ldg}, act,
              dtype == SUBMCONV_DTYPE_BF16};
  const FfnGrads g{grad_x, grad_w_in, grad_w_out, grad_b_in, grad_b_out, false};
  Arena count;
  SUBMCONV_TRY(ffn_backward(f, pre, g, count, stream));
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, count.used));
  Arena ws{false, static_cast<char*>(workspace)};
  return ffn_backward(f, pre, g, ws, stream);
}
