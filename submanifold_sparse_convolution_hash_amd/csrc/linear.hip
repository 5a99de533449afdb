// Linear layer on site features with its epilogue fused, and its gradients:
// the point-wise layers around a SubMConv3d (a 1x1x1 convolution is x W + b).
//
//   z = x W + b,  out = act(z) + residual
//   dz = dout act'(z),  dx = dz W^T,  dW = x^T dz,  db = sum over rows of dz
//
// The products run on the MFMA tile of dense_tile.h with fp32 accumulation;
// bias, activation and residual are applied to the fp32 accumulators and each
// stored tensor is rounded once. dz is rounded to 16 bits before its two
// products, as MFMA operands have to be; the bias gradient adds it unrounded.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "linear_epilogue.h"

namespace submconv {
namespace {

// ---- forward ----

// B_ROW: W [K][N] as stored (forward); else W [N][K] (input gradient). A row
// strip of A is read once from memory and shared by its n tiles through the
// XCD's L2 (tile_pos). With few channels it is bound by memory: 209715 x 128 ->
// 512 bf16 with pre-activations moves 484 MB in 95-100 us, a copy's rate; with
// many by LDS, which feeds the matrix units about 100 bytes a clock: 209715 x
// 2048 -> 256 281 us (780 TFLOP/s), 8192^3 on the wide tile 920 us (1195).
template <bool BF16, bool B_ROW, bool A_TILED, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * 64, tile_waves(BM, BN, STAGES)) void k_linear(Operand A, Operand B, int64_t K, int64_t N,
                                                        uint32_t m_tiles, uint32_t n_tiles,
                                                        LinearEpi e) {
  using T = Tile<BF16, false, B_ROW, false, BM, BN, WM, WN, STAGES, A_TILED>;
  __shared__ __attribute__((aligned(16))) char smem[T::LDS_BYTES];
  const TilePos t = tile_pos(m_tiles, n_tiles, blockIdx.x);
  const int64_t m0 = t.m * BM, n0 = t.n * BN;
  float4v acc[T::FN][T::FM];
  T::run(A, B, 0, m0, n0, 0, K, smem, acc);
#pragma unroll 1
  for (int ph = 0; ph < T::PHASES; ++ph) {
    T::to_rows(smem, ph, acc);
    with_act(e.act, [&](auto a) {
      linear_epilogue<BF16, decltype(a)::value, typename T::Rows>(e, A.rows, N, m0 + ph * T::Rows::PH_ROWS,
                                                   static_cast<uint32_t>(n0), smem);
    });
  }
}

template <bool B_ROW, bool A_TILED, int BM, int BN, int WM, int WN, int STAGES>
int launch_linear(const Operand& A, const Operand& B, int64_t K, int64_t N, bool bf16,
                  const LinearEpi& e, hipStream_t stream) {
  const int64_t mt = div_up(A.rows, BM), nt = div_up(N, BN);
  if (mt * nt > INT32_MAX)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%lld output tiles", (long long)(mt * nt));
  const dim3 grid(static_cast<unsigned>(mt * nt));
  if (bf16)
    k_linear<true, B_ROW, A_TILED, BM, BN, WM, WN, STAGES><<<grid, WM * WN * 64, 0, stream>>>(A, B, K, N, mt, nt, e);
  else
    k_linear<false, B_ROW, A_TILED, BM, BN, WM, WN, STAGES><<<grid, WM * WN * 64, 0, stream>>>(A, B, K, N, mt, nt, e);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

// The tile of a product: 256 x 256 reads half as much LDS and cache per product
// as 128 x 128, but is alone on its compute unit, where nothing covers its
// epilogue or its wait for memory. It is taken where a product has many
// products per element moved (K N / (K + N)) and enough tiles for every unit.
// Measured alone, repeated on the same operands, 128 against 256: 209715 x 2048 ->
// 256 (228) 284 against 287 us, 65536 x 1024 -> 1024 (512) 154 against 140, 8192^3
// 1229 against 920; 209715 x 1024 -> 256 (205) 150 against 156, 100003 x 1024 -> 256
// 67.5 against 72, 209715 x 512 -> 128 (102) 51 against 80.
bool wide_tile(int64_t M, int64_t K, int64_t N) {
  return N >= 256 && K * N / (K + N) >= 240 && div_up(M, 256) * div_up(N, 256) >= 256;
}

// a [M][K], and B [K][N] (B_ROW) or [N][K]
template <bool B_ROW>
int linear_product(const Mat16& a, const Operand& B, int64_t N, bool bf16, const LinearEpi& e,
                   hipStream_t stream) {
  if (a.rows == 0 || N == 0) return SUBMCONV_OK;
  const Operand A{a.p, a.ld, a.rows, a.cols};
  if (wide_tile(a.rows, a.cols, N))
    return a.blocked ? launch_linear<B_ROW, true, 256, 256, 2, 4, 2>(A, B, a.cols, N, bf16, e, stream)
                     : launch_linear<B_ROW, false, 256, 256, 2, 4, 2>(A, B, a.cols, N, bf16, e, stream);
  if (few_tiles(a.rows, N))
    return a.blocked ? launch_linear<B_ROW, true, 128, 128, 2, 4, 4>(A, B, a.cols, N, bf16, e, stream)
                     : launch_linear<B_ROW, false, 128, 128, 2, 4, 4>(A, B, a.cols, N, bf16, e, stream);
  return a.blocked ? launch_linear<B_ROW, true, 128, 128, 2, 4, 3>(A, B, a.cols, N, bf16, e, stream)
                   : launch_linear<B_ROW, false, 128, 128, 2, 4, 3>(A, B, a.cols, N, bf16, e, stream);
}

// ---- padded copies ----

// Up to kPacks copies in one launch, one grid row each: thread i of a copy
// writes its 16-byte piece i. I: 32-bit indices where a copy has fewer pieces
// (a division of 64 bits costs more than the rest of the loop).
struct Packs {
  PackJob job[kPacks];
};
template <typename I>
__global__ __launch_bounds__(256) void k_pack16(Packs p) {
  const PackJob& a = p.job[blockIdx.y];
  const I row_pieces = static_cast<I>(a.row_pieces), to_cols = static_cast<I>(a.to_cols);
  const I pieces = static_cast<I>(a.rows) * row_pieces, step = gridDim.x * blockDim.x;
  for (I i = blockIdx.x * blockDim.x + threadIdx.x; i < pieces; i += step) {
    const I r = i / row_pieces, c = (i - r * row_pieces) * 8;
    const I grp = c / to_cols, cc = c - grp * to_cols;
    reinterpret_cast<u32x4*>(a.to)[i] =
        load_piece(a.from + static_cast<int64_t>(r) * a.ld + grp * a.from_cols, cc, a.from_cols);
  }
}

// ---- dz and column sums ----

constexpr int kSumThreads = 256;
constexpr int kSumLanes = 32;                      // pieces (of 8 columns) a workgroup covers
constexpr int kSumRows = kSumThreads / kSumLanes;  // rows per pass

// Memory-bound: 100003 x 1024 bf16 with silu, 614 MB in 112-115 us (5.4 TB/s).
// dz = dy act'(z), rounded, into a blocked matrix of `blocks` x 64 columns
// (zeros past the width), where dz is not null; and the unrounded column sums of this
// workgroup's rows, where partial is not null. grid (column strips, row runs).
template <bool BF16, int ACT>
__device__ __forceinline__ void act_grad_rows(const uint16_t* dy, int64_t ldy,
                                              const uint16_t* z, int64_t rows, int64_t cols,
                                              int64_t run, uint16_t* dz, int64_t blocks,
                                              float* partial, float (*sums)[kSumLanes * 8 + 1]) {
  const int cl = threadIdx.x % kSumLanes, rl = threadIdx.x / kSumLanes;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * kSumLanes + cl) * 8;
  const int64_t r_end = min(rows, (static_cast<int64_t>(blockIdx.y) + 1) * run);
  float s[8] = {};
  if (c < (dz ? blocks * 64 : cols)) {
    for (int64_t r = blockIdx.y * run + rl; r < r_end; r += kSumRows) {
      float d[8];
      unpack8<BF16>(load_piece(dy + r * ldy, c, cols), d);
      if constexpr (ACT != kActNone) {
        float w[8];
        unpack8<BF16>(load_piece(z + r * cols, c, cols), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float a, g;
          act_both<ACT>(w[e], a, g);
          d[e] *= g;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += d[e];
      if (dz) *reinterpret_cast<u32x4*>(dz + blocked_at(r, c, blocks)) = pack8<BF16>(d);
    }
  }
  if (!partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[rl][cl * 8 + e] = s[e];
  __syncthreads();
  const int64_t cc = static_cast<int64_t>(blockIdx.x) * (kSumLanes * 8) + threadIdx.x;
  const int64_t cp = (cols + 7) & ~int64_t{7};
  if (cc < cp) {
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < kSumRows; ++r) t += sums[r][threadIdx.x];
    partial[blockIdx.y * cp + cc] = t;
  }
}
static_assert(kSumLanes * 8 == kSumThreads, "one thread per column of a strip");

template <bool BF16>
__global__ __launch_bounds__(kSumThreads) void k_act_grad(const uint16_t* dy, int64_t ldy,
                                                          const uint16_t* z, int act, int64_t rows, int64_t cols,
                                                          int64_t run, uint16_t* dz, int64_t blocks,
                                                          float* partial) {
  __shared__ float sums[kSumRows][kSumLanes * 8 + 1];
  with_act(act, [&](auto a) {
    act_grad_rows<BF16, decltype(a)::value>(dy, ldy, z, rows, cols, run, dz, blocks,
                                            partial, sums);
  });
}

// out[c] = sum of partial[0 .. parts)[c]: 16 columns a workgroup, thread (q, c)
// adds the parts q, q + 64, ... in order, then the 64 sums are added pairwise
struct Sums {
  SumJob job[kSums];
};
__global__ __launch_bounds__(1024) void k_sum_parts(Sums list) {
  const SumJob& a = list.job[blockIdx.y];
  const float* __restrict__ partial = a.partial;
  const int64_t parts = a.parts, ld = a.ld, cols = a.cols, groups = a.groups;
  __shared__ float sums[64][17];
  const int cl = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 16 + cl;
  float s = 0.0f;
  if (c < cols) {
    const int64_t gc = cols / groups, gp = ld / groups;
    const int64_t at = c / gc * gp + c % gc;
#pragma unroll 8
    for (int64_t p = q; p < parts; p += 64) s += partial[p * ld + at];
  }
  sums[q][cl] = s;
  __syncthreads();
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) {
    if (q < w) sums[q][cl] += sums[q + w][cl];
    __syncthreads();
  }
  if (q != 0 || c >= cols) return;
  if (c < a.split) a.out[c] = sums[0][cl];
  else a.out2[c - a.split] = sums[0][cl];
}

int act_grad(const Mat16& dy, const uint16_t* z, int act, bool bf16, uint16_t* dz, float* partial,
             hipStream_t stream) {
  const int64_t blocks = div_up(dy.cols, 64);
  const int64_t strips = div_up(dz ? blocks * 8 : div_up(dy.cols, 8), kSumLanes);
  const int64_t parts = column_parts(dy.rows, dy.cols);
  const int64_t run = div_up(div_up(dy.rows, parts), kSumRows) * kSumRows;
  const dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(parts));
  if (bf16)
    k_act_grad<true><<<grid, kSumThreads, 0, stream>>>(dy.p, dy.ld, z, act, dy.rows,
                                                       dy.cols, run, dz, blocks, partial);
  else
    k_act_grad<false><<<grid, kSumThreads, 0, stream>>>(dy.p, dy.ld, z, act, dy.rows,
                                                        dy.cols, run, dz, blocks, partial);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

// ---- weight gradient ----

// A wave's accumulators into a plane of fp32 partial sums [rows][cols], cols a
// multiple of 8.
template <typename T, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void store_partial(float* plane, int64_t rows, int64_t cols, int64_t m0,
                                              int64_t n0, const float4v (&acc)[T::FN][T::FM]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, s = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int64_t m = m0 + (wave / WN) * (BM / WM) + i * 16 + s;
    if (m >= rows) continue;
#pragma unroll
    for (int j = 0; j < T::FN; ++j) {
      const int64_t n = n0 + (wave % WN) * (BN / WN) + j * 16 + g * 4;
      if (n < cols) *reinterpret_cast<float4v*>(plane + m * cols + n) = acc[j][i];
    }
  }
}

// One BM x BN tile of x^T dz over one run of rows, as fp32 partial sums: the
// output is small and the sum long, so the rows are split over all units. All
// tiles of a run are neighbours on one XCD and share its rows there. Bound by
// memory at 209715 rows of 256 x 2048 (dz read once: 237 us, 4.4 TB/s, 930
// TFLOP/s).
template <bool BF16, bool X_TILED, bool Z_TILED, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * 64, tile_waves(BM, BN, STAGES)) void k_weight_grad(Operand X, Operand Z, int64_t rows,
                                                             int64_t run, uint32_t m_tiles,
                                                             uint32_t n_tiles,
                                                             float* __restrict__ partial) {
  using T = Tile<BF16, true, true, false, BM, BN, WM, WN, STAGES, X_TILED, Z_TILED>;
  __shared__ __attribute__((aligned(16))) char smem[T::LDS_BYTES];
  const TilePos t = tile_pos(gridDim.x / (m_tiles * n_tiles), m_tiles * n_tiles, blockIdx.x);
  const int64_t m0 = t.n / n_tiles * BM, n0 = t.n % n_tiles * BN;
  const int64_t kb = t.m * run, ke = min(rows, kb + run);
  float4v acc[T::FN][T::FM];
  T::run(X, Z, 0, m0, n0, kb, ke, smem, acc);
  store_partial<T, BM, BN, WM, WN>(partial + t.m * X.rows * Z.rows, X.rows, Z.rows, m0, n0, acc);
}

// One tile of an input gradient over one run of k, as fp32 partial sums: for a
// product of few tiles and many steps, whose time is the steps' latency.
template <bool BF16, bool A_TILED>
__global__ __launch_bounds__(512, 2) void k_product_part(Operand A, Operand B, int64_t K, int64_t run,
                                                         int64_t cols, uint32_t m_tiles,
                                                         uint32_t n_tiles, float* __restrict__ partial) {
  using T = Tile<BF16, false, false, false, 128, 128, 2, 4, 4, A_TILED>;
  __shared__ __attribute__((aligned(16))) char smem[T::LDS_BYTES];
  const TilePos t = tile_pos(gridDim.x / (m_tiles * n_tiles), m_tiles * n_tiles, blockIdx.x);
  const int64_t m0 = t.n / n_tiles * 128, n0 = t.n % n_tiles * 128;
  const int64_t kb = t.m * run, ke = min(K, kb + run);
  float4v acc[T::FN][T::FM];
  T::run(A, B, 0, m0, n0, kb, ke, smem, acc);
  store_partial<T, 128, 128, 2, 4>(partial + t.m * A.rows * cols, A.rows, cols, m0, n0, acc);
}

// out = the partial sums of the runs added in order, rounded once; columns of
// `groups` padded groups are closed up
struct Planes {
  PlaneJob job[kPlanes];
};
template <bool BF16>
__global__ __launch_bounds__(256) void k_weight_sum(Planes list) {
  const PlaneJob& a = list.job[blockIdx.y];
  const float* __restrict__ partial = a.partial;
  uint16_t* __restrict__ out = a.out;
  const int64_t runs = a.runs, plane = a.plane, ldp = a.ldp, rows = a.rows, cols = a.cols;
  const int64_t groups = a.groups;
  __shared__ float4v sums[4][64];
  const int cl = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + cl;  // float4 of a plane
  const bool in = i * 4 < plane;
  float4v s = {};
  if (in) {
    const int64_t per = (runs + 3) / 4, end = min(runs, (q + 1) * per);
#pragma unroll 4
    for (int64_t p = q * per; p < end; ++p)
      s += *reinterpret_cast<const float4v*>(partial + p * plane + i * 4);
  }
  sums[q][cl] = s;
  __syncthreads();
  if (q != 0 || !in) return;
  s = (sums[0][cl] + sums[1][cl]) + (sums[2][cl] + sums[3][cl]);
  const int64_t r = i * 4 / ldp, c = i * 4 - r * ldp;
  if (r >= rows) return;
  const int64_t gp = ldp / groups, gc = cols / groups;
  const int64_t grp = c / gp, cc = c - grp * gp;
  uint16_t* o = out + r * cols + grp * gc + cc;
  if (cc + 4 <= gc && (reinterpret_cast<uintptr_t>(o) & 7) == 0) {
    *reinterpret_cast<u32x2*>(o) = pack4<BF16>(s);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (cc + e < gc) o[e] = to_16<BF16>(s[e]);
  }
}

// A weight gradient's tile: 256 x 256 (one workgroup a compute unit), or 128 x
// 128 (two) where the weights are no larger than that, so that three quarters
// or more of the wide tile would be empty, or where the wide tiles of all runs
// of 256 rows would leave half of the units idle (a tile's 256 KiB of partial
// sums then take longer to write than its products: 300 rows of 256 x 2048 15 us).
int64_t grad_tile(int64_t rows, int64_t cin, int64_t cols) {
  if (cin <= 128 && cols <= 128) return 128;
  return div_up(cin, 256) * div_up(cols, 256) * div_up(rows, 256) < 128 ? 128 : 256;
}

// Runs of rows of a weight gradient: a workgroup for every place, runs of at
// least 256 rows and a multiple of 64.
int64_t grad_run(int64_t rows, int64_t cin, int64_t cols) {
  const int64_t tile = grad_tile(rows, cin, cols), places = tile == 256 ? 256 : 512;
  const int64_t tiles = div_up(cin, tile) * div_up(cols, tile);
  const int64_t runs = std::max<int64_t>(1, std::min(div_up(places, tiles), div_up(rows, 256)));
  return std::max<int64_t>(kStepK, div_up(div_up(rows, runs), kStepK) * kStepK);
}

// Runs of k of an input gradient (1: not split): at most a quarter of the
// units have a tile and a tile at least eight steps; runs of at least four.
int64_t split_k(int64_t M, int64_t K, int64_t N) {
  const int64_t tiles = div_up(M, 128) * div_up(N, 128), steps = div_up(K, kStepK);
  if (tiles == 0 || tiles > 64 || steps < 8) return 1;
  const int64_t runs = std::min(256 / tiles, steps / 4), per = div_up(steps, runs);
  return div_up(steps, per);
}

}  // namespace

bool pieces_fit(const Mat16& a) { return aligned16(a.p) && a.ld % 8 == 0 && a.cols % 8 == 0; }

int run_packs(const PackList& list, hipStream_t stream) {
  int64_t most = 0;
  Packs p{};
  for (int q = 0; q < list.count; ++q) {
    p.job[q] = list.job[q];
    most = std::max(most, list.job[q].rows * list.job[q].row_pieces);
  }
  if (most == 0) return SUBMCONV_OK;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(div_up(most, 256), 8192)),
                  static_cast<unsigned>(list.count));
  if (most < INT32_MAX / 2) k_pack16<uint32_t><<<grid, 256, 0, stream>>>(p);
  else k_pack16<int64_t><<<grid, 256, 0, stream>>>(p);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int run_sums(const SumList& list, hipStream_t stream) {
  int64_t most = 0;
  Sums sums{};
  for (int q = 0; q < list.count; ++q) {
    sums.job[q] = list.job[q];
    most = std::max(most, list.job[q].cols);
  }
  if (most == 0) return SUBMCONV_OK;
  const dim3 grid(static_cast<unsigned>(div_up(most, 16)), static_cast<unsigned>(list.count));
  k_sum_parts<<<grid, 1024, 0, stream>>>(sums);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int run_planes(const PlaneList& list, bool bf16, hipStream_t stream) {
  int64_t most = 0;
  Planes planes{};
  for (int q = 0; q < list.count; ++q) {
    planes.job[q] = list.job[q];
    most = std::max(most, list.job[q].plane);
  }
  if (most == 0) return SUBMCONV_OK;
  const dim3 grid(static_cast<unsigned>(div_up(most, 256)), static_cast<unsigned>(list.count));
  if (bf16) k_weight_sum<true><<<grid, 256, 0, stream>>>(planes);
  else k_weight_sum<false><<<grid, 256, 0, stream>>>(planes);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int64_t column_parts(int64_t rows, int64_t cols) {
  const int64_t strips = div_up(div_up(cols, 8), kSumLanes);
  return std::max<int64_t>(1, std::min(div_up(1024, strips), div_up(rows, 4 * kSumRows)));
}

int column_sums(const Mat16& a, bool bf16, float* partial, float* out, SumList* list,
                hipStream_t stream) {
  list->job[list->count++] = SumJob{partial, column_parts(a.rows, a.cols), round8(a.cols), a.cols, 1, out};
  return act_grad(a, nullptr, kActNone, bf16, nullptr, partial, stream);
}

int linear_forward(const Mat16& x, const Mat16& W, const float* bias, int act, bool bf16,
                   const uint16_t* residual, int64_t ldr, uint16_t* out, int64_t ldo, uint16_t* pre,
                   int64_t cols, hipStream_t stream) {
  const LinearEpi e{bias, residual, ldr, out, ldo, pre, act,
                    cols % 8 == 0 && ldr % 8 == 0 && aligned16(residual),
                    cols % 8 == 0 && ldo % 8 == 0 && aligned16(out),
                    cols % 8 == 0 && aligned16(pre)};
  return linear_product<true>(x, Operand{W.p, W.ld, W.cols, W.rows}, cols, bf16, e, stream);
}

int64_t product_nt_bytes(int64_t rows, int64_t k, int64_t cols) {
  const int64_t runs = split_k(rows, k, cols);
  return runs > 1 ? runs * rows * round8(cols) * 4 : 0;
}

int product_nt(const Mat16& dz, const Mat16& W, bool bf16, float* partial, uint16_t* out,
               int64_t cols, PlaneList* list, hipStream_t stream) {
  const int64_t runs = split_k(dz.rows, dz.cols, cols);
  if (runs > 1) {
    const int64_t mt = div_up(dz.rows, 128), nt = div_up(cols, 128), cp = round8(cols);
    const int64_t run = div_up(div_up(dz.cols, kStepK), runs) * kStepK;
    const Operand A{dz.p, dz.ld, dz.rows, dz.cols}, B{W.p, W.ld, W.rows, W.cols};
    const dim3 grid(static_cast<unsigned>(runs * mt * nt));
    auto go = [&](auto bf, auto blocked) {
      k_product_part<bf, blocked><<<grid, 512, 0, stream>>>(A, B, dz.cols, run, cp, mt, nt, partial);
    };
    if (bf16 && dz.blocked) go(std::true_type{}, std::true_type{});
    else if (bf16) go(std::true_type{}, std::false_type{});
    else if (dz.blocked) go(std::false_type{}, std::true_type{});
    else go(std::false_type{}, std::false_type{});
    SUBMCONV_HIP_CHECK(hipGetLastError());
    list->job[list->count++] = PlaneJob{partial, runs, dz.rows * cp, cp, dz.rows, cols, 1, out};
    return SUBMCONV_OK;
  }
  const LinearEpi e{nullptr, nullptr, 0, out, cols, nullptr, kActNone,
                    false, cols % 8 == 0 && aligned16(out), false};
  return linear_product<false>(dz, Operand{W.p, W.ld, W.rows, W.cols}, cols, bf16, e, stream);
}

int64_t product_tn_bytes(int64_t rows, int64_t cin, int64_t cols) {
  return std::max<int64_t>(1, div_up(rows, grad_run(rows, cin, cols))) * cin * cols * 4;
}

int product_tn(const Mat16& x, const Mat16& dz, bool bf16, float* partial, uint16_t* out,
               int64_t cols_x, int64_t cols_z, int groups, PlaneList* list, hipStream_t stream) {
  const int64_t run = grad_run(x.rows, x.cols, dz.cols);
  const int64_t runs = std::max<int64_t>(1, div_up(x.rows, run));
  const int64_t tile = grad_tile(x.rows, x.cols, dz.cols);
  const int64_t mt = div_up(x.cols, tile), nt = div_up(dz.cols, tile);
  if (runs * mt * nt > INT32_MAX || div_up(x.cols * dz.cols, 256) > INT32_MAX)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "weight gradient %lld x %lld",
                     (long long)x.cols, (long long)dz.cols);
  const Operand X{x.p, x.ld, x.cols, x.rows}, Z{dz.p, dz.ld, dz.cols, x.rows};
  const dim3 grid(static_cast<unsigned>(runs * mt * nt));
  auto launch = [&](auto xt, auto zt) {
    auto go = [&](auto t) {
      if (bf16)
        k_weight_grad<true, xt, zt, t, t, 2, 4, 3><<<grid, 512, 0, stream>>>(X, Z, x.rows, run, mt, nt, partial);
      else
        k_weight_grad<false, xt, zt, t, t, 2, 4, 3><<<grid, 512, 0, stream>>>(X, Z, x.rows, run, mt, nt, partial);
    };
    if (tile == 256) go(std::integral_constant<int, 256>{});
    else go(std::integral_constant<int, 128>{});
  };
  if (x.blocked) launch(std::true_type{}, std::false_type{});
  else if (dz.blocked) launch(std::false_type{}, std::true_type{});
  else launch(std::false_type{}, std::false_type{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  list->job[list->count++] = PlaneJob{partial, runs, x.cols * dz.cols, dz.cols, cols_x, cols_z, groups, out};
  return SUBMCONV_OK;
}

Mat16 readable(const Mat16& a, int groups, int unit, Arena& ws, PackList* list) {
  if (pieces_fit(a) && a.cols % (unit * groups) == 0) return a;
  const int64_t from = a.cols / groups, to = round_to(from, unit);
  uint16_t* p = static_cast<uint16_t*>(ws.take(a.rows * groups * to * 2));
  list->job[list->count++] = PackJob{a.p, a.rows, a.ld, from, to, groups * to / 8, p};
  return Mat16{p, a.rows, groups * to, groups * to};
}

int check_shape(const char* name, int64_t rows, int64_t cols) {
  if (cols < 1 || cols > (int64_t{1} << 20))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%s has %lld columns", name, (long long)cols);
  if (rows < 0)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s has %lld rows", name, (long long)rows);
  return SUBMCONV_OK;
}

int check_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  SUBMCONV_TRY(check_shape(name, rows, cols));
  if (rows > 0 && !p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (rows > 1 && ld < cols)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: row stride %lld below %lld columns", name,
                     (long long)ld, (long long)cols);
  if (rows > 1 && ld > kMaxLd)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%s: row stride %lld above %lld", name,
                     (long long)ld, (long long)kMaxLd);
  if (reinterpret_cast<uintptr_t>(p) & 1)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  return SUBMCONV_OK;
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need > 0 && (!ws || have < need))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "workspace of %lld bytes, %lld are needed",
                     (long long)(ws ? have : 0), (long long)need);
  if (!aligned16(ws)) return set_error(SUBMCONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return SUBMCONV_OK;
}

int check_kind(int32_t act, int32_t dtype) {
  if (act < kActNone || act > kActGeluTanh)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "act = %d", act);
  if (dtype != SUBMCONV_DTYPE_F16 && dtype != SUBMCONV_DTYPE_BF16)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "dtype = %d", dtype);
  return SUBMCONV_OK;
}

Mat16 shape_of(int64_t rows, int64_t cols, bool aligned) {
  return Mat16{reinterpret_cast<const uint16_t*>(aligned ? 16 : 2), rows, cols, aligned ? round8(cols) : cols};
}

namespace {

struct LinearGradNeeds {
  bool x, w, b;
};
// The gradients' steps, or with an arena that counts, their workspace.
int linear_grad(const Mat16& dy, const Mat16& x, const Mat16& W, const uint16_t* pre, int act,
                bool bf16, uint16_t* gx, uint16_t* gw, float* gb, LinearGradNeeds need, Arena& ws,
                hipStream_t stream) {
  const bool run = !ws.counting;
  const int64_t cp = round8(dy.cols);
  const bool own_dz = (act != kActNone || !pieces_fit(dy)) && (need.x || need.w);
  PackList packs;
  Mat16 dz = dy, Wr, xr;
  uint16_t* dz_to = nullptr;
  if (own_dz) {
    const int64_t cq = round64(dy.cols);
    dz_to = static_cast<uint16_t*>(ws.take(blocked_bytes(dy.rows, cq)));
    dz = blocked16(dz_to, dy.rows, cq);
  }
  if (need.x) Wr = readable(W, 1, own_dz ? 64 : 8, ws, &packs);
  if (need.w) xr = readable(x, 1, 8, ws, &packs);
  const int64_t parts = column_parts(dy.rows, dy.cols);
  float* sums = need.b ? static_cast<float*>(ws.take(parts * cp * 4)) : nullptr;
  float* part_x = need.x ? static_cast<float*>(ws.take(product_nt_bytes(dz.rows, dz.cols, x.cols))) : nullptr;
  float* part_w = need.w ? static_cast<float*>(ws.take(product_tn_bytes(x.rows, round8(x.cols), dz.cols))) : nullptr;
  if (!run) return SUBMCONV_OK;
  PlaneList planes;
  SumList columns;
  SUBMCONV_TRY(run_packs(packs, stream));
  if (own_dz || need.b) SUBMCONV_TRY(act_grad(dy, pre, act, bf16, dz_to, sums, stream));
  if (need.x) SUBMCONV_TRY(product_nt(dz, Wr, bf16, part_x, gx, x.cols, &planes, stream));
  if (need.w) SUBMCONV_TRY(product_tn(xr, dz, bf16, part_w, gw, x.cols, dy.cols, 1, &planes, stream));
  SUBMCONV_TRY(run_planes(planes, bf16, stream));
  if (need.b) columns.job[columns.count++] = SumJob{sums, parts, cp, dy.cols, 1, gb};
  return run_sums(columns, stream);
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int64_t submconv_linear_workspace_bytes(int64_t n, int32_t cin, int32_t cout,
                                                   int32_t aligned) {
  clear_error();
  SUBMCONV_TRY(check_shape("x", n, cin));
  SUBMCONV_TRY(check_shape("W", cin, cout));
  Arena ws;
  PackList packs;
  if (n > kFewRows) {
    readable(shape_of(n, cin, aligned), 1, 8, ws, &packs);
    readable(shape_of(cin, cout, aligned), 1, 8, ws, &packs);
  }
  return ws.used;
}

extern "C" int submconv_linear(const uint16_t* x, int64_t ldx, int64_t n, const uint16_t* W,
                               const float* bias, const uint16_t* residual, int64_t ldr,
                               uint16_t* out, uint16_t* pre, int32_t cin, int32_t cout, int32_t act,
                               int32_t dtype, void* workspace, int64_t workspace_bytes,
                               hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_kind(act, dtype));
  SUBMCONV_TRY(check_matrix("x", x, n, cin, ldx));
  SUBMCONV_TRY(check_matrix("W", W, cin, cout, cout));
  SUBMCONV_TRY(check_matrix("out", out, n, cout, cout));
  if (residual) SUBMCONV_TRY(check_matrix("residual", residual, n, cout, ldr));
  if (pre) SUBMCONV_TRY(check_matrix("pre", pre, n, cout, cout));
  if (n == 0) return SUBMCONV_OK;
  const Mat16 xm{x, n, cin, ldx}, wm{W, cin, cout, cout};
  const bool bf16 = dtype == SUBMCONV_DTYPE_BF16;
  if (n <= kFewRows) return few_linear(xm, wm, bias, act, bf16, residual, ldr, out, pre, stream);
  Arena ws{false, static_cast<char*>(workspace)};
  PackList packs;
  const Mat16 xr = readable(xm, 1, 8, ws, &packs), wr = readable(wm, 1, 8, ws, &packs);
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, ws.used));
  SUBMCONV_TRY(run_packs(packs, stream));
  return linear_forward(xr, wr, bias, act, bf16, residual, ldr, out, cout, pre, cout, stream);
}

extern "C" int64_t submconv_linear_backward_workspace_bytes(int64_t n, int32_t cin, int32_t cout,
                                                            int32_t act, int32_t aligned) {
  clear_error();
  SUBMCONV_TRY(check_kind(act, SUBMCONV_DTYPE_F16));
  SUBMCONV_TRY(check_shape("x", n, cin));
  SUBMCONV_TRY(check_shape("W", cin, cout));
  Arena ws;
  SUBMCONV_TRY(linear_grad(shape_of(n, cout, aligned), shape_of(n, cin, aligned),
                           shape_of(cin, cout, aligned), nullptr, act, false, nullptr, nullptr,
                           nullptr, {true, true, true}, ws, nullptr));
  return ws.used;
}

extern "C" int submconv_linear_backward(const uint16_t* grad_out, int64_t ldg, int64_t n,
                                        const uint16_t* x, int64_t ldx, const uint16_t* W,
                                        const uint16_t* pre, uint16_t* grad_x, uint16_t* grad_w,
                                        float* grad_b, int32_t cin, int32_t cout, int32_t act,
                                        int32_t dtype, void* workspace, int64_t workspace_bytes,
                                        hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_kind(act, dtype));
  SUBMCONV_TRY(check_matrix("grad_out", grad_out, n, cout, ldg));
  if (grad_w) SUBMCONV_TRY(check_matrix("x", x, n, cin, ldx));
  SUBMCONV_TRY(check_matrix("W", W, cin, cout, cout));
  if (act != kActNone) SUBMCONV_TRY(check_matrix("pre", pre, n, cout, cout));
  const Mat16 dy{grad_out, n, cout, n == 1 ? round8(cout) : ldg};
  const Mat16 xm{x, n, cin, n == 1 ? round8(cin) : ldx}, wm{W, cin, cout, cout};
  const LinearGradNeeds need{grad_x != nullptr, grad_w != nullptr, grad_b != nullptr};
  Arena count;
  const bool bf16 = dtype == SUBMCONV_DTYPE_BF16;
  SUBMCONV_TRY(linear_grad(dy, xm, wm, pre, act, bf16, grad_x, grad_w, grad_b, need, count, stream));
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, count.used));
  Arena ws{false, static_cast<char*>(workspace)};
  return linear_grad(dy, xm, wm, pre, act, bf16, grad_x, grad_w, grad_b, need, ws, stream);
}
