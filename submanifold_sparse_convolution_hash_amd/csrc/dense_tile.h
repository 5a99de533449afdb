// Tiled 16-bit matrix products on MFMA for the dense layers (linear, gated
// feed-forward): out[m][n] = sum_k A(m, k) B(k, n), fp32 accumulation.
//
// A workgroup of WM x WN waves owns a BM x BN tile of the output and walks k
// in steps of 64. Each step's two operand tiles go straight from memory into
// LDS (buffer_load ... lds, 16 bytes a lane): STAGES buffers in turn for A,
// which comes from HBM, two for B, which stays in the caches; the loads of the
// coming steps are in flight while the waves multiply the current one. Buffer
// bounds give zeros past the last row and the last k.
// An operand is read either with k contiguous in memory (x, and a weight
// matrix under its transpose) by ds_read_b128, or with k as the row index (a
// weight matrix as it is stored, both operands of a weight gradient) by
// ds_read_b64_tr_b16, which transposes 4 x 16 pieces on the way out of LDS:
// no operand is ever transposed in memory.
//
// v_mfma_f32_16x16x32 takes n as its row index and m as its column index, so
// that a lane ends with 4 consecutive n of one m. The epilogue passes the fp32
// accumulators through LDS once, so that each thread then holds 8 consecutive
// columns of a row and neighbouring threads the row's next ones: bias,
// activation, residual and every load and store work on whole memory lines.
#pragma once

#include <type_traits>

#include "submconv_internal.h"

namespace submconv {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kStepK = 64;                  // k per LDS buffer
constexpr uint32_t kOobOff = 0x80000000u;   // past every buffer's bound
constexpr int64_t kMaxLd = int64_t{1} << 22;  // row strides: a tile's byte offsets fit 31 bits

__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}

// ---- 16-bit elements ----

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (BF16) return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
  else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}
template <bool BF16>
__device__ __forceinline__ uint16_t to_16(float v) {  // round to nearest even
  if constexpr (BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}
template <bool BF16>
__device__ __forceinline__ u32x2 pack4(float4v v) {
  if constexpr (BF16) {
    bf16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = static_cast<__bf16>(v[e]);
    return __builtin_bit_cast(u32x2, h);
  } else {
    half4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = static_cast<_Float16>(v[e]);
    return __builtin_bit_cast(u32x2, h);
  }
}
template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  const u32x2 a = pack4<BF16>(float4v{v[0], v[1], v[2], v[3]});
  const u32x2 b = pack4<BF16>(float4v{v[4], v[5], v[6], v[7]});
  return u32x4{a[0], a[1], b[0], b[1]};
}
template <bool BF16>
__device__ __forceinline__ void unpack8(u32x4 p, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32<BF16>(static_cast<uint16_t>(p[e >> 1] >> (16 * (e & 1))));
}

template <bool BF16>
__device__ __forceinline__ float4v mfma16(half8 a, half8 b, float4v c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// ---- 8 columns of a 16-bit matrix row ----

// Row `row`'s columns n .. n + 7, zeros past n_end (16 bytes at any element's
// address: the memory system takes an access that is not aligned to its size).
__device__ __forceinline__ u32x4 load_piece(const uint16_t* row, int64_t n, int64_t n_end) {
  typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
  if (n + 8 <= n_end) return *reinterpret_cast<const loose*>(row + n);
  u32x4 r = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < n_end) r[e >> 1] |= static_cast<uint32_t>(row[n + e]) << (16 * (e & 1));
  return r;
}

// The rows m0 .. of a 16-bit matrix that an epilogue reads or writes, through
// a buffer whose bound ends with the matrix: lanes outside it load zeros and
// store nothing, without a branch. Stores are marked as not to be kept in the
// caches (kStream): 209715 x 128 -> 512 with pre-activations writes 430 MB and
// takes 95 us with the mark, at the rate of a copy, and 128 to 146 us without.
// A product alone is never slower with it (128 -> 512, 40000 rows 19.0 against 20.5
// us, 1000 rows 6.0 against 6.1). A product and the next one that reads its result
// (128 -> 512 -> 128), with / without: 15.1 / 15.1 us at 1000 rows, 23.0 / 23.5 at
// 20000, 70 / 68 at 80000 and 122 / 118 at 160000, whose 82 and 164 MB the 256 MB
// cache would have held, 233 / 279 at 320000.
constexpr int kStream = 2;  // the instructions' nt bit
struct RowsView {
  __amdgpu_buffer_rsrc_t r;
  const uint16_t* p;
  int64_t ld;
  uint32_t ld2, n_end, rows;
  bool vec;
  __device__ __forceinline__ RowsView(const uint16_t* q, int64_t ld_, int64_t m0, int64_t M,
                                      int64_t N, int tile_rows, bool vec_)
      : p(q ? q + m0 * ld_ : nullptr), ld(ld_), ld2(static_cast<uint32_t>(ld_) * 2u),
        n_end(static_cast<uint32_t>(N)), vec(vec_) {
    const int64_t left = M - m0 < tile_rows ? M - m0 : tile_rows;
    rows = q && left > 0 ? static_cast<uint32_t>(left) : 0u;
    r = tile_rsrc(p, rows ? static_cast<uint32_t>((left - 1) * ld_ + N) * 2u : 0u);
  }
  __device__ __forceinline__ u32x4 load(uint32_t m, uint32_t n) const {
    if (vec)
      return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                           r, n < n_end ? m * ld2 + n * 2u : kOobOff, 0, 0));
    u32x4 v = {};
    if (m < rows) v = load_piece(p + m * ld, n, n_end);
    return v;
  }
  __device__ __forceinline__ void store(uint32_t m, uint32_t n, u32x4 v) const {
    if (vec) {
      __builtin_amdgcn_raw_buffer_store_b128(v, r, n < n_end ? m * ld2 + n * 2u : kOobOff, 0, kStream);
      return;
    }
    if (m >= rows) return;
    typedef uint32_t loose __attribute__((ext_vector_type(4), aligned(2)));
    uint16_t* row = const_cast<uint16_t*>(p) + m * ld;
    if (n + 8 <= n_end) {
      *reinterpret_cast<loose*>(row + n) = v;
      return;
    }
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e)
      if (n + e < n_end) row[n + e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
  }
};

// Eight consecutive values of an fp32 vector, zeros past its end (all of them
// for a null vector, whose buffer holds nothing).
__device__ __forceinline__ void load_bias8(const float* p, int64_t n_end, uint32_t n, float (&v)[8]) {
  const __amdgpu_buffer_rsrc_t r = tile_rsrc(p, p ? static_cast<uint32_t>(n_end) * 4u : 0u);
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e)
    v[e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (n + e) * 4u, 0, 0));
}

// ---- activations ----

enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f;  // 2 sqrt(2 / pi)

__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}
// gelu_tanh = z / 2 (1 + tanh t) = z logistic(2 t): no cancellation for z < 0
__device__ __forceinline__ float tanh_arg(float z) {
  return kTwoSqrt2OverPi * (z + 0.044715f * z * z * z);
}
// gelu = z Phi(z). Phi(-a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) s P(s), s = 1 /
// (1 + 0.305 a), a >= 0: P is a least-squares polynomial, reweighted towards its
// largest relative error, 1.1e-7 for a up to 15; with the roundings Phi is within
// 2^-22 for z > 0 and, relative to itself, 1.3e-6 down to z = -6 and 4.1e-6 down to
// -13 (the exponent's own rounding). 1 + erf loses all digits by z = -5.5, which
// bf16 results show. `e`: exp(-z^2 / 2), which the slope needs as well. 209715 x
// 128 -> 512 with pre-activations takes 118 us (with the library's erff 137, erfcf 172).
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float s = __builtin_amdgcn_rcpf(1.0f + 0.305f * fabsf(z));
  float p = 0.0364274792f;
  p = p * s - 0.151897117f;
  p = p * s + 0.183906615f;
  p = p * s - 0.036374446f;
  p = p * s + 0.120207421f;
  p = p * s + 0.103657544f;
  p = p * s + 0.122430496f;
  p = p * s + 0.121642001f;
  const float q = p * s * e;
  return z < 0.0f ? q : 1.0f - q;
}
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  else if constexpr (ACT == kActSilu) return z * logistic(z);
  else if constexpr (ACT == kActGelu) return z * normal_cdf(z, __expf(-0.5f * z * z));
  else if constexpr (ACT == kActGeluTanh) return z * logistic(tanh_arg(z));
  else return z;
}
// value and derivative
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& a, float& d) {
  if constexpr (ACT == kActRelu) {
    a = z < 0.0f ? 0.0f : z;
    d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActSilu) {
    const float p = logistic(z);
    a = z * p;
    d = p + a * (1.0f - p);
  } else if constexpr (ACT == kActGelu) {
    const float e = __expf(-0.5f * z * z), c = normal_cdf(z, e);
    a = z * c;
    d = c + z * kInvSqrt2Pi * e;
  } else if constexpr (ACT == kActGeluTanh) {
    const float p = logistic(tanh_arg(z));
    a = z * p;
    // (p is 0 or 1 long before z^2 reaches the bound, and z^2 infinite would make 0 inf of it)
    d = p + a * (1.0f - p) * kTwoSqrt2OverPi * (1.0f + 0.134145f * fminf(z * z, 1e30f));
  } else {
    a = z;
    d = 1.0f;
  }
}
// runs f<ACT>() for a uniform run-time activation
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

// ---- matrices between two kernels ----
//
// h, dg, du and dz live in the workspace only, between the kernel that forms
// them and the products that read them, so they are laid out for those: blocks
// of kBlockRows x 64 elements, each 16 KiB in one piece, a row of blocks after
// the other. A product's tile of k = 64 is then contiguous memory, whichever
// way it runs, instead of 128-byte pieces a row stride apart.
constexpr int kBlockRows = 128;

// Elements before element (row, col) of a blocked matrix with `blocks` = its
// columns / 64.
__host__ __device__ inline int64_t blocked_at(int64_t row, int64_t col, int64_t blocks) {
  return ((row / kBlockRows * blocks + col / 64) * kBlockRows + row % kBlockRows) * 64 + col % 64;
}
// Rows of a tile of at most `most` that start at row m0 of M: none where m0 is
// past the end (a later phase of a last tile). RowsView counts by itself: through
// this its stores compiled to slower code (209715 x 128 -> 512 with
// pre-activations 95 -> 97, gated 128 / 512 255 -> 279 us).
__host__ __device__ constexpr uint32_t rows_left(int64_t M, int64_t m0, int most) {
  const int64_t left = M - m0;
  return left <= 0 ? 0u : static_cast<uint32_t>(left < most ? left : most);
}
static_assert(rows_left(300, 256, 128) == 44 && rows_left(300, 128, 128) == 128, "rows of a tile");
static_assert(rows_left(256, 256, 128) == 0 && rows_left(300, 384, 128) == 0, "no rows");

// Stores 8 columns at tile row `m`, column n < n_end (a multiple of 64) of the
// block row that starts at tile row 0.
struct BlockView {
  uint16_t* p;
  uint32_t rows, n_end;
  __device__ __forceinline__ BlockView(uint16_t* q, int64_t m0, int64_t M, int64_t N)
      : p(q + m0 / kBlockRows * kBlockRows * N + m0 % kBlockRows * 64),
        rows(rows_left(M, m0, kBlockRows)),
        n_end(static_cast<uint32_t>(N)) {}
  __device__ __forceinline__ void store(uint32_t m, uint32_t n, u32x4 v) const {
    if (m < rows && n < n_end)
      *reinterpret_cast<u32x4*>(p + static_cast<size_t>(n / 64) * (kBlockRows * 64) + m * 64 + n % 64) = v;
  }
};

// ---- operand tiles ----

typedef uint32_t rsrc4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ rsrc4 load_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return rsrc4{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// 16 bytes a lane from r + voff to LDS byte `lds` + 16 lane. Written as
// assembly, without an output register, because for the builtin the compiler
// waits for every such load before the next LDS read, of whatever buffer;
// Tile::run waits for them by count instead. m0 is a reserved register, which
// takes no clobber: nothing else in these kernels uses it.
__device__ __forceinline__ void load_to_lds(rsrc4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(voff), "s"(r));
}
// The wait states between a vector instruction that writes a scalar register
// and a load that reads it, which the compiler does not place before assembly.
__device__ __forceinline__ void settle_rsrc(rsrc4& r) { asm volatile("s_nop 4" : "+s"(r)); }
__device__ __forceinline__ uint32_t lds_addr(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)p));
}

// One operand: R rows of the tile (m or n) by k. `ld`: elements between
// memory rows. All of p, ld, `rows` of a KRow operand and k of a KCol
// one are multiples of 8 elements, so a 16-byte piece is inside or outside.
struct Operand {
  const uint16_t* p;
  int64_t ld;    // columns, for a blocked matrix
  int64_t rows;  // m or n extent
  int64_t k;     // k extent; a product's k is the k-contiguous operand's, whose
                 // zeros may go up to 7 past the memory rows of a KRow one
};

// The k-contiguous form. LDS: row r is 128 bytes, its piece c (8 k) in slot c
// ^ ((r / 2) % 8), so that the 16 rows a read pass takes fall on distinct
// banks.
// TILED: a blocked matrix.
template <int R, int NT, bool TILED>
struct LoadKCol {
  static constexpr int SL = R * 8 / NT;
  static_assert(R * 8 % NT == 0 && NT / 8 % 16 == 0, "slots");
  const uint16_t* base;
  uint32_t bytes;
  uint32_t voff[SL];
  int kc;
  __device__ __forceinline__ void init(const Operand& o, int64_t row0, int64_t k_end, int tid) {
    const int64_t left = o.rows - row0;
    const int r0 = tid >> 3;
    kc = ((tid & 7) ^ ((r0 >> 1) & 7)) * 8;
    if constexpr (TILED) {
      // R / kBlockRows blocks of 16 KiB, a row of blocks apart
      static_assert(R % kBlockRows == 0, "whole blocks");
      base = o.p + row0 * o.ld;
      bytes = static_cast<uint32_t>((R / kBlockRows - 1) * kBlockRows * o.ld + kBlockRows * 64) * 2u;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        const int r = r0 + i * (NT / 8);
        voff[i] = r < left ? static_cast<uint32_t>(r / kBlockRows * kBlockRows * o.ld + r % kBlockRows * 64 + kc) * 2u
                           : kOobOff;
      }
    } else {
      base = o.p + row0 * o.ld;
      bytes = left > 0 ? static_cast<uint32_t>(((left < R ? left : R) - 1) * o.ld + k_end) * 2u : 0u;
#pragma unroll
      for (int i = 0; i < SL; ++i)
        voff[i] = static_cast<uint32_t>((r0 + i * (NT / 8)) * o.ld + kc) * 2u;
    }
  }
  __device__ __forceinline__ void issue(uint32_t lds, int64_t k0, int64_t k_end, int wave) const {
    rsrc4 r = load_rsrc(TILED ? base + k0 * kBlockRows : base, bytes);
    settle_rsrc(r);
    const bool in = TILED || k0 + kc < k_end;  // a blocked matrix has whole steps
    const uint32_t step = TILED ? 0u : static_cast<uint32_t>(k0) * 2u;
#pragma unroll
    for (int i = 0; i < SL; ++i)
      load_to_lds(r, in ? voff[i] + step : kOobOff, lds + (i * NT + wave * 64) * 16);
  }
};

// The form with k as the memory row. LDS: k row r is 2 R bytes; its 32-byte
// pair of pieces p sits at p ^ f(r), f(r) = r % 4 + 4 (r / 8 % 2), so that the
// 8 k rows that a transposed read takes at a time fall on distinct banks. At
// R = 64 two rows share the banks' width and f(r) = r / 2 % 2 + 2 (r / 8 % 2).
template <int CH>
__device__ __forceinline__ int krow_swizzle(int k) {
  if constexpr (CH == 8) return ((k >> 1 & 1) | ((k >> 3 & 1) << 1)) << 1;
  else return ((k & 3) | ((k >> 3 & 1) << 2)) << 1;
}
// PAIR: the tile's columns are R / 2 of the first half of the matrix (gate)
// and the R / 2 at the same place of its second half (up, `half` further on).
// TILED: a blocked matrix, whose rows past the last are not to be read.
template <int R, int NT, bool PAIR, bool TILED>
struct LoadKRow {
  static constexpr int CH = R / 8;  // pieces per k row
  static constexpr int SL = kStepK * CH / NT;
  static constexpr int KS = NT / CH;  // k rows between a thread's slots
  static_assert(kStepK * CH % NT == 0, "slots");
  const uint16_t* p;
  int64_t ld, width, k_rows;
  uint32_t voff[SL];
  int k_thread;
  int64_t pair_col;
  static __device__ __forceinline__ int swz(int k) { return krow_swizzle<CH>(k); }
  __device__ __forceinline__ void init(const Operand& o, int64_t col0, int64_t half, int tid) {
    p = o.p;
    ld = o.ld;
    k_rows = o.k;
    width = PAIR ? half + o.rows : o.rows;
    const int k0 = tid / CH, cs = tid % CH;
    k_thread = k0;
    if constexpr (TILED) p = o.p + col0 * kBlockRows;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int k = k0 + i * KS;
      const int c = (cs ^ swz(k)) * 8;
      if constexpr (TILED) {
        voff[i] = col0 + c < o.rows
                      ? static_cast<uint32_t>((c / 64 * kBlockRows + k) * 64 + c % 64) * 2u : kOobOff;
        continue;
      }
      int64_t col;
      bool in;
      if constexpr (PAIR) {
        const bool up = c >= R / 2;
        const int64_t cc = col0 + (up ? c - R / 2 : c);
        in = cc < o.rows;
        col = up ? cc + half : cc;
      } else {
        col = col0 + c;
        in = col < o.rows;
      }
      voff[i] = in ? static_cast<uint32_t>(k * ld + col) * 2u : kOobOff;
    }
    if constexpr (PAIR) {
      const int c = (cs ^ swz(k0)) * 8;
      pair_col = col0 + (c >= R / 2 ? c - R / 2 : c);
    }
  }
  // PAIR: the tile `step` columns further on. (A thread's slots share their
  // column: swz repeats every 16 k rows, which KS is a multiple of.)
  __device__ __forceinline__ void next(int step, int64_t cols) {
    static_assert(!PAIR || KS % 16 == 0, "one column per thread");
    pair_col += step;
#pragma unroll
    for (int i = 0; i < SL; ++i) voff[i] = pair_col < cols ? voff[i] + step * 2u : kOobOff;
  }
  __device__ __forceinline__ void issue(uint32_t lds, int64_t k0, int64_t k_end, int wave) const {
    const int64_t left = (k_rows < k_end ? k_rows : k_end) - k0;
    if constexpr (TILED) {
      // k0 starts one of a block's halves; the tile spans R / 64 blocks
      rsrc4 r = load_rsrc(p + k0 / kBlockRows * kBlockRows * ld + k0 % kBlockRows * 64,
                          R / 64 * kBlockRows * 128u);
      settle_rsrc(r);
#pragma unroll
      for (int i = 0; i < SL; ++i)
        load_to_lds(r, k_thread + i * KS < left ? voff[i] : kOobOff, lds + (i * NT + wave * 64) * 16);
    } else {
      const uint32_t bytes =
          left > 0 ? static_cast<uint32_t>(((left < kStepK ? left : kStepK) - 1) * ld + width) * 2u : 0u;
      rsrc4 r = load_rsrc(p + k0 * ld, bytes);
      settle_rsrc(r);
#pragma unroll
      for (int i = 0; i < SL; ++i) load_to_lds(r, voff[i], lds + (i * NT + wave * 64) * 16);
    }
  }
};

// Waits until at most N of this wave's loads to LDS are in flight, and for its
// LDS reads.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// ---- accumulators as rows ----

// ROWS rows of BN fp32 columns in LDS, 8 columns of a row per thread and turn.
// The 16-byte piece p of row r sits at p ^ (r % 16) ^ (p / 16 % 2), which keeps
// the 16 rows of an accumulator's write and the 16 pieces of a read apart.
template <int ROWS, int BN, int NT>
struct LdsRows {
  static constexpr int PH_ROWS = ROWS;
  static constexpr int PIECES = BN / 8;          // 8-column pieces per row
  static constexpr int ROW_STEP = NT / PIECES;   // rows between a thread's pieces
  static constexpr int ROW_PASSES = ROWS / ROW_STEP;
  static __device__ __forceinline__ int row_byte(int r, int p) {
    return r * (BN * 4) + ((p ^ (r & 15) ^ (p >> 4 & 1)) << 4);
  }
  static __device__ __forceinline__ void read8(const char* smem, int r, int piece, float (&v)[8]) {
    const float4v a = *reinterpret_cast<const float4v*>(smem + row_byte(r, 2 * piece));
    const float4v b = *reinterpret_cast<const float4v*>(smem + row_byte(r, 2 * piece + 1));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  }
};

// ---- the tile ----

// A_ROW, B_ROW: k is the memory row of that operand; A_TILED, B_TILED: it is
// blocked (k as the row for B). PAIR: see LoadKRow
// (B only); accumulator columns j < FN / 2 are then gate columns, the others
// the up columns at the same place.
template <bool BF16, bool A_ROW, bool B_ROW, bool PAIR, int BM, int BN, int WM, int WN, int STAGES,
          bool A_TILED = false, bool B_TILED = false>
struct Tile {
  static constexpr bool DEEP = STAGES > 3;  // as many buffers for B as for A
  static constexpr int NT = WM * WN * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
  static constexpr int A_BYTES = BM * kStepK * 2, B_BYTES = BN * kStepK * 2;
  static constexpr int B_STAGES = DEEP ? STAGES : 2;
  static constexpr int LDS_BYTES = STAGES * A_BYTES + B_STAGES * B_BYTES;
  static_assert(FM >= 1 && FN >= 1 && (!PAIR || FN % 2 == 0), "wave tile");
  static_assert(STAGES >= 2 && STAGES <= 4, "buffers");
  using LA = std::conditional_t<A_ROW, LoadKRow<BM, NT, false, A_TILED>, LoadKCol<BM, NT, A_TILED>>;
  using LB = std::conditional_t<B_ROW, LoadKRow<BN, NT, PAIR, B_TILED>, LoadKCol<BN, NT, false>>;

  // first column (in the tile) of accumulator column j of wave column wn
  static __device__ __forceinline__ int ncol(int wn, int j) {
    if constexpr (PAIR)
      return j < FN / 2 ? wn * (BN / WN / 2) + j * 16
                        : BN / 2 + wn * (BN / WN / 2) + (j - FN / 2) * 16;
    else
      return wn * (BN / WN) + j * 16;
  }

  template <int R, bool ROW>
  static __device__ __forceinline__ half8 frag(const char* t, int row, int kk, int lane) {
    const int g = lane >> 4, s = lane & 15;
    if constexpr (!ROW) {
      return *reinterpret_cast<const half8*>(
          t + (row + s) * 128 + (((kk * 4 + g) ^ (s >> 1)) << 4));
    } else {
      // lane s of group g names k row 32 kk + 8 g + 4 half + s / 4, columns 4
      // (s % 4) .. + 3 of the block; it receives column s of the 4 k rows
      constexpr int CH = R / 8;
      const int c = ((row >> 3) + ((s & 3) >> 1)) ^ krow_swizzle<CH>(g * 8 + (s >> 2));
      const char* q = t + (kk * 32 + g * 8 + (s >> 2)) * (R * 2) + c * 16 + (s & 1) * 8;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)q);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(q + 4 * R * 2));
      return __builtin_bit_cast(half8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }

  // acc[j][i]: n block j, m block i of the wave; k from k_begin (a multiple
  // of 64) to k_end.
  static __device__ __forceinline__ void run(const Operand& A, const Operand& B, int64_t half,
                                             int64_t m0, int64_t n0, int64_t k_begin, int64_t k_end,
                                             char* smem, float4v (&acc)[FN][FM]) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    LA la;
    LB lb;
    if constexpr (A_ROW) la.init(A, m0, 0, tid);
    else la.init(A, m0, k_end, tid);
    if constexpr (B_ROW) lb.init(B, n0, half, tid);
    else lb.init(B, n0, k_end, tid);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[j][i] = float4v{};

    const int steps = static_cast<int>((k_end - k_begin + kStepK - 1) / kStepK);
    const uint32_t lds = lds_addr(smem);
    auto k_of = [&](int st) { return k_begin + static_cast<int64_t>(st) * kStepK; };
    auto issue_a = [&](int st, int buf) { la.issue(lds + buf * A_BYTES, k_of(st), k_end, wave); };
    auto issue_b = [&](int st, int buf) {
      lb.issue(lds + STAGES * A_BYTES + buf * B_BYTES, k_of(st), k_end, wave);
    };
#pragma unroll
    for (int st = 0; st < STAGES - 1; ++st)
      if (st < steps) {
        issue_a(st, st);
        if (st < B_STAGES - 1) issue_b(st, st);
      }

    int buf = 0;
    for (int st = 0; st < steps; ++st) {
      // this step's loads are the oldest: all but those of the later steps
      // (A's only, unless DEEP) are waited for (and this wave's LDS reads of
      // the last step), then every wave's through the barrier, after which the
      // buffers that were read in the last step are overwritten
      if constexpr (DEEP) {
        static_assert(STAGES == 4, "waits");
        if (st + 2 < steps) wait_loads<2 * (LA::SL + LB::SL)>();
        else if (st + 1 < steps) wait_loads<LA::SL + LB::SL>();
        else wait_loads<0>();
      } else if (STAGES == 3 && st + 1 < steps) {
        wait_loads<LA::SL>();
      } else {
        wait_loads<0>();
      }
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      const int last = buf == 0 ? STAGES - 1 : buf - 1;
      if (DEEP ? st + STAGES - 1 < steps : st + 1 < steps)
        issue_b(DEEP ? st + STAGES - 1 : st + 1, DEEP ? last : (st + 1) & 1);
      if (st + STAGES - 1 < steps) issue_a(st + STAGES - 1, last);
      const char* ta = smem + buf * A_BYTES;
      const char* tb = smem + STAGES * A_BYTES + (DEEP ? buf : st & 1) * B_BYTES;
#pragma unroll
      for (int kk = 0; kk < kStepK / 32; ++kk) {
        half8 fb[FN], fa[FM];
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = frag<BN, B_ROW>(tb, ncol(wn, j), kk, lane);
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = frag<BM, A_ROW>(ta, wm * (BM / WM) + i * 16, kk, lane);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[j][i] = mfma16<BF16>(fb[j], fa[i], acc[j][i]);
      }
      buf = buf + 1 == STAGES ? 0 : buf + 1;
    }
  }

  // ---- the accumulators as rows ----
  //
  // to_rows leaves the rows of phase `ph` (as many as fit the operand buffers)
  // in LDS.
  static constexpr int PHASES = BM * BN * 4 <= LDS_BYTES ? 1 : WM;
  using Rows = LdsRows<BM / PHASES, BN, NT>;
  static_assert(Rows::PH_ROWS * BN * 4 <= LDS_BYTES, "a phase's rows fit the operand buffers");
  static __device__ __forceinline__ void to_rows(char* smem, int ph, const float4v (&acc)[FN][FM]) {
    const int lane = threadIdx.x & 63, g = lane >> 4, s = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    __syncthreads();  // every wave has read its last operands, or the phase before
    if (PHASES == 1 || wm == ph) {
      const int r0 = PHASES == 1 ? wm * (BM / WM) : 0;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<float4v*>(smem + Rows::row_byte(r0 + i * 16 + s, ncol(wn, j) / 4 + g)) = acc[j][i];
    }
    __syncthreads();
  }
};

// Products of at most one 128 x 128 tile a compute unit take four buffers of
// both operands: their time is the latency of their steps' loads, and the LDS
// of a second workgroup is free.
inline bool few_tiles(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * ((cols + 127) / 128) <= 256;
}

// Waves per SIMD that the register budget leaves room for: two workgroups of
// a 128 x 128 tile on a compute unit, one of a larger or deeper one (LDS allows no
// more).
constexpr int tile_waves(int bm, int bn, int stages) {
  return bm * bn > 128 * 128 || stages > 3 ? 2 : 4;
}

// Output tile of a workgroup: tiles are walked n first, and each XCD
// (blockIdx % 8) takes a contiguous run of them, so that the n tiles which
// read the same rows of A share that XCD's L2.
struct TilePos {
  int64_t m, n;
};
__device__ __forceinline__ TilePos tile_pos(uint32_t m_tiles, uint32_t n_tiles, uint32_t bid) {
  const uint32_t total = m_tiles * n_tiles;  // a grid's size: 31 bits
  const uint32_t q = total >> 3, r = total & 7, x = bid & 7, j = bid >> 3;
  const uint32_t t = x * q + (x < r ? x : r) + j;
  const uint32_t m = t / n_tiles;
  return TilePos{m, t - m * n_tiles};
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int64_t round_to(int64_t v, int64_t unit) { return (v + unit - 1) / unit * unit; }
inline int64_t round8(int64_t v) { return round_to(v, 8); }
inline int64_t round64(int64_t v) { return round_to(v, 64); }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace
}  // namespace submconv
