// Rotary positions: the first 2 P columns of each head are P pairs that turn by
// the angle of their row's position.
//
//   pair p = a F + f of axis a:  t = position[row][a] freq[f]
//   (u, v) -> amplitude (u cos t - v sin t, v cos t + u sin t)
//
// Interleaved, pair p is columns 2 p and 2 p + 1; by halves, p and P + p. The
// columns from 2 P on are copied. The gradient is the turn by -t.
//
// Bound by memory: each value is read and written once. A workgroup takes a run
// of rows: it puts the cosines and sines of their pairs into LDS, then streams the
// rows through, 16 bytes a thread, neighbouring threads neighbouring pieces of all
// heads: 209715 x 8 x 64 fp16 with three axes (60 columns turn) takes 80 us, as a
// copy does. Angles are formed in 64 bits, as turns, and only the part within a
// turn goes on in 32: position times frequency keeps 2^-24 of a turn up to 2^28
// turns, where 32 bits would lose all of it.
#include <algorithm>

#include "dense_common.h"

namespace submconv {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kMaxAxes = 4;

// The first n of VEC values at any element's address, in at most three pieces
// of a power of two (a last piece of a row taken value by value made 209715 rows
// of 60 turned columns in 64 three times slower).
template <typename T, int N, int AT, int VEC>
__device__ __forceinline__ void get_part(const T* p, float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  const vec t = *reinterpret_cast<const vec*>(p + AT);
#pragma unroll
  for (int e = 0; e < N; ++e) v[AT + e] = static_cast<float>(t[e]);
}
template <typename T, int N, int AT, int VEC>
__device__ __forceinline__ void put_part(T* p, const float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  vec t;
#pragma unroll
  for (int e = 0; e < N; ++e) t[e] = static_cast<T>(v[AT + e]);  // round to nearest even
  *reinterpret_cast<vec*>(p + AT) = t;
}
#define SUBMCONV_ROTARY_PARTS(part)                        \
  if (n >= VEC) {                                          \
    part<T, VEC, 0>(p, v);                                 \
    return;                                                \
  }                                                        \
  if constexpr (VEC == 8) {                                \
    if (n >= 4) {                                          \
      part<T, 4, 0>(p, v);                                 \
      if (n >= 6) part<T, 2, 4>(p, v);                     \
      if (n == 7) part<T, 1, 6>(p, v);                     \
      if (n == 5) part<T, 1, 4>(p, v);                     \
      return;                                              \
    }                                                      \
  }                                                        \
  if (n >= 2) part<T, 2, 0>(p, v);                         \
  if (n == 3) part<T, 1, 2>(p, v);                         \
  if (n == 1) part<T, 1, 0>(p, v);
template <typename T, int VEC>
__device__ __forceinline__ void get(const T* p, int n, float (&v)[VEC]) {
  SUBMCONV_ROTARY_PARTS(get_part)
}
template <typename T, int VEC>
__device__ __forceinline__ void put(T* p, int n, const float (&v)[VEC]) {
  SUBMCONV_ROTARY_PARTS(put_part)
}
#undef SUBMCONV_ROTARY_PARTS

// u c + v s, one way for all columns and layouts, so that a value does not depend
// on where its piece starts
__device__ __forceinline__ float turned(float u, float c, float v, float s) { return fmaf(u, c, v * s); }

struct Rotary {
  int64_t n;
  int heads, dim;
  int64_t ldx, hx, ldo, ho;  // elements between rows and between heads
  const int32_t* positions;
  int64_t ldp, ap;      // elements between rows and between axes
  const double* freqs;  // radians per position [F]
  int F, pairs;
  float amplitude;
  int inverse;
  int stride;            // of a row's cosines and sines in LDS
  int turn_units, units;  // pieces of a head, those that turn first
  int rows, share;        // rows and heads of a workgroup
};

constexpr int kRotaryPairs = 4096;  // at most, in LDS: 32 KB of cosines and sines
constexpr int kRotaryRun = 512;     // of a workgroup's rows, where a row has fewer
constexpr int kPiecesAhead = 4;     // of a thread in flight

// What a thread's piece of VEC is. Interleaved: columns. Halves: pairs, both of
// whose halves it reads and writes, and behind them columns that do not turn.
//
// Where pairs are no multiple of VEC, the last piece of halves lies over the one
// before it and both write the same values: a shorter piece would cost seven
// memory instructions a turn in place of two (209715 rows of 60 turned columns in
// 64: 176 us with shorter pieces, 135 so). Not in place, where the one would
// read what the other has written.
template <int VEC>
__device__ __forceinline__ int piece_start(int u, int total, bool over) {
  return over ? min(u * VEC, total - VEC) : u * VEC;
}

template <typename T, int VEC, bool PAIRS>
__global__ __launch_bounds__(kRotaryThreads) void k_rotary(const T* x, T* out, Rotary a) {
  extern __shared__ float2 turns[];  // [rows][stride] {cos, sin}
  const int stride = a.stride, others = a.dim - 2 * a.pairs;
  const bool over = x != out && a.pairs >= VEC, over_others = x != out && others >= VEC;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  const int rows = static_cast<int>(min(a.n - row0, static_cast<int64_t>(a.rows)));
  const int head0 = blockIdx.y * a.share, heads = min(a.share, a.heads - head0);
  for (int id = threadIdx.x; id < rows * stride; id += kRotaryThreads) {
    const int row = id / stride, p = min(id - row * stride, a.pairs - 1), axis = p / a.F;
    const double at = a.positions[(row0 + row) * a.ldp + axis * a.ap];
    const double t = at * (a.freqs[p - axis * a.F] * 0.15915494309189533577);
    float sn, cs;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &sn, &cs);  // of -1/2 .. 1/2 turns
    turns[id] = float2{cs * a.amplitude, (a.inverse ? -sn : sn) * a.amplitude};
  }
  __syncthreads();
  x += row0 * a.ldx + head0 * a.hx;
  out += row0 * a.ldo + head0 * a.ho;
  // piece (row, head, unit), the unit running fastest; a thread's next one is 256 on
  const int du = kRotaryThreads % a.units, dh = kRotaryThreads / a.units % heads;
  const int dr = kRotaryThreads / a.units / heads;
  int unit = threadIdx.x % a.units, head = threadIdx.x / a.units % heads, row = threadIdx.x / a.units / heads;
  while (row < rows) {
    float v[kPiecesAhead][VEC], w[PAIRS ? 1 : kPiecesAhead][VEC];
    int at[kPiecesAhead][3];
#pragma unroll
    for (int i = 0; i < kPiecesAhead; ++i) {
      at[i][0] = unit;
      at[i][1] = head;
      at[i][2] = row;
      unit += du;
      head += dh;
      row += dr;
      if (unit >= a.units) {
        unit -= a.units;
        ++head;
      }
      if (head >= heads) {
        head -= heads;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < kPiecesAhead; ++i) {
      const auto [u, h, r] = at[i];
      if (r >= rows) break;
      const T* p = x + r * a.ldx + h * a.hx;
      if constexpr (PAIRS) {
        get<T, VEC>(p + u * VEC, a.dim - u * VEC, v[i]);
      } else if (u < a.turn_units) {
        const int c = piece_start<VEC>(u, a.pairs, over);
        get<T, VEC>(p + c, a.pairs - c, v[i]);
        get<T, VEC>(p + a.pairs + c, a.pairs - c, w[i]);
      } else {
        const int c = piece_start<VEC>(u - a.turn_units, others, over_others);
        get<T, VEC>(p + 2 * a.pairs + c, others - c, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kPiecesAhead; ++i) {
      const auto [u, h, r] = at[i];
      if (r >= rows) break;
      T* p = out + r * a.ldo + h * a.ho;
      if constexpr (PAIRS) {
        const float2* t = turns + r * stride + u * (VEC / 2);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          if (u * (VEC / 2) + e >= a.pairs) break;  // columns that do not turn
          const float f = v[i][2 * e], g = v[i][2 * e + 1];
          v[i][2 * e] = turned(f, t[e].x, -g, t[e].y);
          v[i][2 * e + 1] = turned(g, t[e].x, f, t[e].y);
        }
        put<T, VEC>(p + u * VEC, a.dim - u * VEC, v[i]);
      } else if (u < a.turn_units) {
        const int c = piece_start<VEC>(u, a.pairs, over);
        const float2* t = turns + r * stride + c;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float f = v[i][e];
          v[i][e] = turned(f, t[e].x, -w[i][e], t[e].y);
          w[i][e] = turned(w[i][e], t[e].x, f, t[e].y);
        }
        put<T, VEC>(p + c, a.pairs - c, v[i]);
        put<T, VEC>(p + a.pairs + c, a.pairs - c, w[i]);
      } else {
        const int c = piece_start<VEC>(u - a.turn_units, others, over_others);
        put<T, VEC>(p + 2 * a.pairs + c, others - c, v[i]);
      }
    }
  }
}

template <typename T>
int rotate(const void* x, void* out, Rotary a, bool interleaved, hipStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  a.turn_units = ((interleaved ? 2 * a.pairs : a.pairs) + VEC - 1) / VEC;
  // (in place, columns that do not turn stay where they are)
  const int others = interleaved ? a.dim - a.turn_units * VEC : a.dim - 2 * a.pairs;
  a.units = a.turn_units + (x == out || others <= 0 ? 0 : (others + VEC - 1) / VEC);
  a.stride = interleaved ? a.turn_units * (VEC / 2) : a.turn_units * VEC;
  // As many rows as fill 512 pairs, where there are 2048 workgroups of them
  // (209715 x 8 x 64 with one axis: 79 us; 4096 pairs 105, 256 88). With few rows
  // their heads are shared out as well, 256 pieces or more a workgroup. With very many
  // rows no more workgroups than a launch can have.
  a.rows = static_cast<int>(std::clamp<int64_t>(a.n / 2048, 1, std::max(1, kRotaryRun / a.stride)));
  while (!launch_fits((a.n + a.rows - 1) / a.rows, kRotaryThreads)) ++a.rows;
  const int64_t blocks = (a.n + a.rows - 1) / a.rows;
  const int64_t shares = std::clamp<int64_t>(256 / blocks, 1, std::max<int64_t>(1, int64_t{a.heads} * a.units / 256));
  a.share = static_cast<int>((a.heads + shares - 1) / shares);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((a.heads + a.share - 1) / a.share));
  const int lds = a.rows * a.stride * static_cast<int>(sizeof(float2));
  if (lds > 65536)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%lld rows of %d pairs", (long long)a.n, a.pairs);
  const T* from = static_cast<const T*>(x);
  T* to = static_cast<T*>(out);
  if (interleaved) k_rotary<T, VEC, true><<<grid, kRotaryThreads, lds, stream>>>(from, to, a);
  else k_rotary<T, VEC, false><<<grid, kRotaryThreads, lds, stream>>>(from, to, a);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int check_heads(const char* name, const void* p, int64_t n, int32_t heads, int32_t dim, int64_t ld, int64_t hs,
                int32_t dtype) {
  if (n > 0 && !p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  const bool rows_of_heads = hs >= dim && ld >= (heads - 1) * hs + dim;
  const bool heads_of_rows = ld >= dim && hs >= (n - 1) * ld + dim;
  if ((heads > 1 && hs < dim) || (n > 1 && ld < dim) || (heads > 1 && n > 1 && !rows_of_heads && !heads_of_rows))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: rows or heads overlap with strides %lld and %lld", name,
                     (long long)ld, (long long)hs);
  if (reinterpret_cast<uintptr_t>(p) & (dtype == SUBMCONV_DTYPE_F32 ? 3 : 1))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  return SUBMCONV_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int submconv_rotary(const void* x, int64_t ldx, int64_t hx, int64_t n, int32_t heads, int32_t dim,
                               const int32_t* positions, int64_t ldp, int64_t ap, int32_t axes, const double* freqs,
                               int32_t nfreqs, int32_t interleaved, int32_t inverse, float amplitude, void* out,
                               int64_t ldo, int64_t ho, int32_t dtype, hipStream_t stream) {
  clear_error();
  if (n < 0 || n > INT32_MAX) return set_error(SUBMCONV_ERR_INVALID_ARG, "n = %lld", (long long)n);
  if (heads < 1 || dim < 2 || heads > 65536 || dim > 2 * kRotaryPairs)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%d heads of %d columns", heads, dim);
  if (axes < 1 || axes > kMaxAxes)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%d axes, 1 to %d are supported", axes, kMaxAxes);
  if (nfreqs < 1 || static_cast<int64_t>(nfreqs) * axes * 2 > dim)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d axes of %d pairs in %d columns", axes, nfreqs, dim);
  if (dtype != SUBMCONV_DTYPE_F16 && dtype != SUBMCONV_DTYPE_BF16 && dtype != SUBMCONV_DTYPE_F32)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "dtype = %d", dtype);
  SUBMCONV_TRY(check_heads("x", x, n, heads, dim, ldx, hx, dtype));
  SUBMCONV_TRY(check_heads("out", out, n, heads, dim, ldo, ho, dtype));
  if (n > 0 && (!positions || !freqs)) return set_error(SUBMCONV_ERR_INVALID_ARG, "positions or freqs is NULL");
  if ((reinterpret_cast<uintptr_t>(positions) & 3) || (reinterpret_cast<uintptr_t>(freqs) & 7))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "positions or freqs is not aligned to its elements");
  if (x == out && n > 0 && ((n > 1 && ldx != ldo) || (heads > 1 && hx != ho)))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "in place, but with other strides");
  if (n == 0) return SUBMCONV_OK;
  const Rotary a{n, heads, dim, ldx, hx, ldo, ho, positions, ldp, ap, freqs, nfreqs, nfreqs * axes, amplitude, inverse, 0, 0, 0};
  if (dtype == SUBMCONV_DTYPE_F16) return rotate<_Float16>(x, out, a, interleaved, stream);
  if (dtype == SUBMCONV_DTYPE_BF16) return rotate<__bf16>(x, out, a, interleaved, stream);
  return rotate<float>(x, out, a, interleaved, stream);
}
