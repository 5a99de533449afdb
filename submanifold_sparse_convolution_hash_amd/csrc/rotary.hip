// Rotary positions: the first 2 P columns of each head are P pairs that turn by
// the angle of their row's position.
//
//   pair p = a F + f of axis a:  t = position[row][a] freq[f]
//   (u, v) -> amplitude (u cos t - v sin t, v cos t + u sin t)
//
// Interleaved, pair p is columns 2 p and 2 p + 1; by halves, p and P + p. The
// columns from 2 P on are copied. The gradient is the turn by -t.
//
// Bound by memory: each value is read and written once. A thread computes the
// sines and cosines of its 16 bytes of pairs once and applies them to all heads
// of its row (or, where rows are few, to every heads-th one). Angles are formed
// in 64 bits, as turns, and only the part within a turn goes on in 32: position
// times frequency keeps 2^-24 of a turn up to 2^28 turns, where 32 bits would
// lose all of it.
#include <algorithm>

#include "dense_common.h"

namespace submconv {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kMaxAxes = 4;

template <typename T, int VEC>
__device__ __forceinline__ void get(const T* p, int n, float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  if (n >= VEC) {
    const vec t = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = e < n ? static_cast<float>(p[e]) : 0.0f;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void put(T* p, int n, const float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  if (n >= VEC) {
    vec t;
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = static_cast<T>(v[e]);  // round to nearest even
    *reinterpret_cast<vec*>(p) = t;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < n) p[e] = static_cast<T>(v[e]);
  }
}

struct Rotary {
  int64_t n;
  int heads, dim;
  int64_t ldx, hx, ldo, ho;  // elements between rows and between heads
  const int32_t* positions;
  int64_t ldp, ap;  // elements between rows and between axes
  const double* turns;  // radians per position [F]
  int F, pairs;
  float amplitude;
  int inverse;
  int turn_units, units;  // units of VEC columns (interleaved) or pairs (halves) a row; copies behind them
  int lanes;              // threads that share a row's unit, each with every lanes-th head
};

// cos and sin of pair p's angle, times the amplitude
__device__ __forceinline__ void turn_of(const Rotary& a, const int32_t* position, int p, float& c, float& s) {
  const int axis = p / a.F;
  const double t = static_cast<double>(position[axis * a.ap]) * (a.turns[p - axis * a.F] * 0.15915494309189533577);
  const float part = static_cast<float>(t - rint(t));  // of a turn, -1/2 .. 1/2
  float sn, cs;
  sincospif(2.0f * part, &sn, &cs);
  c = cs * a.amplitude;
  s = (a.inverse ? -sn : sn) * a.amplitude;
}

template <typename T, int VEC, bool PAIRS>
__global__ __launch_bounds__(kRotaryThreads) void k_rotary(const T* x, T* out, Rotary a) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
  const int unit = static_cast<int>(id % a.units);
  const int64_t rest = id / a.units;
  const int lane = static_cast<int>(rest % a.lanes);
  const int64_t row = rest / a.lanes;
  if (row >= a.n) return;
  const T* xr = x + row * a.ldx;
  T* yr = out + row * a.ldo;
  if (unit >= a.turn_units) {  // columns that do not turn
    const int c = 2 * a.pairs + (unit - a.turn_units) * VEC, n = a.dim - c;
#pragma unroll 4
    for (int h = lane; h < a.heads; h += a.lanes) {
      float v[VEC];
      get<T, VEC>(xr + h * a.hx + c, n, v);
      put<T, VEC>(yr + h * a.ho + c, n, v);
    }
    return;
  }
  const int32_t* position = a.positions + row * a.ldp;
  if constexpr (PAIRS) {
    const int c = unit * VEC, n = 2 * a.pairs - c;
    float cs[VEC / 2], sn[VEC / 2];
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) turn_of(a, position, min(c / 2 + e, a.pairs - 1), cs[e], sn[e]);
#pragma unroll 4
    for (int h = lane; h < a.heads; h += a.lanes) {
      float v[VEC];
      get<T, VEC>(xr + h * a.hx + c, n, v);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float u = v[2 * e], w = v[2 * e + 1];
        v[2 * e] = u * cs[e] - w * sn[e];
        v[2 * e + 1] = w * cs[e] + u * sn[e];
      }
      put<T, VEC>(yr + h * a.ho + c, n, v);
    }
  } else {
    const int c = unit * VEC, n = a.pairs - c;
    float cs[VEC], sn[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) turn_of(a, position, min(c + e, a.pairs - 1), cs[e], sn[e]);
#pragma unroll 2
    for (int h = lane; h < a.heads; h += a.lanes) {
      float v[VEC], w[VEC];
      get<T, VEC>(xr + h * a.hx + c, n, v);
      get<T, VEC>(xr + h * a.hx + a.pairs + c, n, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float u = v[e];
        v[e] = u * cs[e] - w[e] * sn[e];
        w[e] = w[e] * cs[e] + u * sn[e];
      }
      put<T, VEC>(yr + h * a.ho + c, n, v);
      put<T, VEC>(yr + h * a.ho + a.pairs + c, n, w);
    }
  }
}

template <typename T>
int rotate(const void* x, void* out, Rotary a, bool interleaved, hipStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  a.turn_units = static_cast<int>(((interleaved ? 2 * a.pairs : a.pairs) + VEC - 1) / VEC);
  a.units = a.turn_units + (x == out ? 0 : (a.dim - 2 * a.pairs + VEC - 1) / VEC);
  // A thread takes all heads where the rows alone fill the chip, else a share
  // of them, so that there are about 2^17 threads or one a head.
  const int64_t wide = std::max<int64_t>(1, (int64_t{1} << 17) / (a.n * a.units));
  a.lanes = static_cast<int>(std::min<int64_t>(a.heads, wide));
  const int64_t threads = a.n * a.units * a.lanes, blocks = (threads + kRotaryThreads - 1) / kRotaryThreads;
  if (blocks > INT32_MAX) return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%lld rows", (long long)a.n);
  const T* from = static_cast<const T*>(x);
  T* to = static_cast<T*>(out);
  if (interleaved) k_rotary<T, VEC, true><<<static_cast<unsigned>(blocks), kRotaryThreads, 0, stream>>>(from, to, a);
  else k_rotary<T, VEC, false><<<static_cast<unsigned>(blocks), kRotaryThreads, 0, stream>>>(from, to, a);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

int check_heads(const char* name, const void* p, int64_t n, int32_t heads, int32_t dim, int64_t ld, int64_t hs,
                int32_t dtype) {
  if (n > 0 && !p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (heads > 1 && hs < dim)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: head stride %lld below %d columns", name, (long long)hs, dim);
  if (n > 1 && ld < (heads - 1) * (heads > 1 ? hs : 0) + dim)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: row stride %lld below a row's columns", name, (long long)ld);
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
  if (heads < 1 || dim < 2 || heads > 65536 || dim > 65536)
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
