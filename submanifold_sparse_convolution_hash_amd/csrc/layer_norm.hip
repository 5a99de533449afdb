// Layer norm over the channels of site features, and its gradients.
//
//   m = mean_c x,  v = mean_c (x - m)^2,  r = 1 / sqrt(v + eps)
//   xh = (x - m) r,  y = xh w + b
//   d = dy w,  dx = r (d - mean_c d - xh mean_c (d xh))
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory: x (and dy) are read once and y (dx) is written once. A row
// is held in the registers of G lanes, so the variance is a second pass over
// registers about the mean (no cancellation) and not over memory; several
// rows share a wave when a row needs fewer than 64 lanes. All arithmetic and
// the statistics are fp32, y and dx are rounded once. dw and db stay in
// registers over all rows a workgroup walks; the workgroups' sums are added
// by a second small kernel in a fixed order, so results repeat bit for bit.
#include <algorithm>

#include "dense_common.h"
#include "lane_ops.h"
#include "submconv_internal.h"

namespace submconv {
namespace {

constexpr int kNormThreads = 256;
constexpr int64_t kMaxChannels = 8192;  // 256 lanes of 32 values

// ---- elements ----

// Columns c .. c + VEC - 1 of a row, zeros past C (16 bytes at any element's
// address: the memory system takes an access that is not aligned to its size,
// at the cost of the lines it straddles).
template <typename T, int VEC>
__device__ __forceinline__ void load_piece(const T* row, int c, int C, float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  if (c + VEC <= C) {
    const vec t = *reinterpret_cast<const vec*>(row + c);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = static_cast<float>(t[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = c + e < C ? static_cast<float>(row[c + e]) : 0.0f;
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T* row, int c, int C, const float (&v)[VEC]) {
  typedef T vec __attribute__((ext_vector_type(VEC), aligned(sizeof(T))));
  if (c + VEC <= C) {
    vec t;
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = static_cast<T>(v[e]);  // round to nearest even
    *reinterpret_cast<vec*>(row + c) = t;
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (c + e < C) row[c + e] = static_cast<T>(v[e]);
  }
}

// VEC weights from column c of [C] (zeros past it, or from a null vector),
// without a branch.
template <int VEC>
__device__ __forceinline__ void load_weights(const float* w, int C, int c, float (&v)[VEC]) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(w), static_cast<short>(0), w ? C * 4 : 0, 0x00020000);
  typedef float float4v __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int e = 0; e < VEC; e += 4) {
    const float4v t = __builtin_bit_cast(float4v, __builtin_amdgcn_raw_buffer_load_b128(r, (c + e) * 4, 0, 0));
#pragma unroll
    for (int q = 0; q < 4; ++q) v[e + q] = t[q];
  }
}

// ---- sums over the G lanes of a row, the same in each of them ----

// G = 256: the four waves' sums through LDS (`slot`: a place per use, so that
// one barrier is enough)
template <int G>
__device__ __forceinline__ float row_sum(float x, float* slot) {
  x = lanes_sum<(G < 64 ? G : 64)>(x);
  if constexpr (G > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (slot[0] + slot[1]) + (slot[2] + slot[3]);
  }
  return x;
}

// 209715 x 128 fp16 19 us (107 MB), 1 x 1024 2.4 us.
// Lane l of a row's G holds V pieces of VEC columns, piece i at column
// (i G + l) VEC.
template <typename T, int VEC, int G, int V>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm(
    const T* __restrict__ x, int64_t ldx, int64_t n, int C, const float* __restrict__ w,
    const float* __restrict__ b, float eps, float inv_c, T* __restrict__ y,
    float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int RPB = kNormThreads / G;  // rows at a time
  __shared__ float slots[2][2][4];
  const int l = threadIdx.x % G;
  const bool lead = l == 0;
  float wv[V][VEC], bv[V][VEC];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    load_weights<VEC>(w, C, (i * G + l) * VEC, wv[i]);
    load_weights<VEC>(b, C, (i * G + l) * VEC, bv[i]);
  }
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPB; r0 < n;
       r0 += static_cast<int64_t>(gridDim.x) * RPB, turn ^= 1) {
    const int64_t r = r0 + threadIdx.x / G;
    const bool live = r < n;  // for G = 256 the same in all threads
    float v[V][VEC];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.0f;
      if (live) load_piece<T, VEC>(x + r * ldx, c, C, v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[i][e];
    }
    const float m = row_sum<G>(s, slots[turn][0]) * inv_c;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] -= m;
        q += c + e < C ? v[i][e] * v[i][e] : 0.0f;
      }
    }
    const float rs = 1.0f / sqrtf(row_sum<G>(q, slots[turn][1]) * inv_c + eps);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = v[i][e] * rs * (w ? wv[i][e] : 1.0f) + bv[i][e];
      store_piece<T, VEC>(y + r * C, c, C, v[i]);
    }
    if (lead) {
      if (mean) mean[r] = m;
      if (rstd) rstd[r] = rs;
    }
  }
}

// dx, and where partial is not null this workgroup's sums of dy xh and dy,
// [2][C] of it. 209715 x 128 bf16 28 us (161 MB), 20011 x 515 fp32 24 us
// (124 MB): a copy's rate.
template <typename T, int VEC, int G, int V>
__global__ __launch_bounds__(kNormThreads) void k_layer_norm_grad(
    const T* __restrict__ dy, int64_t ldg, const T* __restrict__ x, int64_t ldx, int64_t n, int C,
    const float* __restrict__ mean, const float* __restrict__ rstd, const float* __restrict__ w,
    float inv_c, T* __restrict__ dx, float* __restrict__ partial) {
  constexpr int RPB = kNormThreads / G;
  constexpr int COLS = G * V * VEC;
  __shared__ float slots[2][2][4];
  __shared__ float sums[G <= 64 ? 4 * 2 * COLS : 1];
  const int l = threadIdx.x % G;
  float wv[V][VEC], sw[V][VEC] = {}, sb[V][VEC] = {};
#pragma unroll
  for (int i = 0; i < V; ++i) {
    load_weights<VEC>(w, C, (i * G + l) * VEC, wv[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) wv[i][e] = w ? wv[i][e] : 1.0f;
  }
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * RPB; r0 < n;
       r0 += static_cast<int64_t>(gridDim.x) * RPB, turn ^= 1) {
    const int64_t r = r0 + threadIdx.x / G;
    const bool live = r < n;
    const float m = live ? mean[r] : 0.0f, rs = live ? rstd[r] : 0.0f;
    float d[V][VEC], xh[V][VEC];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[i][e] = xh[i][e] = 0.0f;
      if (live) {
        load_piece<T, VEC>(dy + r * ldg, c, C, d[i]);
        load_piece<T, VEC>(x + r * ldx, c, C, xh[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        xh[i][e] = live && c + e < C ? (xh[i][e] - m) * rs : 0.0f;
        sw[i][e] += d[i][e] * xh[i][e];
        sb[i][e] += d[i][e];
        d[i][e] *= wv[i][e];
        s1 += d[i][e];
        s2 += d[i][e] * xh[i][e];
      }
    }
    if (!dx) continue;
    s1 = row_sum<G>(s1, slots[turn][0]) * inv_c;
    s2 = row_sum<G>(s2, slots[turn][1]) * inv_c;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * G + l) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[i][e] = rs * (d[i][e] - s1 - xh[i][e] * s2);
      store_piece<T, VEC>(dx + r * C, c, C, d[i]);
    }
  }
  if (!partial) return;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * C;
  if constexpr (G > 64) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * G + l) * VEC + e;
        if (c < C) {
          out[c] = sw[i][e];
          out[C + c] = sb[i][e];
        }
      }
  } else {
    // the wave's rows, then the four waves
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float a = sw[i][e], c = sb[i][e];
#pragma unroll
        for (int o = G; o < 64; o <<= 1) {
          a += __shfl_xor(a, o, 64);
          c += __shfl_xor(c, o, 64);
        }
        if (lane < G) {
          sums[(wave * 2) * COLS + (i * G + l) * VEC + e] = a;
          sums[(wave * 2 + 1) * COLS + (i * G + l) * VEC + e] = c;
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * COLS; c += kNormThreads) {
      const int col = c % COLS;
      if (col < C)
        out[c / COLS * C + col] = (sums[c] + sums[2 * COLS + c]) + (sums[4 * COLS + c] + sums[6 * COLS + c]);
    }
  }
}

// ---- dispatch: lanes and values per row by the width ----

// Workgroups: eight a compute unit for the forward (its loop keeps the
// weights), four for the gradient, whose column sums cost 8 C bytes each.
constexpr int64_t kNormBlocks = 2048, kNormGradBlocks = 1024;

template <int VEC, typename F>
int by_width(int64_t C, F&& f) {
  using std::integral_constant;
  auto go = [&](auto g, auto v) { return f(g, v); };
#define SUBMCONV_NORM(G, V) return go(integral_constant<int, G>{}, integral_constant<int, V>{})
  if (C <= 8 * VEC) SUBMCONV_NORM(8, 1);
  if (C <= 16 * VEC) SUBMCONV_NORM(16, 1);
  if (C <= 32 * VEC) SUBMCONV_NORM(32, 1);
  if (C <= 64 * VEC) SUBMCONV_NORM(64, 1);
  if (C <= 128 * VEC) SUBMCONV_NORM(64, 2);
  if (C <= 256 * VEC) SUBMCONV_NORM(64, 4);
  if constexpr (VEC == 4)
    if (C <= 512 * VEC) SUBMCONV_NORM(64, 8);
  SUBMCONV_NORM(256, 32 / VEC);
#undef SUBMCONV_NORM
}

template <typename T>
int norm_forward(const void* x, int64_t ldx, int64_t n, int C, const float* w, const float* b,
                 float eps, void* y, float* mean, float* rstd, hipStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  return by_width<VEC>(C, [&](auto g, auto v) {
    const int64_t rpb = kNormThreads / g;
    const int64_t blocks = std::min((n + rpb - 1) / rpb, kNormBlocks);
    k_layer_norm<T, VEC, g, v><<<static_cast<unsigned>(blocks), kNormThreads, 0, stream>>>(
        static_cast<const T*>(x), ldx, n, C, w, b, eps, 1.0f / static_cast<float>(C),
        static_cast<T*>(y), mean, rstd);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  });
}

template <typename T>
int norm_backward(const void* dy, int64_t ldg, const void* x, int64_t ldx, int64_t n, int C,
                  const float* mean, const float* rstd, const float* w, void* dx, float* partial,
                  int64_t* parts, hipStream_t stream) {
  constexpr int VEC = 16 / sizeof(T);
  return by_width<VEC>(C, [&](auto g, auto v) {
    const int64_t rpb = kNormThreads / g;
    const int64_t blocks = std::max<int64_t>(1, std::min((n + rpb - 1) / rpb, kNormGradBlocks));
    *parts = blocks;
    k_layer_norm_grad<T, VEC, g, v><<<static_cast<unsigned>(blocks), kNormThreads, 0, stream>>>(
        static_cast<const T*>(dy), ldg, static_cast<const T*>(x), ldx, n, C, mean, rstd, w,
        1.0f / static_cast<float>(C), static_cast<T*>(dx), partial);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  });
}

int check_norm(int64_t n, int32_t cdim, int32_t dtype) {
  if (n < 0) return set_error(SUBMCONV_ERR_INVALID_ARG, "n = %lld", (long long)n);
  if (cdim < 1 || cdim > kMaxChannels)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "C = %d, 1 to %lld are supported", cdim,
                     (long long)kMaxChannels);
  if (dtype != SUBMCONV_DTYPE_F16 && dtype != SUBMCONV_DTYPE_BF16 && dtype != SUBMCONV_DTYPE_F32)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "dtype = %d", dtype);
  return SUBMCONV_OK;
}

int check_rows(const char* name, const void* p, int64_t n, int32_t cdim, int64_t ld, int32_t dtype) {
  if (n > 0 && !p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (n > 1 && ld < cdim)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: row stride %lld below %d columns", name,
                     (long long)ld, cdim);
  const uintptr_t mask = dtype == SUBMCONV_DTYPE_F32 ? 3 : 1;
  if (reinterpret_cast<uintptr_t>(p) & mask)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  return SUBMCONV_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int submconv_layer_norm(const void* x, int64_t ldx, int64_t n, int32_t cdim,
                                   const float* weight, const float* bias, float eps, void* y,
                                   float* mean, float* rstd, int32_t dtype, hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_norm(n, cdim, dtype));
  SUBMCONV_TRY(check_rows("x", x, n, cdim, ldx, dtype));
  SUBMCONV_TRY(check_rows("y", y, n, cdim, cdim, dtype));
  if (!(eps >= 0.0f)) return set_error(SUBMCONV_ERR_INVALID_ARG, "eps = %g", eps);
  if (n == 0) return SUBMCONV_OK;
  const int64_t ld = n == 1 ? cdim : ldx;
  if (dtype == SUBMCONV_DTYPE_F16)
    return norm_forward<_Float16>(x, ld, n, cdim, weight, bias, eps, y, mean, rstd, stream);
  if (dtype == SUBMCONV_DTYPE_BF16)
    return norm_forward<__bf16>(x, ld, n, cdim, weight, bias, eps, y, mean, rstd, stream);
  return norm_forward<float>(x, ld, n, cdim, weight, bias, eps, y, mean, rstd, stream);
}

extern "C" int64_t submconv_layer_norm_backward_workspace_bytes(int64_t n, int32_t cdim) {
  clear_error();
  SUBMCONV_TRY(check_norm(n, cdim, SUBMCONV_DTYPE_F32));
  return std::max<int64_t>(1, std::min(n, kNormGradBlocks)) * 2 * cdim * 4;
}

extern "C" int submconv_layer_norm_backward(const void* grad_out, int64_t ldg, const void* x,
                                            int64_t ldx, int64_t n, int32_t cdim, const float* mean,
                                            const float* rstd, const float* weight, void* grad_x,
                                            float* grad_weight, float* grad_bias, int32_t dtype,
                                            void* workspace, int64_t workspace_bytes,
                                            hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_norm(n, cdim, dtype));
  SUBMCONV_TRY(check_rows("grad_out", grad_out, n, cdim, ldg, dtype));
  SUBMCONV_TRY(check_rows("x", x, n, cdim, ldx, dtype));
  SUBMCONV_TRY(check_rows("grad_x", grad_x, grad_x ? n : 0, cdim, cdim, dtype));
  if (n > 0 && (!mean || !rstd)) return set_error(SUBMCONV_ERR_INVALID_ARG, "mean or rstd is NULL");
  const bool params = grad_weight || grad_bias;
  const int64_t need =
      params ? std::max<int64_t>(1, std::min(n, kNormGradBlocks)) * 2 * cdim * 4 : 0;
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, need));
  if (!grad_x && !params) return SUBMCONV_OK;
  if (n == 0 && !params) return SUBMCONV_OK;
  float* partial = params ? static_cast<float*>(workspace) : nullptr;
  const int64_t lg = n == 1 ? cdim : ldg, lx = n == 1 ? cdim : ldx;
  int64_t parts = 0;
  if (dtype == SUBMCONV_DTYPE_F16)
    SUBMCONV_TRY(norm_backward<_Float16>(grad_out, lg, x, lx, n, cdim, mean, rstd, weight, grad_x,
                                         partial, &parts, stream));
  else if (dtype == SUBMCONV_DTYPE_BF16)
    SUBMCONV_TRY(norm_backward<__bf16>(grad_out, lg, x, lx, n, cdim, mean, rstd, weight, grad_x,
                                       partial, &parts, stream));
  else
    SUBMCONV_TRY(norm_backward<float>(grad_out, lg, x, lx, n, cdim, mean, rstd, weight, grad_x,
                                      partial, &parts, stream));
  SumList sums;
  if (grad_weight && grad_bias)
    sums.job[sums.count++] = SumJob{partial, parts, 2 * cdim, 2 * cdim, 1, grad_weight, cdim, grad_bias};
  else if (grad_weight)
    sums.job[sums.count++] = SumJob{partial, parts, 2 * cdim, cdim, 1, grad_weight};
  else if (grad_bias)
    sums.job[sums.count++] = SumJob{partial + cdim, parts, 2 * cdim, cdim, 1, grad_bias};
  return run_sums(sums, stream);
}
