// Group norm over the rows of packed items with an activation, and its
// gradients. Per item and group of C / G neighbouring channels, over the item's
// rows and the group's channels:
//
//   m = mean x,  v = mean (x - m)^2,  r = 1 / sqrt(v + eps)
//   xh = (x - m) r,  z = xh w + b,  y = act(z)
//   dz = dy act'(z),  d = dz w,  dx = r (d - mean d - xh mean (d xh))
//   dw = sum over all rows of dz xh,  db = sum of dz
//
// Bound by memory: the statistics need all of an item before its first output,
// so x (and dy) are read twice. The rows are cut into chunks of one item each:
// a first launch leaves each chunk's sums, a second joins them, a third makes
// the outputs. A thread keeps its 16 bytes of columns for all rows of its
// chunk, so that sums per channel stay in registers. All sums are fp32 and
// joined in a fixed order: results repeat bit for bit. Means and squares about
// the mean are joined pairwise (n, mean, square sum), so that a mean of many
// deviations costs no digits.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "items.h"

namespace submconv {
namespace {

constexpr int kGroupThreads = 256;
constexpr int kGroupChannels = 8192;
constexpr int kRowsAhead = 4;  // rows of a thread in flight

// ---- elements ----

// Columns c .. c + VEC - 1 of a row, zeros past C, at any element's address.
template <typename T, int VEC>
__device__ __forceinline__ void read_piece(const T* row, int c, int C, float (&v)[VEC]) {
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
__device__ __forceinline__ void write_piece(T* row, int c, int C, const float (&v)[VEC]) {
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

// ---- a thread's place: piece l + i lanes of V, row r of `rl` at a time ----

struct Lanes {
  int lanes, rl;  // rl = 256 / lanes where V = 1, else 1
};
inline Lanes lanes_of(int cols, int vec) {
  const int pieces = (cols + vec - 1) / vec;
  return pieces <= kGroupThreads ? Lanes{pieces, kGroupThreads / pieces} : Lanes{kGroupThreads, 1};
}
// floats of LDS for two values per channel and row of threads
inline int lanes_lds(const Lanes& g, int vec, int v) { return 2 * g.rl * g.lanes * vec * v; }

// ---- running mean and sum of squares about it ----

struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments joined(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  const float w = n > 0.0f ? b.n / n : 0.0f, d = b.mean - a.mean;
  return Moments{n, a.mean + d * w, a.m2 + b.m2 + d * d * (a.n * w)};
}
__device__ __forceinline__ Moments lanes_joined(Moments m, int width) {
  for (int o = 1; o < width; o <<= 1)
    m = joined(m, Moments{__shfl_xor(m.n, o, 64), __shfl_xor(m.mean, o, 64), __shfl_xor(m.m2, o, 64)});
  return m;
}

// Threads that work on one group: a power of two up to 64.
__device__ __forceinline__ int group_width(int groups) {
  int w = 1;
  while (w < 64 && 2 * w * groups <= kGroupThreads) w <<= 1;
  return w;
}

// The moments of `rows` rows of columns 0 .. cols - 1 per group, to f(group,
// moments) in one thread of each. lds: [2][rl][lanes V VEC].
template <typename T, int VEC, int V, typename F>
__device__ __forceinline__ void chunk_moments(const T* x, int64_t ldx, int64_t rows, int cols, int cpg, Lanes g,
                                              float* lds, F&& f) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  const int wide = g.lanes * VEC * V;
  float mean[V][VEC] = {}, m2[V][VEC] = {};
  if (rr < g.rl) {
    float cnt = 0.0f;
    for (int64_t r = rr; r < rows; r += g.rl * kRowsAhead) {
      const int64_t left = (rows - r + g.rl - 1) / g.rl;
      const int live = left < kRowsAhead ? static_cast<int>(left) : kRowsAhead;
      const float nb = static_cast<float>(live), inv = 1.0f / nb;
      const float w = nb / (cnt + nb), k = cnt * w;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[kRowsAhead][VEC];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
          // (a row past the last reads the last again and counts for nothing)
          const int64_t at = r + static_cast<int64_t>(u < live ? u : live - 1) * g.rl;
          read_piece<T, VEC>(x + at * ldx, (i * g.lanes + l) * VEC, cols, v[u]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float s = 0.0f, q = 0.0f;
#pragma unroll
          for (int u = 0; u < kRowsAhead; ++u) s += u < live ? v[u][e] : 0.0f;
          const float mb = s * inv;
#pragma unroll
          for (int u = 0; u < kRowsAhead; ++u) {
            const float d = v[u][e] - mb;
            q += u < live ? d * d : 0.0f;
          }
          const float d = mb - mean[i][e];
          mean[i][e] += d * w;
          m2[i][e] += q + d * d * k;
        }
      }
      cnt += nb;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int at = rr * wide + (i * g.lanes + l) * VEC + e;
        lds[at] = mean[i][e];
        lds[g.rl * wide + at] = m2[i][e];
      }
  }
  __syncthreads();
  // the rows of threads, in order: row i of them took (rows - i + rl - 1) / rl rows
  for (int c = threadIdx.x; c < cols; c += kGroupThreads) {
    Moments m{0.0f, 0.0f, 0.0f};
    for (int i = 0; i < g.rl; ++i) {
      const int64_t n = rows > i ? (rows - i + g.rl - 1) / g.rl : 0;
      m = joined(m, Moments{static_cast<float>(n), lds[i * wide + c], lds[(g.rl + i) * wide + c]});
    }
    lds[c] = m.mean;  // only this thread reads or writes this column
    lds[g.rl * wide + c] = m.m2;
  }
  __syncthreads();
  // the channels of a group
  const int groups = cols / cpg, width = group_width(groups);
  const int t = threadIdx.x % width;
  for (int k = threadIdx.x / width; k < groups; k += kGroupThreads / width) {
    Moments m{0.0f, 0.0f, 0.0f};
    for (int c = t; c < cpg; c += width)
      m = joined(m, Moments{static_cast<float>(rows), lds[k * cpg + c], lds[g.rl * wide + k * cpg + c]});
    m = lanes_joined(m, width);
    if (t == 0) f(k, m);
  }
}

// ---- forward ----

// partial [slots][G] {mean, square sum} of each chunk of 2^shift rows.
template <typename T, int VEC, int V>
__global__ __launch_bounds__(kGroupThreads) void k_group_moments(const T* __restrict__ x, int64_t ldx, Items it,
                                                                 int C, int cpg, Lanes g, int shift,
                                                                 float2* __restrict__ partial) {
  extern __shared__ float lds[];
  const ItemTile t = find_item(it, 1, shift, blockIdx.x);
  const int64_t r0 = t.tile << shift;
  if (t.item == it.items || t.tile < 0 || r0 >= t.rows) return;
  const int64_t rows = min(t.rows - r0, int64_t{1} << shift);
  const int G = C / cpg;
  chunk_moments<T, VEC, V>(x + (t.row0 + r0) * ldx, ldx, rows, C, cpg, g, lds, [&](int k, const Moments& m) {
    partial[static_cast<int64_t>(blockIdx.x) * G + k] = float2{m.mean, m.m2};
  });
}

// A wave joins the chunks of one item and group.
__global__ __launch_bounds__(kGroupThreads) void k_group_join(const float2* __restrict__ partial, Items it, int G,
                                                              int cpg, int shift, float eps,
                                                              float* __restrict__ mean, float* __restrict__ rstd) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (kGroupThreads / 64) + (threadIdx.x >> 6);
  if (at >= static_cast<int64_t>(it.items) * G) return;
  const int item = static_cast<int>(at / G), k = static_cast<int>(at % G), lane = threadIdx.x & 63;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1);
  const int64_t rows = e > s ? e - s : 0, slot = (s >> shift) + item, chunk = int64_t{1} << shift;
  Moments m{0.0f, 0.0f, 0.0f};
  for (int64_t c = lane; c * chunk < rows; c += 64) {
    const float2 p = partial[(slot + c) * G + k];
    m = joined(m, Moments{static_cast<float>(min(chunk, rows - c * chunk) * cpg), p.x, p.y});
  }
  m = lanes_joined(m, 64);
  if (lane == 0) {
    mean[at] = m.mean;
    rstd[at] = 1.0f / sqrtf((m.n > 0.0f ? m.m2 / m.n : 0.0f) + eps);
  }
}

// What a thread's columns are normalised with. mean and rstd of the item.
template <int VEC>
struct Affine {
  float m[VEC], r[VEC], w[VEC], b[VEC];
  __device__ __forceinline__ Affine(const float* mean, const float* rstd, const float* wp, const float* bp, int c,
                                    int C, int cpg) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int q = c + e < C ? c + e : C - 1;
      m[e] = mean[q / cpg];
      r[e] = rstd[q / cpg];
      w[e] = wp ? wp[q] : 1.0f;
      b[e] = bp ? bp[q] : 0.0f;
    }
  }
};

// y of `rows` rows of columns 0 .. cols - 1.
template <typename T, int VEC, int V, int ACT>
__device__ __forceinline__ void chunk_outputs(const T* x, int64_t ldx, T* y, int64_t ldy, int64_t rows, int cols,
                                              int cpg, Lanes g, const float* mean, const float* rstd,
                                              const float* w, const float* b) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  if (rr >= g.rl) return;
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const int c = (i * g.lanes + l) * VEC;
    if (c >= cols) return;
    const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = a.r[e] * a.w[e];
    for (int64_t r = rr; r < rows; r += g.rl * kRowsAhead) {
      const int64_t left = (rows - r + g.rl - 1) / g.rl;
      const int live = left < kRowsAhead ? static_cast<int>(left) : kRowsAhead;
      float v[kRowsAhead][VEC];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        read_piece<T, VEC>(x + (r + static_cast<int64_t>(u < live ? u : live - 1) * g.rl) * ldx, c, cols, v[u]);
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        if (u >= live) break;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[u][e] = act_value<ACT>((v[u][e] - a.m[e]) * s[e] + a.b[e]);
        write_piece<T, VEC>(y + (r + static_cast<int64_t>(u) * g.rl) * ldy, c, cols, v[u]);
      }
    }
  }
}

template <typename T, int VEC, int V>
__device__ __forceinline__ void chunk_zeros(T* y, int64_t ldy, int64_t rows, int cols, Lanes g) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  if (rr >= g.rl) return;
  const float zero[VEC] = {};
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const int c = (i * g.lanes + l) * VEC;
    if (c >= cols) return;
    for (int64_t r = rr; r < rows; r += g.rl) write_piece<T, VEC>(y + r * ldy, c, cols, zero);
  }
}

template <typename T, int VEC, int V>
__global__ __launch_bounds__(kGroupThreads) void k_group_apply(const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                               int cpg, Lanes g, int shift,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd,
                                                               const float* __restrict__ w,
                                                               const float* __restrict__ b, int act,
                                                               T* __restrict__ y) {
  const ItemTile t = find_item(it, 1, shift, blockIdx.x);
  const int64_t r0 = t.tile << shift;
  if (t.tile < 0 || r0 >= t.rows) return;
  const int64_t rows = min(t.rows - r0, int64_t{1} << shift), at = t.row0 + r0;
  if (t.item == it.items) {
    chunk_zeros<T, VEC, V>(y + at * C, C, rows, C, g);
    return;
  }
  const int64_t G = C / cpg;
  with_act(act, [&](auto a) {
    chunk_outputs<T, VEC, V, decltype(a)::value>(x + at * ldx, ldx, y + at * C, C, rows, C, cpg, g,
                                                 mean + t.item * G, rstd + t.item * G, w, b);
  });
}

// All of a few rows in one launch: a workgroup takes one item's columns of
// `gpw` groups. Workgroups of item number `items` clear the rows of no item.
template <typename T, int VEC>
__global__ __launch_bounds__(kGroupThreads) void k_group_norm(const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                              int cpg, int gpw, Lanes g,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ b, float eps, int act,
                                                              T* __restrict__ y, float* __restrict__ mean,
                                                              float* __restrict__ rstd) {
  extern __shared__ float lds[];
  __shared__ float gm[kGroupThreads], gr[kGroupThreads];
  const int item = blockIdx.x, G = C / cpg, k0 = blockIdx.y * gpw;
  const int groups = min(gpw, G - k0), c0 = k0 * cpg, cols = groups * cpg;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1), rows = e > s ? e - s : 0;
  y += s * C + c0;
  if (item == it.items) {
    chunk_zeros<T, VEC, 1>(y, C, rows, cols, g);
    return;
  }
  x += s * ldx + c0;
  chunk_moments<T, VEC, 1>(x, ldx, rows, cols, cpg, g, lds, [&](int k, const Moments& m) {
    const float r = 1.0f / sqrtf((m.n > 0.0f ? m.m2 / m.n : 0.0f) + eps);
    gm[k] = m.mean;
    gr[k] = r;
    const int64_t at = static_cast<int64_t>(item) * G + k0 + k;
    if (mean) mean[at] = m.mean;
    if (rstd) rstd[at] = r;
  });
  __syncthreads();
  with_act(act, [&](auto a) {
    chunk_outputs<T, VEC, 1, decltype(a)::value>(x, ldx, y, C, rows, cols, cpg, g, gm, gr, w ? w + c0 : nullptr,
                                                 b ? b + c0 : nullptr);
  });
}

// ---- gradients ----

// This chunk's sums of dz and dz xh per channel, to f(channel, sum dz, sum dz
// xh) in one thread of each.
template <typename T, int VEC, int V, int ACT, typename F>
__device__ __forceinline__ void chunk_sums(const T* dy, int64_t ldg, const T* x, int64_t ldx, int64_t rows, int cols,
                                           int cpg, Lanes g, const float* mean, const float* rstd, const float* w,
                                           const float* b, float* lds, F&& f) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  const int wide = g.lanes * VEC * V;
  if (rr < g.rl) {
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
      const int c = (i * g.lanes + l) * VEC;
      if (c >= cols) break;
      const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
      float sz[VEC] = {}, sx[VEC] = {};
      for (int64_t r = rr; r < rows; r += g.rl * kRowsAhead) {
        const int64_t left = (rows - r + g.rl - 1) / g.rl;
        const int live = left < kRowsAhead ? static_cast<int>(left) : kRowsAhead;
        float v[kRowsAhead][VEC], d[kRowsAhead][VEC];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
          const int64_t at = r + static_cast<int64_t>(u < live ? u : live - 1) * g.rl;
          read_piece<T, VEC>(x + at * ldx, c, cols, v[u]);
          read_piece<T, VEC>(dy + at * ldg, c, cols, d[u]);
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
          if (u >= live) break;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float xh = (v[u][e] - a.m[e]) * a.r[e];
            float value, slope;
            act_both<ACT>(xh * a.w[e] + a.b[e], value, slope);
            const float dz = d[u][e] * slope;
            sz[e] += dz;
            sx[e] += dz * xh;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        lds[rr * wide + c + e] = sz[e];
        lds[(g.rl + rr) * wide + c + e] = sx[e];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += kGroupThreads) {
    float z = 0.0f, q = 0.0f;
    for (int i = 0; i < g.rl; ++i) {
      z += lds[i * wide + c];
      q += lds[(g.rl + i) * wide + c];
    }
    f(c, z, q);
  }
}

// The groups' mean (dz w) and mean (dz w xh) from sums per channel, to s1 and s2
// [groups] of LDS, followed by a barrier.
template <typename Z, typename X>
__device__ __forceinline__ void group_means(int cols, int cpg, const float* w, float inv, Z&& z, X&& q, float* s1,
                                            float* s2) {
  const int groups = cols / cpg, width = group_width(groups);
  const int t = threadIdx.x % width;
  for (int k = threadIdx.x / width; k < groups; k += kGroupThreads / width) {
    float a = 0.0f, b = 0.0f;
    for (int c = t; c < cpg; c += width) {
      const int at = k * cpg + c;
      const float ww = w ? w[at] : 1.0f;
      a += ww * z(at);
      b += ww * q(at);
    }
    for (int o = 1; o < width; o <<= 1) {
      a += __shfl_xor(a, o, 64);
      b += __shfl_xor(b, o, 64);
    }
    if (t == 0) {
      s1[k] = a * inv;
      s2[k] = b * inv;
    }
  }
  __syncthreads();
}

// dx of `rows` rows.
template <typename T, int VEC, int V, int ACT>
__device__ __forceinline__ void chunk_grads(const T* dy, int64_t ldg, const T* x, int64_t ldx, T* dx, int64_t ldd,
                                            int64_t rows, int cols, int cpg, Lanes g, const float* mean,
                                            const float* rstd, const float* w, const float* b, const float* s1,
                                            const float* s2) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  if (rr >= g.rl) return;
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const int c = (i * g.lanes + l) * VEC;
    if (c >= cols) return;
    const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
    float t1[VEC], t2[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int q = c + e < cols ? c + e : cols - 1;
      t1[e] = s1[q / cpg];
      t2[e] = s2[q / cpg];
    }
    for (int64_t r = rr; r < rows; r += g.rl * kRowsAhead) {
      const int64_t left = (rows - r + g.rl - 1) / g.rl;
      const int live = left < kRowsAhead ? static_cast<int>(left) : kRowsAhead;
      float v[kRowsAhead][VEC], d[kRowsAhead][VEC];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const int64_t at = r + static_cast<int64_t>(u < live ? u : live - 1) * g.rl;
        read_piece<T, VEC>(x + at * ldx, c, cols, v[u]);
        read_piece<T, VEC>(dy + at * ldg, c, cols, d[u]);
      }
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        if (u >= live) break;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (v[u][e] - a.m[e]) * a.r[e];
          float value, slope;
          act_both<ACT>(xh * a.w[e] + a.b[e], value, slope);
          v[u][e] = a.r[e] * (d[u][e] * slope * a.w[e] - t1[e] - xh * t2[e]);
        }
        write_piece<T, VEC>(dx + (r + static_cast<int64_t>(u) * g.rl) * ldd, c, cols, v[u]);
      }
    }
  }
}

// partial [slots][2][C]: each chunk's sums of dz and of dz xh.
template <typename T, int VEC, int V>
__global__ __launch_bounds__(kGroupThreads) void k_group_sums(const T* __restrict__ dy, int64_t ldg,
                                                              const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                              int cpg, Lanes g, int shift,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ b, int act,
                                                              float* __restrict__ partial) {
  extern __shared__ float lds[];
  const ItemTile t = find_item(it, 1, shift, blockIdx.x);
  const int64_t r0 = t.tile << shift;
  if (t.item == it.items || t.tile < 0 || r0 >= t.rows) return;
  const int64_t rows = min(t.rows - r0, int64_t{1} << shift), at = t.row0 + r0, G = C / cpg;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * C;
  with_act(act, [&](auto a) {
    chunk_sums<T, VEC, V, decltype(a)::value>(dy + at * ldg, ldg, x + at * ldx, ldx, rows, C, cpg, g,
                                              mean + t.item * G, rstd + t.item * G, w, b, lds,
                                              [&](int c, float z, float q) {
                                                out[c] = z;
                                                out[C + c] = q;
                                              });
  });
}

// Sums of an item's chunks: 16 columns of the 2 C a workgroup, 64 chunks at a
// time. sz and sx [items][C].
constexpr int kJoinThreads = 1024, kJoinCols = 16;
__global__ __launch_bounds__(kJoinThreads) void k_group_join_sums(const float* __restrict__ partial, Items it, int C,
                                                                  int shift, float* __restrict__ sz,
                                                                  float* __restrict__ sx) {
  constexpr int LANES = kJoinThreads / kJoinCols;
  __shared__ float lds[LANES][kJoinCols];
  const int item = blockIdx.y, q = threadIdx.x % kJoinCols, t = threadIdx.x / kJoinCols;
  const int col = blockIdx.x * kJoinCols + q;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1), rows = e > s ? e - s : 0;
  const int64_t slot = (s >> shift) + item, chunks = (rows + (int64_t{1} << shift) - 1) >> shift;
  float sum = 0.0f;
  if (col < 2 * C) {
#pragma unroll 4
    for (int64_t c = t; c < chunks; c += LANES) sum += partial[(slot + c) * 2 * C + col];
  }
  lds[t][q] = sum;
  __syncthreads();
  if (t != 0 || col >= 2 * C) return;
  sum = 0.0f;
  for (int i = 0; i < LANES; ++i) sum += lds[i][q];
  if (col < C) sz[static_cast<int64_t>(item) * C + col] = sum;
  else sx[static_cast<int64_t>(item) * C + col - C] = sum;
}

// dx of a chunk, and in workgroups from `slots` on 256 columns' dw and db, the
// sums over the items.
template <typename T, int VEC, int V>
__global__ __launch_bounds__(kGroupThreads) void k_group_dx(const T* __restrict__ dy, int64_t ldg,
                                                            const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                            int cpg, Lanes g, int shift, int64_t slots,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd,
                                                            const float* __restrict__ w, const float* __restrict__ b,
                                                            int act, const float* __restrict__ sz,
                                                            const float* __restrict__ sx, T* __restrict__ dx,
                                                            float* __restrict__ dw, float* __restrict__ db) {
  extern __shared__ float lds[];
  const int64_t G = C / cpg;
  if (blockIdx.x >= slots) {
    const int64_t c = (blockIdx.x - slots) * kGroupThreads + threadIdx.x;
    if (c >= C) return;
    float a = 0.0f, q = 0.0f;
    for (int64_t i = 0; i < it.items; ++i) {
      a += sz[i * C + c];
      q += sx[i * C + c];
    }
    if (dw) dw[c] = q;
    if (db) db[c] = a;
    return;
  }
  const ItemTile t = find_item(it, 1, shift, blockIdx.x);
  const int64_t r0 = t.tile << shift;
  if (t.tile < 0 || r0 >= t.rows) return;
  const int64_t rows = min(t.rows - r0, int64_t{1} << shift), at = t.row0 + r0;
  if (t.item == it.items) {
    chunk_zeros<T, VEC, V>(dx + at * C, C, rows, C, g);
    return;
  }
  const float* z = sz + static_cast<int64_t>(t.item) * C;
  const float* q = sx + static_cast<int64_t>(t.item) * C;
  group_means(C, cpg, w, 1.0f / (static_cast<float>(t.rows) * static_cast<float>(cpg)), [&](int c) { return z[c]; },
              [&](int c) { return q[c]; }, lds, lds + G);
  with_act(act, [&](auto a) {
    chunk_grads<T, VEC, V, decltype(a)::value>(dy + at * ldg, ldg, x + at * ldx, ldx, dx + at * C, C, rows, C, cpg, g,
                                               mean + t.item * G, rstd + t.item * G, w, b, lds, lds + G);
  });
}

// Few rows: one workgroup for an item's columns of `gpw` groups, sz and sx
// [items][C] to be summed over the items (or dw and db themselves).
template <typename T, int VEC>
__global__ __launch_bounds__(kGroupThreads) void k_group_norm_grad(const T* __restrict__ dy, int64_t ldg,
                                                                   const T* __restrict__ x, int64_t ldx, Items it,
                                                                   int C, int cpg, int gpw, Lanes g,
                                                                   const float* __restrict__ mean,
                                                                   const float* __restrict__ rstd,
                                                                   const float* __restrict__ w,
                                                                   const float* __restrict__ b, int act,
                                                                   T* __restrict__ dx, float* __restrict__ sz,
                                                                   float* __restrict__ sx) {
  extern __shared__ float lds[];
  __shared__ float s1[kGroupThreads], s2[kGroupThreads];
  const int item = blockIdx.x, G = C / cpg, k0 = blockIdx.y * gpw;
  const int groups = min(gpw, G - k0), c0 = k0 * cpg, cols = groups * cpg;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1), rows = e > s ? e - s : 0;
  if (item == it.items) {
    if (dx) chunk_zeros<T, VEC, 1>(dx + s * C + c0, C, rows, cols, g);
    return;
  }
  dy += s * ldg + c0;
  x += s * ldx + c0;
  w = w ? w + c0 : nullptr;
  b = b ? b + c0 : nullptr;
  mean += static_cast<int64_t>(item) * G + k0;
  rstd += static_cast<int64_t>(item) * G + k0;
  float* const z = lds;
  float* const q = lds + g.rl * g.lanes * VEC;
  with_act(act, [&](auto a) {
    chunk_sums<T, VEC, 1, decltype(a)::value>(dy, ldg, x, ldx, rows, cols, cpg, g, mean, rstd, w, b, lds,
                                              [&](int c, float sum_z, float sum_x) {
                                                z[c] = sum_z;  // this thread alone has read the column
                                                q[c] = sum_x;
                                                const int64_t to = static_cast<int64_t>(item) * C + c0 + c;
                                                if (sz) sz[to] = sum_z;
                                                if (sx) sx[to] = sum_x;
                                              });
    if (!dx) return;
    __syncthreads();
    group_means(cols, cpg, w, 1.0f / (static_cast<float>(rows) * static_cast<float>(cpg)),
                [&](int c) { return z[c]; }, [&](int c) { return q[c]; }, s1, s2);
    chunk_grads<T, VEC, 1, decltype(a)::value>(dy, ldg, x, ldx, dx + s * C + c0, C, rows, cols, cpg, g, mean, rstd, w,
                                               b, s1, s2);
  });
}

// ---- dispatch ----

struct GroupShape {
  Items it;
  int C, G, cpg;
};

// Chunks of 2^shift rows, at least 8: between 1024 and 2048 of them over many rows.
int chunk_shift(int64_t n) {
  int shift = 3;
  while ((n >> shift) > 2048) ++shift;
  return shift;
}

// One launch where one workgroup per item and run of groups has little to walk:
// it takes columns of about 128 bytes (whole groups), at most 256 groups.
constexpr int64_t kFewGroupRows = 1024;
bool one_launch(const GroupShape& s, int elem) {
  return s.it.n <= kFewGroupRows && s.cpg * elem <= kGroupThreads * 16;
}
int groups_per_workgroup(const GroupShape& s, int elem) {
  return std::clamp(128 / (s.cpg * elem), 1, std::min(s.G, kGroupThreads));
}

int64_t forward_partial_bytes(const GroupShape& s) {
  return item_slots(s.it, 1, chunk_shift(s.it.n)) * s.G * 8;
}

template <typename T, typename F>
int by_pieces(int C, F&& f) {
  constexpr int VEC = 16 / sizeof(T);
  if (C <= kGroupThreads * VEC) return f(std::integral_constant<int, VEC>{}, std::integral_constant<int, 1>{});
  return f(std::integral_constant<int, VEC>{}, std::integral_constant<int, kGroupChannels / kGroupThreads / VEC>{});
}

template <typename T>
int group_forward(const GroupShape& s, const void* xp, int64_t ldx, const float* w, const float* b, float eps,
                  int act, void* yp, float* mean, float* rstd, Arena& ws, hipStream_t stream) {
  const T* x = static_cast<const T*>(xp);
  T* y = static_cast<T*>(yp);
  if (one_launch(s, sizeof(T))) {
    if (ws.counting) return SUBMCONV_OK;
    constexpr int VEC = 16 / sizeof(T);
    const int gpw = groups_per_workgroup(s, sizeof(T));
    const Lanes g = lanes_of(gpw * s.cpg, VEC);
    const dim3 grid(s.it.items + 1, (s.G + gpw - 1) / gpw);
    k_group_norm<T, VEC><<<grid, kGroupThreads, lanes_lds(g, VEC, 1) * 4, stream>>>(
        x, ldx, s.it, s.C, s.cpg, gpw, g, w, b, eps, act, y, mean, rstd);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  }
  const int shift = chunk_shift(s.it.n);
  const int64_t slots = item_slots(s.it, 1, shift), stats = static_cast<int64_t>(s.it.items) * s.G;
  float2* partial = static_cast<float2*>(ws.take(forward_partial_bytes(s)));
  float* spare = static_cast<float*>(ws.take(2 * stats * 4));
  if (ws.counting) return SUBMCONV_OK;
  if (!mean) mean = spare;
  if (!rstd) rstd = spare + stats;
  return by_pieces<T>(s.C, [&](auto vec, auto v) {
    const Lanes g = lanes_of(s.C, vec);
    k_group_moments<T, vec, v><<<static_cast<unsigned>(slots), kGroupThreads, lanes_lds(g, vec, v) * 4, stream>>>(
        x, ldx, s.it, s.C, s.cpg, g, shift, partial);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    k_group_join<<<static_cast<unsigned>((stats + 3) / 4), kGroupThreads, 0, stream>>>(partial, s.it, s.G, s.cpg,
                                                                                       shift, eps, mean, rstd);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    k_group_apply<T, vec, v><<<static_cast<unsigned>(slots), kGroupThreads, 0, stream>>>(
        x, ldx, s.it, s.C, s.cpg, g, shift, mean, rstd, w, b, act, y);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  });
}

template <typename T>
int group_backward(const GroupShape& s, const void* gp, int64_t ldg, const void* xp, int64_t ldx, const float* mean,
                   const float* rstd, const float* w, const float* b, int act, void* dxp, float* dw, float* db,
                   Arena& ws, hipStream_t stream) {
  const T* dy = static_cast<const T*>(gp);
  const T* x = static_cast<const T*>(xp);
  T* dx = static_cast<T*>(dxp);
  const int64_t sums = static_cast<int64_t>(s.it.items) * s.C;
  const bool one = s.it.items == 1;  // its sums are dw and db
  if (one_launch(s, sizeof(T))) {
    float* spare = one ? nullptr : static_cast<float*>(ws.take(2 * sums * 4));
    if (ws.counting) return SUBMCONV_OK;
    constexpr int VEC = 16 / sizeof(T);
    const int gpw = groups_per_workgroup(s, sizeof(T));
    const Lanes g = lanes_of(gpw * s.cpg, VEC);
    const dim3 grid(s.it.items + 1, (s.G + gpw - 1) / gpw);
    float* sz = one ? db : db ? spare : nullptr;
    float* sx = one ? dw : dw ? spare + sums : nullptr;
    k_group_norm_grad<T, VEC><<<grid, kGroupThreads, lanes_lds(g, VEC, 1) * 4, stream>>>(
        dy, ldg, x, ldx, s.it, s.C, s.cpg, gpw, g, mean, rstd, w, b, act, dx, sz, sx);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    SumList list;
    if (!one && db) list.job[list.count++] = SumJob{sz, s.it.items, s.C, s.C, 1, db};
    if (!one && dw) list.job[list.count++] = SumJob{sx, s.it.items, s.C, s.C, 1, dw};
    return list.count ? run_sums(list, stream) : SUBMCONV_OK;
  }
  const int shift = chunk_shift(s.it.n);
  const int64_t slots = item_slots(s.it, 1, shift);
  float* partial = static_cast<float*>(ws.take(slots * 2 * s.C * 4));
  float* spare = static_cast<float*>(ws.take(2 * sums * 4));
  if (ws.counting) return SUBMCONV_OK;
  float* sz = one && db ? db : spare;
  float* sx = one && dw ? dw : spare + sums;
  return by_pieces<T>(s.C, [&](auto vec, auto v) {
    const Lanes g = lanes_of(s.C, vec);
    k_group_sums<T, vec, v><<<static_cast<unsigned>(slots), kGroupThreads, lanes_lds(g, vec, v) * 4, stream>>>(
        dy, ldg, x, ldx, s.it, s.C, s.cpg, g, shift, mean, rstd, w, b, act, partial);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    const dim3 join((2 * s.C + kJoinCols - 1) / kJoinCols, s.it.items);
    k_group_join_sums<<<join, kJoinThreads, 0, stream>>>(partial, s.it, s.C, shift, sz, sx);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    const int64_t rows = dx ? slots : 0, cols = !one && (dw || db) ? (s.C + kGroupThreads - 1) / kGroupThreads : 0;
    if (rows + cols == 0) return SUBMCONV_OK;
    k_group_dx<T, vec, v><<<static_cast<unsigned>(rows + cols), kGroupThreads, 2 * s.G * 4, stream>>>(
        dy, ldg, x, ldx, s.it, s.C, s.cpg, g, shift, rows, mean, rstd, w, b, act, sz, sx, dx, one ? nullptr : dw,
        one ? nullptr : db);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  });
}

template <typename F>
int by_type(int32_t dtype, F&& f) {
  if (dtype == SUBMCONV_DTYPE_F16) return f(_Float16{});
  if (dtype == SUBMCONV_DTYPE_BF16) return f(__bf16{});
  return f(float{});
}

int check_group(int64_t n, int32_t cdim, int32_t groups, int32_t items, int32_t act, int32_t dtype) {
  if (n < 0 || n > INT32_MAX) return set_error(SUBMCONV_ERR_INVALID_ARG, "n = %lld", (long long)n);
  if (cdim < 1 || cdim > kGroupChannels)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "C = %d, 1 to %d are supported", cdim, kGroupChannels);
  if (groups < 1 || cdim % groups)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d channels in %d groups", cdim, groups);
  if (items < 1 || items > 65535)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items, 1 to 65535 are supported", items);
  if (act < kActNone || act > kActGeluTanh) return set_error(SUBMCONV_ERR_INVALID_ARG, "act = %d", act);
  if (dtype != SUBMCONV_DTYPE_F16 && dtype != SUBMCONV_DTYPE_BF16 && dtype != SUBMCONV_DTYPE_F32)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "dtype = %d", dtype);
  return SUBMCONV_OK;
}

int check_rows(const char* name, const void* p, int64_t n, int32_t cdim, int64_t ld, int32_t dtype) {
  if (n > 0 && !p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (n > 1 && ld < cdim)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: row stride %lld below %d columns", name, (long long)ld, cdim);
  if (reinterpret_cast<uintptr_t>(p) & (dtype == SUBMCONV_DTYPE_F32 ? 3 : 1))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  return SUBMCONV_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int64_t submconv_group_norm_workspace_bytes(int64_t n, int32_t cdim, int32_t groups, int32_t items,
                                                       int32_t dtype) {
  clear_error();
  SUBMCONV_TRY(check_group(n, cdim, groups, items, 0, dtype));
  const GroupShape s{Items{nullptr, items, n}, cdim, groups, cdim / groups};
  Arena ws;
  SUBMCONV_TRY(by_type(dtype, [&](auto t) {
    return group_forward<decltype(t)>(s, nullptr, 0, nullptr, nullptr, 0.0f, 0, nullptr, nullptr, nullptr, ws,
                                      nullptr);
  }));
  return ws.used;
}

extern "C" int submconv_group_norm(const void* x, int64_t ldx, int64_t n, int32_t cdim, int32_t groups,
                                   const int32_t* offsets, int32_t items, const float* weight, const float* bias,
                                   float eps, int32_t act, void* y, float* mean, float* rstd, int32_t dtype,
                                   void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_group(n, cdim, groups, items, act, dtype));
  SUBMCONV_TRY(check_rows("x", x, n, cdim, ldx, dtype));
  SUBMCONV_TRY(check_rows("y", y, n, cdim, cdim, dtype));
  if (!offsets && items != 1) return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items without offsets", items);
  if (!(eps >= 0.0f)) return set_error(SUBMCONV_ERR_INVALID_ARG, "eps = %g", eps);
  if (n == 0 && !mean && !rstd) return SUBMCONV_OK;
  const GroupShape s{Items{offsets, items, n}, cdim, groups, cdim / groups};
  return by_type(dtype, [&](auto t) {
    Arena need, ws{false, static_cast<char*>(workspace)};
    SUBMCONV_TRY(group_forward<decltype(t)>(s, x, ldx, weight, bias, eps, act, y, mean, rstd, need, stream));
    SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, need.used));
    return group_forward<decltype(t)>(s, x, ldx, weight, bias, eps, act, y, mean, rstd, ws, stream);
  });
}

extern "C" int64_t submconv_group_norm_backward_workspace_bytes(int64_t n, int32_t cdim, int32_t groups,
                                                                int32_t items, int32_t dtype) {
  clear_error();
  SUBMCONV_TRY(check_group(n, cdim, groups, items, 0, dtype));
  const GroupShape s{Items{nullptr, items, n}, cdim, groups, cdim / groups};
  Arena ws;
  SUBMCONV_TRY(by_type(dtype, [&](auto t) {
    return group_backward<decltype(t)>(s, nullptr, 0, nullptr, 0, nullptr, nullptr, nullptr, nullptr, 0, nullptr,
                                       nullptr, nullptr, ws, nullptr);
  }));
  return ws.used;
}

extern "C" int submconv_group_norm_backward(const void* grad_out, int64_t ldg, const void* x, int64_t ldx, int64_t n,
                                            int32_t cdim, int32_t groups, const int32_t* offsets, int32_t items,
                                            const float* mean, const float* rstd, const float* weight,
                                            const float* bias, int32_t act, void* grad_x, float* grad_weight,
                                            float* grad_bias, int32_t dtype, void* workspace,
                                            int64_t workspace_bytes, hipStream_t stream) {
  clear_error();
  SUBMCONV_TRY(check_group(n, cdim, groups, items, act, dtype));
  SUBMCONV_TRY(check_rows("grad_out", grad_out, n, cdim, ldg, dtype));
  SUBMCONV_TRY(check_rows("x", x, n, cdim, ldx, dtype));
  SUBMCONV_TRY(check_rows("grad_x", grad_x, grad_x ? n : 0, cdim, cdim, dtype));
  if (!offsets && items != 1) return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items without offsets", items);
  if (!mean || !rstd) return set_error(SUBMCONV_ERR_INVALID_ARG, "mean or rstd is NULL");
  if (!grad_x && !grad_weight && !grad_bias) return SUBMCONV_OK;
  if (n == 0 && !grad_weight && !grad_bias) return SUBMCONV_OK;
  const GroupShape s{Items{offsets, items, n}, cdim, groups, cdim / groups};
  return by_type(dtype, [&](auto t) {
    Arena need, ws{false, static_cast<char*>(workspace)};
    SUBMCONV_TRY(group_backward<decltype(t)>(s, grad_out, ldg, x, ldx, mean, rstd, weight, bias, act, grad_x,
                                             grad_weight, grad_bias, need, stream));
    SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, need.used));
    return group_backward<decltype(t)>(s, grad_out, ldg, x, ldx, mean, rstd, weight, bias, act, grad_x, grad_weight,
                                       grad_bias, ws, stream);
  });
}
