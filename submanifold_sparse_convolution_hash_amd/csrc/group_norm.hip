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
// the outputs (and joins the chunks itself, where an item has few). A thread keeps
// its 16 bytes of columns for all rows of its chunk, so that sums per channel stay
// in registers. All sums are fp32 and joined in a fixed order: results repeat bit
// for bit. Means and squares about the mean are joined pairwise (n, mean, square
// sum), so that a mean of many deviations costs no digits.
//
// 209715 x 128 in 32 groups, silu: fp16 forward 20 + 5 + 24 us (54 + 0 + 107 MB at
// the memory), bf16 gradients 27 + 5 + 34 (107 + 0 + 161 MB, 3.9 and 4.7 TB/s); 209715
// x 512 fp16 128 and 223 us, 5.0 and 4.8 TB/s, a copy's rate. At 128 channels the
// three launches' starts and ends weigh.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "items.h"
#include "lane_ops.h"

namespace submconv {
namespace {

constexpr int kGroupThreads = 256;
constexpr int kGroupChannels = 8192;
constexpr int kUnits = 256;  // compute units
// rows of a thread in flight, of one tensor or of two
constexpr int kRowsAhead = 8, kGradRowsAhead = 4;

// ---- elements ----

template <typename T>
constexpr int kVec = 16 / sizeof(T);
template <typename T>
using Piece = T __attribute__((ext_vector_type(kVec<T>)));

// Columns c .. c + kVec - 1 of a row, zeros past C, at any element's address.
template <typename T>
__device__ __forceinline__ Piece<T> read_piece(const T* row, int c, int C) {
  typedef T loose __attribute__((ext_vector_type(kVec<T>), aligned(sizeof(T))));
  if (c + kVec<T> <= C) return *reinterpret_cast<const loose*>(row + c);
  Piece<T> v;
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) v[e] = c + e < C ? row[c + e] : static_cast<T>(0.0f);
  return v;
}
template <typename T>
__device__ __forceinline__ void write_piece(T* row, int c, int C, Piece<T> v) {
  typedef T loose __attribute__((ext_vector_type(kVec<T>), aligned(sizeof(T))));
  if (c + kVec<T> <= C) {
    *reinterpret_cast<loose*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
      if (c + e < C) row[c + e] = v[e];
  }
}

// ---- a thread's place: piece l + i lanes (i < strips), row r of `rl` at a time ----

struct Lanes {
  int lanes, rl, strips;  // rl = 256 / lanes where there is one strip, else 1
};
inline Lanes lanes_of(int cols, int vec) {
  const int pieces = (cols + vec - 1) / vec;
  if (pieces <= kGroupThreads) return Lanes{pieces, kGroupThreads / pieces, 1};
  return Lanes{kGroupThreads, 1, (pieces + kGroupThreads - 1) / kGroupThreads};
}
// floats of LDS for two values per channel and row of threads
inline int lanes_lds(const Lanes& g, int vec) { return 2 * g.rl * g.lanes * vec * g.strips; }

// A batch of a thread's rows r, r + rl, ..: `live` of them, a row past the last
// reads the last again.
template <int N>
__device__ __forceinline__ int live_rows(int rows, int r, int rl) {
  return min((rows - r + rl - 1) / rl, N);
}
template <typename T, int N>
__device__ __forceinline__ void read_rows(Piece<T> (&v)[N], const T* x, int64_t ldx, int r, int rl, int live,
                                          int c, int cols) {
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = read_piece<T>(x + (r + min(u, live - 1) * rl) * ldx, c, cols);
}

// Threads that work on one of `count` sums: a power of two up to 64.
__device__ __forceinline__ int sum_width(int count) {
  int w = 1;
  while (w < 64 && 2 * w * count <= kGroupThreads) w <<= 1;
  return w;
}
__device__ __forceinline__ float width_sum(float v, int width) {
  if (width == 64) return lanes_sum<64>(v);
  if (width == 32) return lanes_sum<32>(v);
  if (width == 16) return lanes_sum<16>(v);
  if (width == 8) return lanes_sum<8>(v);
  if (width == 4) return lanes_sum<4>(v);
  return width == 2 ? v + dpp<0xB1>(v) : v;
}

// The mean and the sum of squares about it of `rows` rows of columns 0 .. cols -
// 1 per group, to f(group, mean, squares) in one thread of each. lds as
// lanes_lds. v: the thread's last batch of rows, where there is one strip.
//
// A thread joins a batch to what it has: n, mean and squares about the mean of
// either side give those of both. The threads' parts of a group are then joined
// in two rounds, the mean first and the squares about it, without a division in
// either. Means are summed as differences from one of them, so that equal values
// have their own value as mean and no variance.
template <typename T, typename F>
__device__ __forceinline__ void chunk_moments(const T* x, int64_t ldx, int rows, int cols, int cpg, Lanes g,
                                              float* lds, Piece<T> (&v)[kRowsAhead], F&& f) {
  constexpr int VEC = kVec<T>;
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  const int wide = g.lanes * VEC * g.strips;
  if (rr < g.rl) {
    for (int c = l * VEC; c < cols; c += g.lanes * VEC) {
      float mean[VEC] = {}, m2[VEC] = {}, cnt = 0.0f;
      for (int r = rr; r < rows; r += g.rl * kRowsAhead) {
        const int live = live_rows<kRowsAhead>(rows, r, g.rl);
        read_rows(v, x, ldx, r, g.rl, live, c, cols);
        const float nb = static_cast<float>(live), inv = 1.0f / nb;
        const float w = nb / (cnt + nb), k = cnt * w;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float t[kRowsAhead], s = 0.0f, q = 0.0f;
#pragma unroll
          for (int u = 0; u < kRowsAhead; ++u) {
            t[u] = static_cast<float>(v[u][e]);
            s += u < live ? t[u] - t[0] : 0.0f;
          }
          const float mb = t[0] + s * inv;
#pragma unroll
          for (int u = 0; u < kRowsAhead; ++u) q += u < live ? (t[u] - mb) * (t[u] - mb) : 0.0f;
          const float d = mb - mean[e];
          mean[e] += d * w;
          m2[e] += q + d * d * k;
        }
        cnt += nb;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        lds[rr * wide + c + e] = mean[e];
        lds[(g.rl + rr) * wide + c + e] = m2[e];
      }
    }
  }
  __syncthreads();
  const int groups = cols / cpg, width = sum_width(groups), t = threadIdx.x % width;
  const int base = rows / g.rl, more = rows % g.rl;  // rows of a row of threads
  const float inv = 1.0f / (static_cast<float>(rows) * static_cast<float>(cpg));
  for (int k = threadIdx.x / width; k < groups; k += kGroupThreads / width) {
    auto each = [&](auto&& take) {  // (row of threads i, channel c) of the group, every width-th
      int i = t / cpg, c = t - i * cpg;
      const int di = width / cpg, dc = width - di * cpg;
      if (dc == 0) {  // always the same channel
#pragma unroll 4
        for (; i < g.rl; i += di) take(static_cast<float>(base + (i < more)), i * wide + k * cpg + c);
        return;
      }
      while (i < g.rl) {
        take(static_cast<float>(base + (i < more)), i * wide + k * cpg + c);
        i += di;
        c += dc;
        if (c >= cpg) {
          c -= cpg;
          ++i;
        }
      }
    };
    float s = 0.0f, q = 0.0f;
    const float near = rows ? lds[k * cpg] : 0.0f;
    each([&](float n, int at) { s += n > 0.0f ? n * (lds[at] - near) : 0.0f; });
    const float mean = rows ? near + width_sum(s, width) * inv : 0.0f;
    each([&](float n, int at) {
      const float d = lds[at] - mean;
      q += n > 0.0f ? lds[g.rl * wide + at] + n * (d * d) : 0.0f;
    });
    q = width_sum(q, width);
    if (t == 0) f(k, mean, q);
  }
}

// ---- forward ----

// partial [slots][G] {mean, square sum} of each chunk of `chunk` rows.
template <typename T>
__global__ __launch_bounds__(kGroupThreads) void k_group_moments(const T* __restrict__ x, int64_t ldx, Items it,
                                                                 int C, int cpg, Lanes g, uint32_t chunk,
                                                                 float2* __restrict__ partial) {
  extern __shared__ float lds[];
  const ItemTile t = find_chunk(it, chunk, blockIdx.x);
  const int64_t r0 = t.tile * chunk;
  if (t.item == it.items || t.tile < 0 || r0 >= t.rows) return;
  const int rows = static_cast<int>(min(t.rows - r0, static_cast<int64_t>(chunk))), G = C / cpg;
  Piece<T> v[kRowsAhead];
  chunk_moments<T>(x + (t.row0 + r0) * ldx, ldx, rows, C, cpg, g, lds, v, [&](int k, float mean, float squares) {
    partial[static_cast<int64_t>(blockIdx.x) * G + k] = float2{mean, squares};
  });
}

// NT threads join the chunks of one item and group, as chunk_moments its threads'
// parts: four waves up to kFewItems items, whose chunks they keep in registers,
// else one wave, which reads most items' few chunks once and others' in turn.
constexpr int kChunks = 8 * kUnits + 1, kFewItems = 16;
template <int NT>
__global__ __launch_bounds__(NT) void k_group_join(const float2* __restrict__ partial, Items it, int G,
                                                              int cpg, uint32_t chunk, float eps,
                                                              float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int MOST = NT == 64 ? 1 : (kChunks + NT - 1) / NT;
  __shared__ float sums[2][NT / 64];
  const int item = blockIdx.y, k = blockIdx.x;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1);
  const int64_t rows = e > s ? e - s : 0, slot = static_cast<uint32_t>(s) / chunk + item;
  auto all = [&](float v, float (&to)[NT / 64]) {
    v = lanes_sum<64>(v);
    if constexpr (NT == 64) return v;
    if ((threadIdx.x & 63) == 0) to[threadIdx.x >> 6] = v;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) sum += to[i];
    return sum;
  };
  float2 p[MOST];
  float n[MOST];
  auto read = [&](int64_t first) {
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int64_t c = first + threadIdx.x + i * NT, left = rows - c * chunk;
      n[i] = left > 0 ? static_cast<float>(min(static_cast<int64_t>(chunk), left) * cpg) : 0.0f;
      p[i] = left > 0 ? partial[(slot + c) * G + k] : float2{0.0f, 0.0f};
    }
  };
  const bool once = rows <= static_cast<int64_t>(chunk) * (MOST * NT);
  const float near = rows ? partial[slot * G + k].x : 0.0f;
  float total = 0.0f, q = 0.0f;
  for (int64_t first = 0; first * chunk < rows; first += MOST * NT) {
    read(first);
#pragma unroll
    for (int i = 0; i < MOST; ++i) total += n[i] > 0.0f ? n[i] * (p[i].x - near) : 0.0f;
  }
  const float inv = rows ? 1.0f / (static_cast<float>(rows) * static_cast<float>(cpg)) : 0.0f;
  const float m = near + all(total, sums[0]) * inv;
  for (int64_t first = 0; first * chunk < rows; first += MOST * NT) {
    if (!once) read(first);
#pragma unroll
    for (int i = 0; i < MOST; ++i)
      if (n[i] > 0.0f) q += p[i].y + n[i] * ((p[i].x - m) * (p[i].x - m));
  }
  q = all(q, sums[1]) * inv;
  if (threadIdx.x == 0) {
    const int64_t at = static_cast<int64_t>(item) * G + k;
    mean[at] = m;
    rstd[at] = 1.0f / sqrtf(q + eps);
  }
}

// The same by a workgroup for all groups of one item, from its first chunk's parts
// on, to f(group, mean, variance) in one thread of each. A thread has up to BATCH
// parts in registers, so that all of them are on their way at once; what is more is
// read twice.
template <typename F>
__device__ __forceinline__ void item_moments(const float2* partial, int64_t rows, uint32_t chunk, int G, int cpg,
                                             F&& f) {
  constexpr int BATCH = 4;
  const int width = sum_width(G), t = threadIdx.x % width;
  const int chunks = static_cast<int>(static_cast<uint32_t>(rows + chunk - 1) / chunk);
  const float whole = static_cast<float>(chunk) * static_cast<float>(cpg);
  const float end = static_cast<float>(rows - (chunks - 1) * static_cast<int64_t>(chunk)) * static_cast<float>(cpg);
  const float inv = 1.0f / (static_cast<float>(rows) * static_cast<float>(cpg));
  for (int k = threadIdx.x / width; k < G; k += kGroupThreads / width) {
    float2 p[BATCH];
    auto read = [&](int first) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int c = min(first + i * width, chunks - 1);
        p[i] = partial[static_cast<int64_t>(c) * G + k];
      }
    };
    auto weight = [&](int c) { return c + 1 < chunks ? whole : c < chunks ? end : 0.0f; };
    const float near = partial[k].x;
    float s = 0.0f, q = 0.0f;
    for (int first = t; first < chunks; first += BATCH * width) {
      read(first);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float n = weight(first + i * width);
        s += n > 0.0f ? n * (p[i].x - near) : 0.0f;
      }
    }
    const float mean = near + width_sum(s, width) * inv;
    for (int first = t; first < chunks; first += BATCH * width) {
      if (chunks > BATCH * width) read(first);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float n = weight(first + i * width);
        q += n > 0.0f ? p[i].y + n * ((p[i].x - mean) * (p[i].x - mean)) : 0.0f;
      }
    }
    q = width_sum(q, width);
    if (t == 0) f(k, mean, q * inv);
  }
}

// What a thread's columns are normalised with. mean and rstd of the item.
template <int VEC>
struct Affine {
  float m[VEC], r[VEC], w[VEC], b[VEC];
  __device__ __forceinline__ Affine(const float* mean, const float* rstd, const float* wp, const float* bp, int c,
                                    int C, int cpg) {
    int k = c / cpg, left = cpg - (c - k * cpg);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int q = c + e < C ? c + e : C - 1;
      m[e] = mean[k];
      r[e] = rstd[k];
      w[e] = wp ? wp[q] : 1.0f;
      b[e] = bp ? bp[q] : 0.0f;
      if (--left == 0 && q < C - 1) {
        left = cpg;
        ++k;
      }
    }
  }
};

// y of `rows` rows of columns 0 .. cols - 1. v holds the thread's first batch
// where `have` (one strip).
template <typename T, int ACT>
__device__ __forceinline__ void chunk_outputs(const T* x, int64_t ldx, T* y, int64_t ldy, int rows, int cols, int cpg,
                                              Lanes g, const float* mean, const float* rstd, const float* w,
                                              const float* b, Piece<T> (&v)[kRowsAhead], bool have) {
  constexpr int VEC = kVec<T>;
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  if (rr >= g.rl || rr >= rows) return;
  for (int c = l * VEC; c < cols; c += g.lanes * VEC) {
    int r = rr, live = live_rows<kRowsAhead>(rows, r, g.rl);
    if (!have) read_rows(v, x, ldx, r, g.rl, live, c, cols);  // on their way beside the parameters
    const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = a.r[e] * a.w[e];
    for (;;) {
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        if (u >= live) break;
        Piece<T> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e)  // rounded to nearest even
          out[e] = static_cast<T>(act_value<ACT>((static_cast<float>(v[u][e]) - a.m[e]) * s[e] + a.b[e]));
        write_piece<T>(y + (r + u * g.rl) * ldy, c, cols, out);
      }
      r += g.rl * kRowsAhead;
      if (r >= rows) break;
      live = live_rows<kRowsAhead>(rows, r, g.rl);
      read_rows(v, x, ldx, r, g.rl, live, c, cols);
    }
  }
}

template <typename T>
__device__ __forceinline__ void chunk_zeros(T* y, int64_t ldy, int64_t rows, int cols, Lanes g) {
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  if (rr >= g.rl) return;
  for (int c = l * kVec<T>; c < cols; c += g.lanes * kVec<T>)
    for (int64_t r = rr; r < rows; r += g.rl) write_piece<T>(y + r * ldy, c, cols, Piece<T>{});
}

// The rows from the last on: what the statistics' walk read last is still in the
// caches (209715 x 512 fp16, 215 MB: 131 us in place of 139; x 128: no change).
// JOIN: a workgroup joins its item's chunks itself, while its first rows are on
// their way, and an item's first one also writes mean and rstd where they are
// wanted. Else they are read.
template <typename T, bool JOIN>
__global__ __launch_bounds__(kGroupThreads) void k_group_apply(const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                               int cpg, Lanes g, uint32_t chunk,
                                                               const float2* __restrict__ partial, float eps,
                                                               float* mean, float* rstd, const float* __restrict__ w,
                                                               const float* __restrict__ b, int act,
                                                               T* __restrict__ y) {
  extern __shared__ float lds[];  // [2][G] where JOIN
  const int64_t slot = gridDim.x - 1 - blockIdx.x;
  const ItemTile t = find_chunk(it, chunk, slot);
  const int64_t r0 = t.tile * chunk;
  const int G = C / cpg;
  if (t.tile < 0) return;
  if (r0 >= t.rows) {
    if (JOIN && t.tile == 0 && t.item < it.items)  // no rows
      for (int k = threadIdx.x; k < G; k += kGroupThreads) {
        const int64_t to = static_cast<int64_t>(t.item) * G + k;
        if (mean) mean[to] = 0.0f;
        if (rstd) rstd[to] = 1.0f / sqrtf(eps);
      }
    return;
  }
  const int rows = static_cast<int>(min(t.rows - r0, static_cast<int64_t>(chunk)));
  const int64_t at = t.row0 + r0;
  x += at * ldx;
  y += at * C;
  if (t.item == it.items) {
    chunk_zeros<T>(y, C, rows, C, g);
    return;
  }
  Piece<T> v[kRowsAhead];
  const float *m = mean + static_cast<int64_t>(t.item) * G, *r = rstd + static_cast<int64_t>(t.item) * G;
  bool have = false;
  if constexpr (JOIN) {
    const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
    have = g.strips == 1;
    if (have && rr < g.rl && rr < rows)
      read_rows(v, x, ldx, rr, g.rl, live_rows<kRowsAhead>(rows, rr, g.rl), l * kVec<T>, C);
    auto keep = [&](int k, float group_mean, float variance) {
      const float group_rstd = 1.0f / sqrtf(variance + eps);
      lds[k] = group_mean;
      lds[G + k] = group_rstd;
      const int64_t to = static_cast<int64_t>(t.item) * G + k;
      if (t.tile == 0 && mean) mean[to] = group_mean;
      if (t.tile == 0 && rstd) rstd[to] = group_rstd;
    };
    const float2* p = partial + (slot - t.tile) * G;
    item_moments(p, t.rows, chunk, G, cpg, keep);
    __syncthreads();
    m = lds;
    r = lds + G;
  }
  with_act(act, [&](auto a) {
    chunk_outputs<T, decltype(a)::value>(x, ldx, y, C, rows, C, cpg, g, m, r, w, b, v, have);
  });
}

// All of a few rows in one launch: a workgroup takes one item's columns of
// `gpw` groups. Workgroups of item number `items` clear the rows of no item.
template <typename T>
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
  const int64_t s = item_start(it, item), e = item_start(it, item + 1);
  const int rows = static_cast<int>(e > s ? e - s : 0);
  y += s * C + c0;
  if (item == it.items) {
    chunk_zeros<T>(y, C, rows, cols, g);
    return;
  }
  x += s * ldx + c0;
  Piece<T> v[kRowsAhead];
  chunk_moments<T>(x, ldx, rows, cols, cpg, g, lds, v, [&](int k, float m, float squares) {
    const float r = 1.0f / sqrtf((rows ? squares / (static_cast<float>(rows) * static_cast<float>(cpg)) : 0.0f) + eps);
    gm[k] = m;
    gr[k] = r;
    const int64_t at = static_cast<int64_t>(item) * G + k0 + k;
    if (mean) mean[at] = m;
    if (rstd) rstd[at] = r;
  });
  __syncthreads();
  const bool have = rows <= g.rl * kRowsAhead;  // x is still in the registers
  with_act(act, [&](auto a) {
    chunk_outputs<T, decltype(a)::value>(x, ldx, y, C, rows, cols, cpg, g, gm, gr, w ? w + c0 : nullptr,
                                         b ? b + c0 : nullptr, v, have);
  });
}

// ---- gradients ----

// This chunk's sums of dz and dz xh per channel, to f(channel, sum dz, sum dz
// xh) in one thread of each. v and d as for chunk_moments.
template <typename T, int ACT, typename F>
__device__ __forceinline__ void chunk_sums(const T* dy, int64_t ldg, const T* x, int64_t ldx, int rows, int cols,
                                           int cpg, Lanes g, const float* mean, const float* rstd, const float* w,
                                           const float* b, float* lds, Piece<T> (&v)[kGradRowsAhead],
                                           Piece<T> (&d)[kGradRowsAhead], F&& f) {
  constexpr int VEC = kVec<T>;
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  const int wide = g.lanes * VEC * g.strips;
  if (rr < g.rl) {
    for (int c = l * VEC; c < cols; c += g.lanes * VEC) {
      float sz[VEC] = {}, sx[VEC] = {};
      int r = rr, live = live_rows<kGradRowsAhead>(rows, r, g.rl);
      if (r < rows) {
        read_rows(v, x, ldx, r, g.rl, live, c, cols);  // on their way beside the parameters
        read_rows(d, dy, ldg, r, g.rl, live, c, cols);
      }
      const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
      while (r < rows) {
#pragma unroll
        for (int u = 0; u < kGradRowsAhead; ++u) {
          if (u >= live) break;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float xh = (static_cast<float>(v[u][e]) - a.m[e]) * a.r[e];
            float value, slope;
            act_both<ACT>(xh * a.w[e] + a.b[e], value, slope);
            const float dz = static_cast<float>(d[u][e]) * slope;
            sz[e] += dz;
            sx[e] += dz * xh;
          }
        }
        r += g.rl * kGradRowsAhead;
        if (r >= rows) break;
        live = live_rows<kGradRowsAhead>(rows, r, g.rl);
        read_rows(v, x, ldx, r, g.rl, live, c, cols);
        read_rows(d, dy, ldg, r, g.rl, live, c, cols);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        lds[rr * wide + c + e] = sz[e];
        lds[(g.rl + rr) * wide + c + e] = sx[e];
      }
    }
  }
  __syncthreads();
  const int width = sum_width(cols), t = threadIdx.x % width;
  for (int c = threadIdx.x / width; c < cols; c += kGroupThreads / width) {
    float z = 0.0f, q = 0.0f;
    for (int i = t; i < g.rl; i += width) {
      z += lds[i * wide + c];
      q += lds[(g.rl + i) * wide + c];
    }
    z = width_sum(z, width);
    q = width_sum(q, width);
    if (t == 0) f(c, z, q);
  }
}

// The groups' mean (dz w) and mean (dz w xh) from sums per channel, to s1 and s2
// [groups] of LDS, followed by a barrier.
template <typename Z, typename X>
__device__ __forceinline__ void group_means(int cols, int cpg, const float* w, float inv, Z&& z, X&& q, float* s1,
                                            float* s2) {
  const int groups = cols / cpg, width = sum_width(groups);
  const int t = threadIdx.x % width;
  for (int k = threadIdx.x / width; k < groups; k += kGroupThreads / width) {
    float a = 0.0f, b = 0.0f;
    for (int c = t; c < cpg; c += width) {
      const int at = k * cpg + c;
      const float ww = w ? w[at] : 1.0f;
      a += ww * z(at);
      b += ww * q(at);
    }
    a = width_sum(a, width);
    b = width_sum(b, width);
    if (t == 0) {
      s1[k] = a * inv;
      s2[k] = b * inv;
    }
  }
  __syncthreads();
}

// dx of `rows` rows, with the groups' means s1 and s2 that `means` makes ready.
// v and d as for chunk_outputs.
template <typename T, int ACT, typename M>
__device__ __forceinline__ void chunk_grads(const T* dy, int64_t ldg, const T* x, int64_t ldx, T* dx, int64_t ldd,
                                            int rows, int cols, int cpg, Lanes g, const float* mean,
                                            const float* rstd, const float* w, const float* b, const float* s1,
                                            const float* s2, Piece<T> (&v)[kGradRowsAhead], Piece<T> (&d)[kGradRowsAhead],
                                            bool have, M&& means) {
  constexpr int VEC = kVec<T>;
  const int l = threadIdx.x % g.lanes, rr = threadIdx.x / g.lanes;
  const bool on = rr < g.rl && rr < rows && l * VEC < cols;
  if (on && !have) {  // on their way beside the means
    read_rows(v, x, ldx, rr, g.rl, live_rows<kGradRowsAhead>(rows, rr, g.rl), l * VEC, cols);
    read_rows(d, dy, ldg, rr, g.rl, live_rows<kGradRowsAhead>(rows, rr, g.rl), l * VEC, cols);
  }
  means();
  if (!on) return;
  for (int c = l * VEC; c < cols; c += g.lanes * VEC) {
    int r = rr, live = live_rows<kGradRowsAhead>(rows, r, g.rl);
    if (c != l * VEC) {
      read_rows(v, x, ldx, r, g.rl, live, c, cols);
      read_rows(d, dy, ldg, r, g.rl, live, c, cols);
    }
    const Affine<VEC> a(mean, rstd, w, b, c, cols, cpg);
    float t1[VEC], t2[VEC];
    int k = c / cpg, left = cpg - (c - k * cpg);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      t1[e] = s1[k];
      t2[e] = s2[k];
      if (--left == 0 && c + e < cols - 1) {
        left = cpg;
        ++k;
      }
    }
    for (;;) {
#pragma unroll
      for (int u = 0; u < kGradRowsAhead; ++u) {
        if (u >= live) break;
        Piece<T> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (static_cast<float>(v[u][e]) - a.m[e]) * a.r[e];
          float value, slope;
          act_both<ACT>(xh * a.w[e] + a.b[e], value, slope);
          out[e] = static_cast<T>(a.r[e] * (static_cast<float>(d[u][e]) * slope * a.w[e] - t1[e] - xh * t2[e]));
        }
        write_piece<T>(dx + (r + u * g.rl) * ldd, c, cols, out);
      }
      r += g.rl * kGradRowsAhead;
      if (r >= rows) break;
      live = live_rows<kGradRowsAhead>(rows, r, g.rl);
      read_rows(v, x, ldx, r, g.rl, live, c, cols);
      read_rows(d, dy, ldg, r, g.rl, live, c, cols);
    }
  }
}

// partial [slots][2][C]: each chunk's sums of dz and of dz xh; zeros of a slot
// without rows. groups [slots][2][G], or null: a chunk's sums of dz w and of dz w xh
// over a group's columns.
template <typename T>
__global__ __launch_bounds__(kGroupThreads) void k_group_sums(const T* __restrict__ dy, int64_t ldg,
                                                              const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                              int cpg, Lanes g, uint32_t chunk,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd,
                                                              const float* __restrict__ w,
                                                              const float* __restrict__ b, int act,
                                                              float* __restrict__ partial,
                                                              float* __restrict__ groups) {
  extern __shared__ float lds[];
  const ItemTile t = find_chunk(it, chunk, blockIdx.x);
  const int64_t r0 = t.tile * chunk;
  float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * C;
  if (t.item == it.items || t.tile < 0 || r0 >= t.rows) {
    for (int c = threadIdx.x; c < 2 * C; c += kGroupThreads) out[c] = 0.0f;
    return;
  }
  const int rows = static_cast<int>(min(t.rows - r0, static_cast<int64_t>(chunk)));
  const int64_t at = t.row0 + r0, G = C / cpg;
  float* const sz = lds;
  float* const sx = lds + g.rl * g.lanes * kVec<T> * g.strips;
  with_act(act, [&](auto a) {
    Piece<T> v[kGradRowsAhead], d[kGradRowsAhead];
    chunk_sums<T, decltype(a)::value>(dy + at * ldg, ldg, x + at * ldx, ldx, rows, C, cpg, g, mean + t.item * G,
                                      rstd + t.item * G, w, b, lds, v, d, [&](int c, float z, float q) {
                                        out[c] = z;
                                        out[C + c] = q;
                                        sz[c] = z;  // (its threads alone have read the column)
                                        sx[c] = q;
                                      });
  });
  if (!groups) return;
  __syncthreads();
  groups += static_cast<int64_t>(blockIdx.x) * 2 * G;
  group_means(C, cpg, w, 1.0f, [&](int c) { return sz[c]; }, [&](int c) { return sx[c]; }, groups, groups + G);
}

// Sums of an item's chunks: 16 columns of the 2 C a workgroup, NT / 16 chunks at a
// time. sz and sx [items][C].
constexpr int kJoinCols = 16;
template <int NT>
__global__ __launch_bounds__(NT) void k_group_join_sums(const float* __restrict__ partial, Items it, int C,
                                                                  uint32_t chunk, float* __restrict__ sz,
                                                                  float* __restrict__ sx) {
  constexpr int LANES = NT / kJoinCols;
  __shared__ float lds[LANES][kJoinCols];
  const int item = blockIdx.y, q = threadIdx.x % kJoinCols, t = threadIdx.x / kJoinCols;
  const int col = blockIdx.x * kJoinCols + q;
  const int64_t s = item_start(it, item), e = item_start(it, item + 1), rows = e > s ? e - s : 0;
  const int64_t slot = static_cast<uint32_t>(s) / chunk + item;
  const int64_t chunks = static_cast<uint32_t>(rows + chunk - 1) / chunk;
  float sum = 0.0f;
  if (col < 2 * C) {
#pragma unroll 8
    for (int64_t c = t; c < chunks; c += LANES) sum += partial[(slot + c) * 2 * C + col];
  }
  lds[t][q] = sum;
  __syncthreads();
  if (t != 0 || col >= 2 * C) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < LANES; ++i) sum += lds[i][q];
  if (col < C) sz[static_cast<int64_t>(item) * C + col] = sum;
  else sx[static_cast<int64_t>(item) * C + col - C] = sum;
}

// dx of a chunk, the chunks from the last on (see k_group_apply). The first `sums`
// workgroups have columns of dw and db (a launch of their own would take 4 us):
// where JOIN 16 of the 2 C columns each, over all slots, else 256 each, over a few
// items. JOIN: a workgroup joins its item's chunks itself, from their groups' sums,
// while its first rows are on their way; else sz and sx [items][C] are read.
template <typename T, bool JOIN>
__global__ __launch_bounds__(kGroupThreads) void k_group_dx(const T* __restrict__ dy, int64_t ldg,
                                                            const T* __restrict__ x, int64_t ldx, Items it, int C,
                                                            int cpg, Lanes g, uint32_t chunk, int sums,
                                                            int64_t slots, const float* __restrict__ mean,
                                                            const float* __restrict__ rstd,
                                                            const float* __restrict__ w, const float* __restrict__ b,
                                                            int act, const float* __restrict__ sz,
                                                            const float* __restrict__ sx,
                                                            const float* __restrict__ partial,
                                                            const float* __restrict__ groups, T* __restrict__ dx,
                                                            float* __restrict__ dw, float* __restrict__ db) {
  extern __shared__ float lds[];
  const int G = C / cpg;
  if (blockIdx.x < sums) {
    if constexpr (JOIN) {
      constexpr int LANES = kGroupThreads / kJoinCols;
      __shared__ float part[LANES][kJoinCols];
      const int q = threadIdx.x % kJoinCols, t = threadIdx.x / kJoinCols;
      const int col = blockIdx.x * kJoinCols + q;
      float sum = 0.0f;
      if (col < 2 * C) {
#pragma unroll 16
        for (int64_t i = t; i < slots; i += LANES) sum += partial[i * 2 * C + col];
      }
      part[t][q] = sum;
      __syncthreads();
      if (t != 0 || col >= 2 * C) return;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < LANES; ++i) sum += part[i][q];
      if (col < C && db) db[col] = sum;
      if (col >= C && dw) dw[col - C] = sum;
    } else {
      const int c = blockIdx.x * kGroupThreads + threadIdx.x;
      if (c >= C) return;
      float z = 0.0f, q = 0.0f;
#pragma unroll 8
      for (int64_t i = 0; i < it.items; ++i) {
        z += sz[i * C + c];
        q += sx[i * C + c];
      }
      if (dw) dw[c] = q;
      if (db) db[c] = z;
    }
    return;
  }
  const int64_t slot = gridDim.x - 1 - blockIdx.x;
  const ItemTile t = find_chunk(it, chunk, slot);
  const int64_t r0 = t.tile * chunk;
  if (t.tile < 0 || r0 >= t.rows) return;
  const int rows = static_cast<int>(min(t.rows - r0, static_cast<int64_t>(chunk)));
  const int64_t at = t.row0 + r0, stats = static_cast<int64_t>(t.item) * G;
  if (t.item == it.items) {
    chunk_zeros<T>(dx + at * C, C, rows, C, g);
    return;
  }
  const float inv = 1.0f / (static_cast<float>(t.rows) * static_cast<float>(cpg));
  with_act(act, [&](auto a) {
    Piece<T> v[kGradRowsAhead], d[kGradRowsAhead];
    chunk_grads<T, decltype(a)::value>(
        dy + at * ldg, ldg, x + at * ldx, ldx, dx + at * C, C, rows, C, cpg, g, mean + stats, rstd + stats, w, b, lds,
        lds + G, v, d, false, [&] {
          if constexpr (JOIN) {
            const float* p = groups + (slot - t.tile) * 2 * G;
            const int chunks = static_cast<int>(static_cast<uint32_t>(t.rows + chunk - 1) / chunk);
            const int width = sum_width(2 * G), l = threadIdx.x % width;
            for (int k = threadIdx.x / width; k < 2 * G; k += kGroupThreads / width) {
              float sum = 0.0f;
#pragma unroll 16
              for (int c = l; c < chunks; c += width) sum += p[static_cast<int64_t>(c) * 2 * G + k];
              sum = width_sum(sum, width);
              if (l == 0) lds[k] = sum * inv;
            }
            __syncthreads();
          } else {
            const float* z = sz + static_cast<int64_t>(t.item) * C;
            const float* q = sx + static_cast<int64_t>(t.item) * C;
            group_means(C, cpg, w, inv, [&](int c) { return z[c]; }, [&](int c) { return q[c]; }, lds, lds + G);
          }
        });
  });
}

// Few rows: one workgroup for an item's columns of `gpw` groups, sz and sx
// [items][C] to be summed over the items (or dw and db themselves).
template <typename T>
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
  const int64_t s = item_start(it, item), e = item_start(it, item + 1);
  const int rows = static_cast<int>(e > s ? e - s : 0);
  if (item == it.items) {
    if (dx) chunk_zeros<T>(dx + s * C + c0, C, rows, cols, g);
    return;
  }
  dy += s * ldg + c0;
  x += s * ldx + c0;
  w = w ? w + c0 : nullptr;
  b = b ? b + c0 : nullptr;
  mean += static_cast<int64_t>(item) * G + k0;
  rstd += static_cast<int64_t>(item) * G + k0;
  float* const z = lds;
  float* const q = lds + g.rl * g.lanes * kVec<T>;
  const bool have = rows <= g.rl * kGradRowsAhead;  // x and dy are still in the registers
  with_act(act, [&](auto a) {
    Piece<T> v[kGradRowsAhead], d[kGradRowsAhead];
    chunk_sums<T, decltype(a)::value>(dy, ldg, x, ldx, rows, cols, cpg, g, mean, rstd, w, b, lds, v, d,
                                      [&](int c, float sum_z, float sum_x) {
                                        z[c] = sum_z;  // (its threads alone have read the column)
                                        q[c] = sum_x;
                                        const int64_t to = static_cast<int64_t>(item) * C + c0 + c;
                                        if (sz) sz[to] = sum_z;
                                        if (sx) sx[to] = sum_x;
                                      });
    if (!dx) return;
    __syncthreads();
    chunk_grads<T, decltype(a)::value>(
        dy, ldg, x, ldx, dx + s * C + c0, C, rows, cols, cpg, g, mean, rstd, w, b, s1, s2, v, d, have, [&] {
          group_means(cols, cpg, w, 1.0f / (static_cast<float>(rows) * static_cast<float>(cpg)),
                      [&](int c) { return z[c]; }, [&](int c) { return q[c]; }, s1, s2);
        });
  });
}

// ---- dispatch ----

struct GroupShape {
  Items it;
  int C, G, cpg;
};

// Rows of a chunk: two batches a thread, as long as that makes whole rounds of a
// workgroup a unit, one to four of them (three for the gradients): each start costs
// more than two batches do. 100000 x 96 fp16, forward / backward us: 256 chunks 28 /
// 37, 768 27 / 36, 1024 30 / 45, 2048 45 / 57; 209715 x 128: 256 48 / 70, 512 45 / 63,
// 768 45 / 64, 1024 43 / 69, 2048 51 / 83. Where the walk is more than the 256 MB that
// the second one finds in the caches, eight rounds: 209715 x 1024, 1024 chunks 278 /
// 465, 2048 262 / 428. At least a row for each row of threads.
uint32_t chunk_rows(const GroupShape& s, int elem, const Lanes& g, bool grad) {
  const int64_t n = s.it.n, two = std::max(1, 2 * kRowsAhead * g.rl / g.strips), round = two * kUnits;
  const bool cached = n * s.C * elem * (grad ? 2 : 1) <= int64_t{256} << 20;
  // (the last chunk of an item is a part of one: they fit into the rounds as well; 100000 x
  // 96 of 70 items 37 / 51 without, 30 / 42 with)
  const int64_t chunks = kUnits * std::clamp<int64_t>((n + round / 2) / round, 1, !cached ? 8 : grad ? 3 : 4) -
                         (s.it.items < kUnits / 2 ? s.it.items + 1 : 0);
  return static_cast<uint32_t>(std::max<int64_t>(std::max(8, g.rl), (n + chunks - 1) / chunks));
}

// Whether the workgroups of the outputs join their item's chunks themselves, in place
// of a launch of 5 us: where an item has few on average, and would not have too many
// had one item nearly all rows. Each workgroup reads 8 bytes a chunk and group, most of
// it from another die's cache. Forward / backward us, three launches -> two, for the parts
// (chunks times groups) of an item on average and of all items:
//   20011 x 60 in 12 groups of 7 items, 276 and 1900: 16 / 21 -> 13 / 18; 100000 x 96 in
//   32 of 100 items, 80 and 4960: 34 / 51 -> 30 / 45; one item, 100000 x 32 in 8, 2000:
//   17.4 / 21.0 -> 17.7 / 19.7, 1000 x 256 in 32, 4000: 16.0 / 20.6 -> 16.6 / 18.5, 20000 x
//   320 in 32, 6700: 23 / 33 -> 25 / 35.
//   16 items, equal ones and one with nearly all rows: 50000 x 96 in 32, 7650: 21.7 / 27.0
//   -> 18.8 / 25.1 and 21.5 / 28.1 -> 24.5 / 29.1; 100000 x 128 in 32, 15800: 30.8 / 43.2 ->
//   27.8 / 42.7 and 30.9 / 45.5 -> 46.5 / 48.5; 100000 x 320 in 32, 24000: backward 73 -> 74
//   and 75 -> 83; of 100 items, 29400: forward 53 -> 58 and 61 -> 131.
bool joins_itself(const GroupShape& s, uint32_t chunk, bool grad) {
  const int64_t chunks = s.it.n / chunk;
  return (chunks / s.it.items + 1) * s.G <= (grad ? 4096 : 1024) && (chunks + 1) * s.G <= (grad ? 16384 : 8192);
}

// A workgroup of the one-launch kernels takes columns of about 128 bytes, whole
// groups, at most 256 of them.
int groups_per_workgroup(const GroupShape& s, int elem) {
  return std::clamp(128 / (s.cpg * elem), 1, std::min(s.G, kGroupThreads));
}
// One launch where a workgroup has at most 64 KB to walk, should one item have
// all rows. One launch against three, fp16 with silu, forward / backward us: 256
// channels in 32 groups, 64 rows 8.3 / 12.3 against 16 / 20, 256 rows 9.7 / 13.9
// against 16 / 20, 512 rows (64 KB) 13.6 / 20.5 against 16 / 20, 1000 rows 21 / 33
// against 15 / 20; one group of 256, 64 rows (32 KB) 29 / 15 against 17 / 21, 256
// rows 24 / 35 against 17 / 20.
constexpr int64_t kFewGroupBytes = 65536;
bool one_launch(const GroupShape& s, int elem) {
  const int64_t row = static_cast<int64_t>(groups_per_workgroup(s, elem)) * s.cpg * elem;
  return s.it.n * row <= kFewGroupBytes && row <= kGroupThreads * 16;
}

template <typename T>
int group_forward(const GroupShape& s, const void* xp, int64_t ldx, const float* w, const float* b, float eps,
                  int act, void* yp, float* mean, float* rstd, Arena& ws, hipStream_t stream) {
  const T* x = static_cast<const T*>(xp);
  T* y = static_cast<T*>(yp);
  if (one_launch(s, sizeof(T))) {
    if (ws.counting) return SUBMCONV_OK;
    const int gpw = groups_per_workgroup(s, sizeof(T));
    const Lanes g = lanes_of(gpw * s.cpg, kVec<T>);
    const dim3 grid(s.it.items + 1, (s.G + gpw - 1) / gpw);
    k_group_norm<T><<<grid, kGroupThreads, lanes_lds(g, kVec<T>) * 4, stream>>>(
        x, ldx, s.it, s.C, s.cpg, gpw, g, w, b, eps, act, y, mean, rstd);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  }
  const Lanes g = lanes_of(s.C, kVec<T>);
  const uint32_t chunk = chunk_rows(s, sizeof(T), g, false);
  const int64_t slots = chunk_slots(s.it, chunk), stats = static_cast<int64_t>(s.it.items) * s.G;
  const bool join = joins_itself(s, chunk, false);
  float2* partial = static_cast<float2*>(ws.take(slots * s.G * 8));
  float* spare = join ? nullptr : static_cast<float*>(ws.take(2 * stats * 4));
  if (ws.counting) return SUBMCONV_OK;
  const unsigned grid = static_cast<unsigned>(slots);
  k_group_moments<T><<<grid, kGroupThreads, lanes_lds(g, kVec<T>) * 4, stream>>>(x, ldx, s.it, s.C, s.cpg, g, chunk,
                                                                                 partial);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  if (join) {
    k_group_apply<T, true><<<grid, kGroupThreads, 2 * s.G * 4, stream>>>(x, ldx, s.it, s.C, s.cpg, g, chunk, partial,
                                                                         eps, mean, rstd, w, b, act, y);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return SUBMCONV_OK;
  }
  if (!mean) mean = spare;
  if (!rstd) rstd = spare + stats;
  const dim3 of(s.G, s.it.items);
  if (s.it.items <= kFewItems) k_group_join<256><<<of, 256, 0, stream>>>(partial, s.it, s.G, s.cpg, chunk, eps, mean, rstd);
  else k_group_join<64><<<of, 64, 0, stream>>>(partial, s.it, s.G, s.cpg, chunk, eps, mean, rstd);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  k_group_apply<T, false><<<grid, kGroupThreads, 0, stream>>>(x, ldx, s.it, s.C, s.cpg, g, chunk, nullptr, eps, mean,
                                                              rstd, w, b, act, y);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

// dw and db from `parts` sums of each column, ld apart.
int sum_parts(const GroupShape& s, int64_t parts, int64_t ld, const float* sz, const float* sx, float* dw, float* db,
              hipStream_t stream) {
  SumList list;
  if (db) list.job[list.count++] = SumJob{sz, parts, ld, s.C, 1, db};
  if (dw) list.job[list.count++] = SumJob{sx, parts, ld, s.C, 1, dw};
  return list.count ? run_sums(list, stream) : SUBMCONV_OK;
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
    const int gpw = groups_per_workgroup(s, sizeof(T));
    const Lanes g = lanes_of(gpw * s.cpg, kVec<T>);
    const dim3 grid(s.it.items + 1, (s.G + gpw - 1) / gpw);
    float* sz = one ? db : db ? spare : nullptr;
    float* sx = one ? dw : dw ? spare + sums : nullptr;
    k_group_norm_grad<T><<<grid, kGroupThreads, lanes_lds(g, kVec<T>) * 4, stream>>>(
        dy, ldg, x, ldx, s.it, s.C, s.cpg, gpw, g, mean, rstd, w, b, act, dx, sz, sx);
    SUBMCONV_HIP_CHECK(hipGetLastError());
    return one ? SUBMCONV_OK : sum_parts(s, s.it.items, s.C, sz, sx, dw, db, stream);
  }
  const Lanes g = lanes_of(s.C, kVec<T>);
  const uint32_t chunk = chunk_rows(s, sizeof(T), g, true);
  const int64_t slots = chunk_slots(s.it, chunk);
  const bool join = joins_itself(s, chunk, true);
  float* partial = static_cast<float*>(ws.take(slots * 2 * s.C * 4));
  float* groups = join ? static_cast<float*>(ws.take(slots * 2 * s.G * 4)) : nullptr;
  float* spare = join ? nullptr : static_cast<float*>(ws.take(2 * sums * 4));
  if (ws.counting) return SUBMCONV_OK;
  k_group_sums<T><<<static_cast<unsigned>(slots), kGroupThreads, lanes_lds(g, kVec<T>) * 4, stream>>>(
      dy, ldg, x, ldx, s.it, s.C, s.cpg, g, chunk, mean, rstd, w, b, act, partial, dx ? groups : nullptr);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  const int64_t tiles = dx ? slots : 0;
  if (join) {
    const bool here = (dw || db) && slots <= kChunks + kFewItems;  // the sums over the slots
    const int extra = here ? (2 * s.C + kJoinCols - 1) / kJoinCols : 0;
    if (tiles + extra > 0) {
      k_group_dx<T, true><<<static_cast<unsigned>(tiles + extra), kGroupThreads, 2 * s.G * 4, stream>>>(
          dy, ldg, x, ldx, s.it, s.C, s.cpg, g, chunk, extra, slots, mean, rstd, w, b, act, nullptr, nullptr, partial,
          groups, dx, dw, db);
      SUBMCONV_HIP_CHECK(hipGetLastError());
    }
    return here ? SUBMCONV_OK : sum_parts(s, slots, 2 * s.C, partial, partial + s.C, dw, db, stream);
  }
  float* sz = one && db ? db : spare;
  float* sx = one && dw ? dw : spare + sums;
  const dim3 of((2 * s.C + kJoinCols - 1) / kJoinCols, s.it.items);
  if (s.it.items <= kFewItems) k_group_join_sums<1024><<<of, 1024, 0, stream>>>(partial, s.it, s.C, chunk, sz, sx);
  else k_group_join_sums<128><<<of, 128, 0, stream>>>(partial, s.it, s.C, chunk, sz, sx);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  const bool here = !one && s.it.items <= kFewItems && (dw || db);  // the sums over the items
  const int extra = here ? (s.C + kGroupThreads - 1) / kGroupThreads : 0;
  if (tiles + extra > 0) {
    k_group_dx<T, false><<<static_cast<unsigned>(tiles + extra), kGroupThreads, 2 * s.G * 4, stream>>>(
        dy, ldg, x, ldx, s.it, s.C, s.cpg, g, chunk, extra, slots, mean, rstd, w, b, act, sz, sx, nullptr, nullptr, dx,
        dw, db);
    SUBMCONV_HIP_CHECK(hipGetLastError());
  }
  return one || here ? SUBMCONV_OK : sum_parts(s, s.it.items, s.C, sz, sx, dw, db, stream);
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
