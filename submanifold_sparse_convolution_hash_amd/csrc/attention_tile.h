// What the attention kernels share: 64-row tiles of one head's rows in LDS and
// their two ways into v_mfma_f32_32x32x16 operands.
//
// A tile row is one token's D columns of a head, padded with zeros to DP (32,
// 64, 96 or 128). Loads go straight to LDS, 16 bytes a lane; a buffer's bound
// gives zeros past the item's last row and an offset past every bound gives them
// past column D. A 16-byte piece c of row r sits in slot c ^ swizzle(r) of its
// row, so that both readings spread over all banks: rows of a product with the
// columns as its k (ds_read_b128: 16 rows of one piece), and rows as k, four
// rows of 64 bytes at a time, transposed on the way out (ds_read_b64_tr_b16).
//
// v_mfma_f32_32x32x16, lane = 32 h + c: an operand holds k = 8 h .. 8 h + 7 of
// row (column) c; the result's register i is row 8 (i / 4) + 4 h + i % 4 of
// column c. Registers 0..7 and 8..15 of a result, rounded to 16 bits, are
// therefore at once operands of a next product over those rows, whose k runs 4 h
// .. + 3 and 8 + 4 h .. + 3: the transposed reading gives the other operand in
// that order, and scores never leave the registers.
#pragma once

#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "items.h"
#include "lane_ops.h"

namespace submconv {
namespace {

typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int kTileKeys = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();

template <bool BF16>
__device__ __forceinline__ float16v mfma32(half8 a, half8 b, float16v c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Rows of one head: `ld` elements between tokens.
struct HeadRows {
  const uint16_t* p;  // the item's first row, this head
  int64_t ld, rows;
};

template <int DP>
struct HeadTile {
  static constexpr int ROW = DP <= 32 ? 64 : DP <= 64 ? 128 : 256;  // bytes
  static constexpr int SLOTS = ROW / 16, BYTES = kTileKeys * ROW;
  static __device__ __forceinline__ int swizzle(int r) {
    if constexpr (SLOTS == 16) return (r & 3) << 2 | (r >> 2 & 3);
    else if constexpr (SLOTS == 8) return (r >> 1 & 1) << 2 | (r >> 2 & 3);
    else return r >> 2 & 3;
  }
  // rows r0 + lane % 32, columns 16 kk + 8 (lane / 32) .. + 7
  static __device__ __forceinline__ half8 rows(const char* tile, int r0, int kk, int lane) {
    const int r = r0 + (lane & 31), c = 2 * kk + (lane >> 5);
    return *reinterpret_cast<const half8*>(tile + r * ROW + (c ^ swizzle(r)) * 16);
  }
  // column 32 j + lane % 32, rows r0 + 4 h .. + 3 and r0 + 8 + 4 h .. + 3
  static __device__ __forceinline__ half8 columns(const char* tile, int r0, int j, int lane) {
    const int g = lane >> 4, s = lane & 15;
    const int r = r0 + 4 * (g >> 1) + (s >> 2), c = 4 * j + (g & 1) * 2 + ((s & 3) >> 1);
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4s*)(tile + r * ROW + (c ^ swizzle(r)) * 16 + (s & 1) * 8));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_v4s*)(tile + (r + 8) * ROW + (c ^ swizzle(r + 8)) * 16 + (s & 1) * 8));
    return __builtin_bit_cast(half8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// A workgroup's loads of a tile. D is a multiple of 8.
template <int DP, int NW>
struct TileLoad {
  using H = HeadTile<DP>;
  static constexpr int N = H::BYTES / 1024 / NW;
  static_assert(N * NW * 1024 == H::BYTES, "whole loads");
  uint32_t voff[N];
  __device__ __forceinline__ void init(int64_t ld, int D, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = (i * NW + wave) * 64 + lane, r = s / H::SLOTS, c = (s % H::SLOTS ^ H::swizzle(r)) * 8;
      voff[i] = c < D ? static_cast<uint32_t>(r * ld + c) * 2u : kOobOff;
    }
  }
  // rows row0 .. + 63, zeros past the head's last
  __device__ __forceinline__ void issue(const HeadRows& h, int64_t row0, int D, uint32_t lds, int wave) const {
    const uint32_t left = rows_left(h.rows, row0, kTileKeys);
    rsrc4 r = load_rsrc(h.p + row0 * h.ld, left ? static_cast<uint32_t>((left - 1) * h.ld + D) * 2u : 0u);
    settle_rsrc(r);
#pragma unroll
    for (int i = 0; i < N; ++i) load_to_lds(r, voff[i], lds + (i * NW + wave) * 1024);
  }
};

// Waits for operands that were loaded to registers. Without it the compiler,
// which does not count the loads to LDS, waits for all loads in flight at the
// operands' first use, in every turn of a loop: the next tile's among them.
template <int N>
__device__ __forceinline__ void settle(half8 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

// 4 bytes a lane, as load_to_lds.
__device__ __forceinline__ void load_word_to_lds(rsrc4 r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(r));
}

}  // namespace

// ---- the operator's arguments ----

struct Strided {
  const uint16_t* p;
  int64_t ld, hs;  // elements between tokens and between heads
};

struct Attention {
  Strided q, k, v;
  Items qi, ki;
  const int32_t* k_lengths;  // or null
  int32_t group, kv_heads, D;
  float scale;  // > 0
  int32_t causal;
};

namespace {

// One item's extents, as a workgroup sees them: its first rows, how many it has,
// and how many queries meet how many keys (none among the rows of no item).
struct Extent {
  int64_t q0, k0;
  int32_t q_rows, k_rows, Lq, Lk;
};
// Of the item of a tile of queries, or of keys (of_keys).
__device__ __forceinline__ Extent extent_of(const Attention& a, const ItemTile& t, bool of_keys) {
  const int64_t s = t.row0, n = t.rows;
  int64_t s2 = s, n2 = n;  // the other side's
  if (a.qi.offsets != a.ki.offsets || a.qi.n != a.ki.n) {
    const Items& other = of_keys ? a.qi : a.ki;
    s2 = item_start(other, t.item);
    const int64_t e2 = item_start(other, t.item + 1);
    n2 = e2 > s2 ? e2 - s2 : 0;
  }
  Extent x;
  x.q0 = of_keys ? s2 : s;
  x.k0 = of_keys ? s : s2;
  x.q_rows = x.Lq = static_cast<int32_t>(of_keys ? n2 : n);
  x.k_rows = x.Lk = static_cast<int32_t>(of_keys ? n : n2);
  if (t.item == a.qi.items) x.Lk = 0, x.Lq = 0;
  else if (a.k_lengths) x.Lk = min(x.Lk, max(a.k_lengths[t.item], 0));
  return x;
}

// Rows of a tile, row = token group + head of the group: `count` of them from the
// tile's first on (32-bit divisions but for the first).
struct TileRows {
  int64_t token0;
  uint32_t rest, group;
  int count;
  __device__ __forceinline__ TileRows(int64_t first, int64_t rows, int most, int32_t group_)
      : token0(group_ == 1 ? first : first / group_),
        rest(static_cast<uint32_t>(first - token0 * group_)),
        group(static_cast<uint32_t>(group_)),
        count(static_cast<int>(min(rows - first, static_cast<int64_t>(most)))) {}
  // of the tile's row i, or its last one
  __device__ __forceinline__ int32_t token(int i) const {
    return static_cast<int32_t>(token0) + static_cast<int32_t>((rest + min(i, count - 1)) / group);
  }
  __device__ __forceinline__ int head(int i) const { return static_cast<int>((rest + min(i, count - 1)) % group); }
};

// Number of the item's keys that its token sees.
__device__ __forceinline__ int32_t keys_of(const Attention& a, const Extent& x, int32_t token) {
  if (!a.causal) return x.Lk;
  const int32_t n = token + (x.Lk - x.Lq) + 1;
  return n < 0 ? 0 : n < x.Lk ? n : x.Lk;
}

// Workgroup -> (slot, head): each die's workgroups (every eighth) walk whole
// heads one after the other, so that a head's rows stay in that die's cache;
// the heads that are left are dealt out slot by slot. Slots go from long walks to
// short ones under the causal mask. Where all workgroups start at once, `two` a
// unit, the second half goes backwards: a unit that has a long walk then gets a
// short one beside it (4096 rows, 16 heads of 128: 114 -> 96 us).
//
// `by_slot`, where there are few keys for many queries: a die's workgroups take all
// heads of one slot after the other instead. Every die then reads all keys, but the
// queries' memory lines that two heads share (72 columns are 144 bytes) come from
// its cache: 12347 rows of 10 heads of 72 on 4 x 77 keys, gradient of the rows 34 ->
// 31 us.
struct Place {
  int64_t slot;
  int head;
};
inline bool few_keys(const Attention& a) { return a.qi.n * a.group > 16 * a.ki.n; }
constexpr int64_t kAtOnce = 512;
__device__ __forceinline__ int64_t folded(int64_t i, int64_t n, bool fold) {
  return fold && i >= n / 2 ? n - 1 - (i - n / 2) : i;
}
__device__ __forceinline__ Place place_of(int64_t b, int64_t slots, int heads, bool causal, bool two, bool by_slot) {
  if (by_slot) {
    const int64_t eights = slots / 8 * 8;
    if (b < eights * heads) return Place{b / 8 / heads * 8 + b % 8, static_cast<int>(b / 8 % heads)};
    b -= eights * heads;
    return Place{eights + b / heads, static_cast<int>(b % heads)};
  }
  const int full = heads / 8, rest = heads % 8;
  const bool fold = causal && two && slots * heads <= kAtOnce + 8 * heads;  // (a few slots have no tile)
  if (b < full * 8 * slots) {
    const int64_t i = folded(b / 8, full * slots, fold);
    return Place{i % slots, static_cast<int>(i / slots) * 8 + static_cast<int>(b % 8)};
  }
  const int64_t i = folded(b - full * 8 * slots, rest * slots, fold);
  return Place{i / rest, full * 8 + static_cast<int>(i % rest)};
}

// A workgroup's tile and split, longest walks first: a tile sees the more keys
// the further behind it lies in its item under the causal mask (of_keys: a tile
// of keys is seen by the more queries the further it lies from the item's end).
// Without it all of an item's walks are as long.
struct Walk {
  ItemTile t;
  int split;
};
__device__ __forceinline__ Walk walk_of(const Items& it, int64_t per, int shift, int64_t slots, int splits,
                                        int64_t slot, bool causal, bool of_keys) {
  Walk w;
  if (causal && it.items > 1 && it.items <= kOrderedItems) {
    w.t = find_item_longest(it, per, shift, slot / splits, of_keys);
    w.split = static_cast<int>(slot % splits);
    return w;
  }
  const int64_t s = of_keys ? slot : slots - 1 - slot;
  w.t = find_item(it, per, shift, s / splits);
  w.split = static_cast<int>(s % splits);
  return w;
}

// Registers i and i + 4 .. of a result's rows (4 of them each), rounded: lane c
// then holds rows 8 h' .. 8 h' + 7 of its column, h' = its half.
template <bool BF16>
__device__ __forceinline__ u32x4 eight_rows(float4v a, float4v b) {
  const u32x2 x = pack4<BF16>(a), y = pack4<BF16>(b);
  const u32x2 s = lane_halves_swap(x[0], y[0]), t = lane_halves_swap(x[1], y[1]);
  return u32x4{s[0], t[0], s[1], t[1]};
}

template <bool BF16>
__device__ __forceinline__ half8 operand_of(const float16v& s, int from) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = s[from + e];
  return __builtin_bit_cast(half8, pack8<BF16>(v));
}

__device__ __forceinline__ float halves_max(float x) {
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  const u32x2 p = lane_halves_swap(v, v);
  const uint32_t a = p[0], b = p[1];
  return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}
__device__ __forceinline__ float halves_sum(float x) {
  const uint32_t v = __builtin_bit_cast(uint32_t, x);
  return swap_sum(lane_halves_swap(v, v));
}

}  // namespace

// Into how many runs a walk is split, each to its own fp32 sums, which a last launch
// joins: the least of what walks and joins take, as measured. `tiles` workgroups
// start in start_us and walk up to `steps` steps of step_us each, `seen` of them on
// average (the causal mask), `places` of them at once, which then share their
// units and take `full` times as long: what counts is the longest walk or all of
// them in turn; the sums of one run are written and read at 2.5 TB/s, and the join's launch takes
// 6 us. 300 rows of 8 heads of 64 on 4000 keys: 55 us in one run, 20 in eight; 2048
// rows of 16 heads of 128: 48 in one, 70 in two.
constexpr int kMostSplits = 256;
struct Splits {
  int splits;
  double us;
};
inline Splits splits_of(int64_t tiles, int64_t steps, double start_us, double step_us, double full, double seen,
                        int64_t places, int64_t run_floats) {
  const double join_us = static_cast<double>(run_floats) * 8 / 2.5e6;
  Splits best{1, 0.0};
  for (int s = 1; s <= kMostSplits && (s == 1 || 2 * s <= steps); ++s) {
    const double rounds = static_cast<double>(tiles) * s / static_cast<double>(places);
    const double walk = static_cast<double>((steps + s - 1) / s) * step_us;
    const double us = std::max(start_us + walk, rounds * (start_us + full * seen * walk)) +
                      (s > 1 ? 6.0 + s * join_us : 0.0);
    if (s == 1 || us < best.us) best = Splits{s, us};
  }
  return best;
}

// The share of an item's pairs of rows and keys that are seen, on average.
inline double seen_share(const Attention& a) {
  const double q = static_cast<double>(a.qi.n), k = static_cast<double>(a.ki.n);
  if (!a.causal || q < 1.0 || k < 1.0) return 1.0;
  return k >= q ? 1.0 - 0.5 * q / k : 0.5 * k / q;
}

// Host side of the checks, shared by both directions.
int check_attention(const Attention& a, int64_t nq, int64_t nk, int32_t heads, int32_t dtype);
int check_strided(const char* name, const Strided& s, int64_t n, int32_t heads, int32_t D);

// One row has no stride, and one head neither: they get one of D, by which a
// tile's rows past the last one still fall outside its buffer.
inline Strided strided(const void* p, int64_t n, int32_t heads, int32_t D, int64_t ld, int64_t hs) {
  return Strided{static_cast<const uint16_t*>(p), n > 1 ? ld : D, heads > 1 ? hs : D};
}

}  // namespace submconv
