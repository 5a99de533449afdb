// Gradients of attention among the rows of packed items. With p_ij = exp(scale
// q_i . k_j - lse_i) as the forward's weights, again formed from q, k and lse:
//
//   dp_ij = do_i . v_j,  delta_i = do_i . o_i = sum_j p_ij dp_ij
//   ds_ij = p_ij (dp_ij - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// Two kernels, each of which owns its rows of the results, so that nothing is
// added by atomics and results repeat bit for bit; the price is that p and dp are
// formed twice, 14 D flops a pair of row and key instead of 10. k_attention_dq
// is the forward's shape: a wave owns 32 rows, scores^T = K Q^T and dp^T = V dO^T,
// and ds^T is at once the operand of dq^T = K^T ds^T. k_attention_dkv owns 32 keys
// a wave: scores = Q K^T, dp = dO V^T, and p and ds are at once the operands of
// dv^T = dO^T p and dk^T = Q^T ds. Both read a tile's rows as they are and
// transposed.
//
// 16384 causal rows of four items, 16 / 4 heads of 128 bf16: 421 and 740-760 us, 1.05
// PFLOP in all; 8192 rows of 8 heads of 128 bf16 890-910 us for both, 1.05 PFLOP/s
// executed, 85 % of what a library product reaches under the same power limit.
//
// p and ds are rounded to 16 bits for the second products. In fp16 small ones
// would be lost below 2^-14: p is taken times 2^12 (it is at most 1), and ds
// times a power of two per column of the result, which is lowered, and what was
// summed with it, when a ds comes near the largest number (Range).
#include <algorithm>

#include "attention_tile.h"

namespace submconv {
namespace {

struct AttnGrad {
  Strided dout;
  const uint16_t* out;  // [nq][heads][D]
  const float* lse;     // [nq][heads]
  float* row_base;      // [heads][nq], written by k_attention_dq: the weights are exp2(score log2(e) + base)
  float* row_delta;     // [heads][nq]
  uint16_t *dq, *dk, *dv;
  float *dq_part, *dk_part, *dv_part;  // [splits][rows][D] where split
  int32_t splits;
  int64_t slots;  // tiles, times the splits
  bool by_slot;   // see place_of
};

// Power of two that a column's ds are taken times.
template <bool BF16>
struct Range {
  static constexpr float kP = BF16 ? 1.0f : 4096.0f, kPLog2 = BF16 ? 0.0f : 12.0f;  // of p
  float g = 0x1p100f;
  // Scales 16 ds of this lane's column; acc are what was summed at the old g.
  template <int DB>
  __device__ __forceinline__ void take(float16v& ds, float16v (&acc)[DB]) {
    if constexpr (!BF16) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(ds[i]));
      top = halves_max(top);
      const bool lower = top * g > 16384.0f;
      if (__ballot(lower)) {
        // to 2^8 at most (an infinite one stays infinite)
        const float next = lower ? __builtin_amdgcn_ldexpf(1.0f, 8 - __builtin_amdgcn_frexp_expf(top)) : g;
        const float f = next / g;
        g = next;
#pragma unroll
        for (int j = 0; j < DB; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j][i] *= f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] *= g;
    }
  }
  __device__ __forceinline__ float back() const { return BF16 ? 1.0f : 1.0f / (g * kP); }
};

// Stores a result^T [D][32 columns] times f: lane c of 32 has column c. `row` is
// the column's row of the tensor.
template <bool BF16, int DB>
__device__ __forceinline__ void store_columns(const float16v (&acc)[DB], float f, uint16_t* out, float* part,
                                              int64_t row, int D, int h) {
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      float4v u, w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = acc[j][i + e] * f;
        w[e] = acc[j][i + 4 + e] * f;
      }
      const int d = j * 32 + i * 2;
      if (part) {
        if (d + h * 4 < D) *reinterpret_cast<float4v*>(part + row * D + d + h * 4) = u;
        if (d + 8 + h * 4 < D) *reinterpret_cast<float4v*>(part + row * D + d + 8 + h * 4) = w;
      } else {
        const u32x4 v = eight_rows<BF16>(u, w);
        if (d + h * 8 < D) *reinterpret_cast<u32x4*>(out + row * D + d + h * 8) = v;
      }
    }
}

template <bool BF16, int DP>
__global__ __launch_bounds__(256, 2) void k_attention_dq(Attention a, AttnGrad o) {
  constexpr int NW = 4, T = 32 * NW, SHIFT = 7;
  static_assert(T == 1 << SHIFT, "rows");
  using H = HeadTile<DP>;
  using L = TileLoad<DP, NW>;
  constexpr int KS = DP / 16, DB = DP / 32;
  __shared__ __attribute__((aligned(16))) char smem[2][2][H::BYTES];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Place at = place_of(blockIdx.x, o.slots, a.kv_heads, a.causal, true, o.by_slot);
  const Walk w = walk_of(a.qi, a.group, SHIFT, o.slots, o.splits, at.slot, a.causal, false);
  const ItemTile t = w.t;
  const int split = w.split;
  const Extent x = extent_of(a, t, false);
  const int64_t rows = static_cast<int64_t>(x.q_rows) * a.group, r_first = t.tile * T;
  if (t.tile < 0 || r_first >= rows) return;

  const TileRows at_row(r_first, rows, T, a.group);
  const int i = wave * 32 + (lane & 31);
  const bool live = i < at_row.count;
  const int32_t token = at_row.token(i);
  const int head = at.head * a.group + at_row.head(i);
  const int32_t see = keys_of(a, x, token);
  const int32_t see_least = keys_of(a, x, at_row.token(wave * 32));  // of the wave's rows: the first's
  const int32_t see_wave = keys_of(a, x, at_row.token(wave * 32 + 31));
  const int32_t see_most = keys_of(a, x, at_row.token(T - 1));
  const int tiles = o.dq || o.dq_part ? (see_most + kTileKeys - 1) / kTileKeys : 0;
  const int first = static_cast<int>(static_cast<int64_t>(tiles) * split / o.splits);
  const int last = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / o.splits);
  const int64_t heads = static_cast<int64_t>(a.kv_heads) * a.group, row = (x.q0 + token) * heads + head;

  const HeadRows kr{a.k.p + x.k0 * a.k.ld + at.head * a.k.hs, a.k.ld, x.Lk};
  const HeadRows vr{a.v.p + x.k0 * a.v.ld + at.head * a.v.hs, a.v.ld, x.Lk};
  L lk, lv;
  lk.init(a.k.ld, a.D, wave, lane);
  lv.init(a.v.ld, a.D, wave, lane);
  const uint32_t lds = lds_addr(&smem[0][0][0]);
  auto issue = [&](int tile) {
    const uint32_t to = lds + (tile & 1) * 2 * H::BYTES;
    lk.issue(kr, static_cast<int64_t>(tile) * kTileKeys, a.D, to, wave);
    lv.issue(vr, static_cast<int64_t>(tile) * kTileKeys, a.D, to + H::BYTES, wave);
  };
  if (first < last) issue(first);  // on its way beside the rows' operands
  half8 q[KS], dy[KS];
  float delta = 0.0f;
  {
    const uint16_t* pq = a.q.p + (x.q0 + token) * a.q.ld + head * a.q.hs;
    const uint16_t* pd = o.dout.p + (x.q0 + token) * o.dout.ld + head * o.dout.hs;
    const uint16_t* po = o.out + row * a.D;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int c = kk * 16 + h * 8;
      q[kk] = dy[kk] = half8{};
      if (c < a.D) {
        q[kk] = *reinterpret_cast<const half8*>(pq + c);
        dy[kk] = *reinterpret_cast<const half8*>(pd + c);
        float u[8], w[8];
        unpack8<BF16>(__builtin_bit_cast(u32x4, dy[kk]), u);
        unpack8<BF16>(*reinterpret_cast<const u32x4*>(po + c), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta += u[e] * w[e];
      }
    }
    delta = halves_sum(delta);
  }
  float base = Range<BF16>::kPLog2 - o.lse[row] * kLog2e;
  if (live && h == 0 && split == 0) {
    o.row_base[head * a.qi.n + x.q0 + token] = base;
    o.row_delta[head * a.qi.n + x.q0 + token] = delta;
  }
  if (!o.dq && !o.dq_part) return;  // (then there is no tile to wait for either)
  settle(q);
  settle(dy);
  const float c = a.scale * kLog2e;
  asm volatile("" : "+v"(base), "+v"(delta));
  Range<BF16> range;
  float16v acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j) acc[j] = float16v{};
  for (int tile = first; tile < last; ++tile) {
    // this tile has landed and all waves are past the last one
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (tile + 1 < last) issue(tile + 1);
    const char* tk = smem[tile & 1][0];
    const char* tv = smem[tile & 1][1];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int j0 = tile * kTileKeys + b * 32;
      if (j0 >= see_wave) break;  // no row of this wave sees the block
      float16v s = {}, dp = {};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        s = mfma32<BF16>(H::rows(tk, b * 32, kk, lane), q[kk], s);
        dp = mfma32<BF16>(H::rows(tv, b * 32, kk, lane), dy[kk], dp);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(s[i] * c + base) * (dp[i] - delta);
      if (j0 + 32 > see_least) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + 8 * (i / 4) + 4 * h + i % 4 >= see) s[i] = 0.0f;
      }
      range.take(s, acc);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const half8 ds = operand_of<BF16>(s, 8 * k);
#pragma unroll
        for (int j = 0; j < DB; ++j) acc[j] = mfma32<BF16>(H::columns(tk, b * 32 + k * 16, j, lane), ds, acc[j]);
      }
    }
  }
  if (!live) return;
  store_columns<BF16>(acc, a.scale * range.back(), o.dq,
                      o.dq_part ? o.dq_part + split * a.qi.n * heads * a.D : nullptr, row, a.D, h);
}

// 32 keys a wave, 128 a workgroup; the walk is over the group's query heads and
// their tiles of 64 queries. Up to 96 columns a wave takes a tile's two blocks of
// 32 queries in turn. Past that the sums (128 registers at 128 columns) leave room
// for K but not for V beside them at two waves a SIMD: V stays in LDS, eight waves
// make a workgroup, two of them share 32 keys and take one block of queries each,
// and their sums are added through LDS at the end.
template <bool BF16, int DP>
__global__ __launch_bounds__(DP > 96 ? 512 : 256, 2) void k_attention_dkv(Attention a, AttnGrad o) {
  constexpr bool PAIRED = DP > 96;
  constexpr int NW = PAIRED ? 8 : 4, T = 128, SHIFT = 7;
  using H = HeadTile<DP>;
  using L = TileLoad<DP, NW>;
  constexpr int KS = DP / 16, DB = DP / 32;
  constexpr int STAGES = PAIRED ? 3 : 2;  // tiles of queries in LDS
  __shared__ __attribute__((aligned(16))) char smem[STAGES][2][H::BYTES];
  __shared__ __attribute__((aligned(16))) char vmem[PAIRED ? 2 * H::BYTES : 16];  // V of the workgroup's keys
  __shared__ __attribute__((aligned(16))) float stats[STAGES][2][kTileKeys];  // base and delta of a tile's queries
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = wave & 3, half = wave >> 2;  // the wave's keys; its block of queries where PAIRED
  const Place at = place_of(blockIdx.x, o.slots, a.kv_heads, a.causal, !PAIRED, o.by_slot);
  const Walk w = walk_of(a.ki, 1, SHIFT, o.slots, o.splits, at.slot, a.causal, true);
  const ItemTile t = w.t;
  const int split = w.split;
  const Extent x = extent_of(a, t, true);
  const int64_t k_first = t.tile * T;
  if (t.tile < 0 || k_first >= x.k_rows) return;

  const int32_t j = static_cast<int32_t>(k_first) + part * 32 + (lane & 31);  // this lane's key
  const bool seen = j < x.Lk;
  // Query i sees key j from i = j - (Lk - Lq) on under the causal mask.
  const int32_t lag = x.Lk - x.Lq;
  const int32_t from = a.causal ? max(0, j - lag) : 0;
  const int32_t wave_last = static_cast<int32_t>(k_first) + part * 32 + 31;
  const int32_t from_most = a.causal ? max(0, wave_last - lag) : 0;
  const bool whole = wave_last < x.Lk;
  const int32_t i_first = a.causal ? max(0, static_cast<int32_t>(k_first) - lag) : 0;
  const int first_tile = i_first / kTileKeys;
  const int q_tiles = x.Lk > k_first ? max(0, (x.Lq + kTileKeys - 1) / kTileKeys - first_tile) : 0;
  const int walk = q_tiles * a.group;
  const int first = static_cast<int>(static_cast<int64_t>(walk) * split / o.splits);
  const int last = static_cast<int>(static_cast<int64_t>(walk) * (split + 1) / o.splits);

  L lq, ld;
  lq.init(a.q.ld, a.D, wave, lane);
  ld.init(o.dout.ld, a.D, wave, lane);
  const uint32_t lds = lds_addr(&smem[0][0][0]);
  const uint32_t lds_stats = lds_addr(reinterpret_cast<const char*>(&stats[0][0][0]));
  if (PAIRED && first < last) {
    L lv;
    lv.init(a.v.ld, a.D, wave, lane);
    const HeadRows vr{a.v.p + x.k0 * a.v.ld + at.head * a.v.hs, a.v.ld, x.Lk};
    const uint32_t to = lds_addr(&vmem[0]);
    lv.issue(vr, k_first, a.D, to, wave);
    lv.issue(vr, k_first + kTileKeys, a.D, to + H::BYTES, wave);
  }
  auto issue = [&](int head, int tile, int buf) {
    const int64_t row0 = static_cast<int64_t>(tile) * kTileKeys;
    const HeadRows qr{a.q.p + x.q0 * a.q.ld + head * a.q.hs, a.q.ld, x.Lq};
    const HeadRows dr{o.dout.p + x.q0 * o.dout.ld + head * o.dout.hs, o.dout.ld, x.Lq};
    lq.issue(qr, row0, a.D, lds + buf * 2 * H::BYTES, wave);
    ld.issue(dr, row0, a.D, lds + buf * 2 * H::BYTES + H::BYTES, wave);
    if (wave < 2) {  // one wave the bases, one the deltas; zeros past the last query
      const float* p = (wave == 0 ? o.row_base : o.row_delta) + head * a.qi.n + x.q0 + row0;
      rsrc4 r = load_rsrc(p, rows_left(x.Lq, row0, kTileKeys) * 4u);
      settle_rsrc(r);
      load_word_to_lds(r, lane * 4, lds_stats + (buf * 2 + wave) * kTileKeys * 4);
    }
  };
  const float c = a.scale * kLog2e;
  Range<BF16> range;
  float16v dk[DB], dv[DB];
#pragma unroll
  for (int i = 0; i < DB; ++i) dk[i] = dv[i] = float16v{};
  // From the item's last queries down: with the causal mask an item's keys start
  // from queries of their own, and this way their workgroups read the same ones at
  // the same time.
  struct Step {
    int head, tile;
  };
  auto next = [&](Step& w) {
    if (w.tile-- == first_tile) {
      w.tile = first_tile + q_tiles - 1;
      ++w.head;
    }
  };
  Step at_step{at.head * a.group, first_tile + q_tiles - 1};
  if (first < last) {
    at_step.head += first / q_tiles;
    at_step.tile -= first % q_tiles;
  }
  Step ahead = at_step;
  for (int i = 0; i < STAGES - 1; ++i)
    if (first + i < last) {
      issue(ahead.head, ahead.tile, i);
      next(ahead);
    }
  half8 kf[KS], vf[PAIRED ? 1 : KS];
  {
    const int64_t at_key = seen ? j : 0;
    const uint16_t* pk = a.k.p + (x.k0 + at_key) * a.k.ld + at.head * a.k.hs;
    const uint16_t* pv = a.v.p + (x.k0 + at_key) * a.v.ld + at.head * a.v.hs;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int c = kk * 16 + h * 8;
      kf[kk] = half8{};
      if (seen && c < a.D) kf[kk] = *reinterpret_cast<const half8*>(pk + c);
      if constexpr (!PAIRED) {
        vf[kk] = half8{};
        if (seen && c < a.D) vf[kk] = *reinterpret_cast<const half8*>(pv + c);
      }
    }
  }
  settle(kf);
  if constexpr (!PAIRED) settle(vf);
  int buf = 0;
  for (int u = first; u < last; ++u) {
    // this tile has landed (the next one may still be on its way) and all waves
    // are past the last one
    if (STAGES == 3 && u + 1 < last) {
      if (wave < 2) wait_loads<2 * L::N + 1>();
      else wait_loads<2 * L::N>();
    } else {
      wait_loads<0>();
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int32_t i0 = at_step.tile * kTileKeys;
    next(at_step);
    if (u + STAGES - 1 < last) {
      issue(ahead.head, ahead.tile, buf == 0 ? STAGES - 1 : buf - 1);
      next(ahead);
    }
    const char* tq = smem[buf][0];
    const char* td = smem[buf][1];
    auto block = [&](int b) {
      float16v s = {}, dp = {};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        s = mfma32<BF16>(H::rows(tq, b * 32, kk, lane), kf[kk], s);
        if constexpr (PAIRED)
          dp = mfma32<BF16>(H::rows(td, b * 32, kk, lane), H::rows(vmem, part * 32, kk, lane), dp);
        else
          dp = mfma32<BF16>(H::rows(td, b * 32, kk, lane), vf[kk], dp);
      }
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int at_row = b * 32 + 2 * i + 4 * h;
        const float4v base = *reinterpret_cast<const float4v*>(&stats[buf][0][at_row]);
        const float4v delta = *reinterpret_cast<const float4v*>(&stats[buf][1][at_row]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i + e] = __builtin_amdgcn_exp2f(s[i + e] * c + base[e]);
          dp[i + e] = s[i + e] * (dp[i + e] - delta[e]);
        }
      }
      if (!whole || i0 + b * 32 < from_most) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool on = seen && i0 + b * 32 + 8 * (i / 4) + 4 * h + i % 4 >= from;
          s[i] = on ? s[i] : 0.0f;
          dp[i] = on ? dp[i] : 0.0f;
        }
      }
      range.take(dp, dk);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const half8 p = operand_of<BF16>(s, 8 * k), ds = operand_of<BF16>(dp, 8 * k);
#pragma unroll
        for (int i = 0; i < DB; ++i) {
          dv[i] = mfma32<BF16>(H::columns(td, b * 32 + k * 16, i, lane), p, dv[i]);
          dk[i] = mfma32<BF16>(H::columns(tq, b * 32 + k * 16, i, lane), ds, dk[i]);
        }
      }
    };
    if constexpr (PAIRED) {
      block(half);
    } else {
      block(0);
      block(1);
    }
    buf = buf + 1 == STAGES ? 0 : buf + 1;
  }
  const int64_t row = (x.k0 + j) * a.kv_heads + at.head;
  const int64_t plane = split * a.ki.n * a.kv_heads * a.D;
  auto finish = [&](float16v (&acc)[DB], float f, uint16_t* out, float* part_out) {
    if (!out && !part_out) return;
    if constexpr (PAIRED) {
      // the second waves' sums, [part][register][lane]
      float* const sums = reinterpret_cast<float*>(&smem[0][0][0]);
      static_assert(4 * DB * 16 * 64 * 4 <= sizeof(smem), "sums fit the tiles");
      __syncthreads();
      if (half == 1) {
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) sums[((part * DB + i) * 16 + e) * 64 + lane] = acc[i][e] * f;
      }
      __syncthreads();
      if (half == 1) return;
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = acc[i][e] * f + sums[((part * DB + i) * 16 + e) * 64 + lane];
      f = 1.0f;
    }
    if (j < x.k_rows) store_columns<BF16>(acc, f, out, part_out ? part_out + plane : nullptr, row, a.D, h);
  };
  finish(dk, a.scale * range.back(), o.dk, o.dk_part);
  finish(dv, 1.0f / Range<BF16>::kP, o.dv, o.dv_part);
}

// ---- dispatch ----

int attention_backward(const Attention& a, const AttnGrad& g, bool bf16, Arena& ws, hipStream_t stream) {
  const int64_t items = a.qi.items, q_rows = a.qi.n * a.group * a.kv_heads, k_rows = a.ki.n * a.kv_heads;
  const int64_t mean_q = (a.qi.n + items - 1) / items, mean_k = (a.ki.n + items - 1) / items;
  AttnGrad o = g;
  o.by_slot = few_keys(a);
  o.row_base = static_cast<float*>(ws.take(q_rows * 4));
  o.row_delta = static_cast<float*>(ws.take(q_rows * 4));
  PlaneList planes;
  auto join = [&](uint16_t*& out, float*& part, int64_t rows, int splits) {
    if (splits == 1 || (!ws.counting && !out)) return;
    part = static_cast<float*>(ws.take(rows * splits * a.D * 4));
    planes.job[planes.count++] = PlaneJob{part, splits, rows * a.D, a.D, rows, a.D, 1, out};
    out = nullptr;
  };
  AttnGrad oq = o, ok = o;
  // (steps of 64 keys or queries, measured: 1.1 and 2.3 us at 64 columns, 1.8 and 2.4, two waves a block, at 128)
  const int64_t q_tiles = (mean_q * a.group + 127) / 128 * items * a.kv_heads;
  const int64_t k_tiles = (mean_k + 127) / 128 * items * a.kv_heads;
  oq.splits = splits_of(q_tiles, (mean_k + 63) / 64, 4.0, 0.5 + 0.01 * a.D, 1.0, seen_share(a), 512, q_rows * a.D).splits;
  ok.splits = splits_of(k_tiles, (mean_q + 63) / 64 * a.group, 4.0, a.D > 96 ? 2.4 : 1.0 + 0.02 * a.D, 1.0,
                        seen_share(a), a.D > 96 ? 256 : 512, 2 * k_rows * a.D)
                  .splits;
  oq.slots = item_slots(a.qi, a.group, 7) * oq.splits;
  ok.slots = item_slots(a.ki, 1, 7) * ok.splits;
  join(oq.dq, oq.dq_part, q_rows, oq.splits);
  join(ok.dk, ok.dk_part, k_rows, ok.splits);
  join(ok.dv, ok.dv_part, k_rows, ok.splits);
  if (ws.counting) return SUBMCONV_OK;
  const int64_t q_blocks = oq.slots * a.kv_heads, k_blocks = ok.slots * a.kv_heads;
  if (!launch_fits(q_blocks, 256) || !launch_fits(k_blocks, a.D > 96 ? 512 : 256))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "too many tiles: %lld and %lld", (long long)q_blocks,
                     (long long)k_blocks);
  const bool keys = a.ki.n > 0 && (g.dk || g.dv);
  auto go = [&](auto b, auto dp) {
    constexpr bool B = decltype(b)::value;
    if (a.qi.n > 0) {
      k_attention_dq<B, dp><<<static_cast<unsigned>(q_blocks), 256, 0, stream>>>(a, oq);
      SUBMCONV_HIP_CHECK(hipGetLastError());
    }
    if (keys) {
      k_attention_dkv<B, dp><<<static_cast<unsigned>(k_blocks), dp > 96 ? 512 : 256, 0, stream>>>(a, ok);
      SUBMCONV_HIP_CHECK(hipGetLastError());
    }
    return SUBMCONV_OK;
  };
  auto by_width = [&](auto b) {
    if (a.D <= 32) return go(b, std::integral_constant<int, 32>{});
    if (a.D <= 64) return go(b, std::integral_constant<int, 64>{});
    if (a.D <= 96) return go(b, std::integral_constant<int, 96>{});
    return go(b, std::integral_constant<int, 128>{});
  };
  SUBMCONV_TRY(bf16 ? by_width(std::true_type{}) : by_width(std::false_type{}));
  return planes.count ? run_planes(planes, bf16, stream) : SUBMCONV_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int64_t submconv_attention_backward_workspace_bytes(int64_t nq, int64_t nk, int32_t heads,
                                                               int32_t kv_heads, int32_t dim, int32_t items,
                                                               int32_t causal) {
  clear_error();
  const Attention a{{}, {}, {}, {reinterpret_cast<const int32_t*>(4), items, nq},
                    {reinterpret_cast<const int32_t*>(4), items, nk}, nullptr,
                    kv_heads > 0 ? heads / kv_heads : 0, kv_heads, dim, 1.0f, causal};
  SUBMCONV_TRY(check_attention(a, nq, nk, heads, SUBMCONV_DTYPE_F16));
  Arena ws;
  SUBMCONV_TRY(attention_backward(a, AttnGrad{}, false, ws, nullptr));
  return ws.used;
}

extern "C" int submconv_attention_backward(const uint16_t* grad_out, int64_t ldg, int64_t hg, const uint16_t* out,
                                           const float* lse, const uint16_t* q, int64_t ldq, int64_t hq, int64_t nq,
                                           const uint16_t* k, int64_t ldk, int64_t hk, const uint16_t* v, int64_t ldv,
                                           int64_t hv, int64_t nk, int32_t heads, int32_t kv_heads, int32_t dim,
                                           const int32_t* q_offsets, const int32_t* k_offsets,
                                           const int32_t* k_lengths, int32_t items, float scale, int32_t causal,
                                           uint16_t* grad_q, uint16_t* grad_k, uint16_t* grad_v, int32_t dtype,
                                           void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const Attention a{strided(q, nq, heads, dim, ldq, hq), strided(k, nk, kv_heads, dim, ldk, hk),
                    strided(v, nk, kv_heads, dim, ldv, hv), Items{q_offsets, items, nq}, Items{k_offsets, items, nk},
                    k_lengths, kv_heads > 0 ? heads / kv_heads : 0, kv_heads, dim, scale, causal};
  SUBMCONV_TRY(check_attention(a, nq, nk, heads, dtype));
  AttnGrad g{};
  g.dout = strided(grad_out, nq, heads, dim, ldg, hg);
  SUBMCONV_TRY(check_strided("q", a.q, nq, heads, dim));
  SUBMCONV_TRY(check_strided("k", a.k, nk, kv_heads, dim));
  SUBMCONV_TRY(check_strided("v", a.v, nk, kv_heads, dim));
  SUBMCONV_TRY(check_strided("grad_out", g.dout, nq, heads, dim));
  SUBMCONV_TRY(check_strided("out", strided(out, nq, 1, dim, dim, dim), nq, 1, dim));
  for (uint16_t* p : {grad_q, grad_k, grad_v})
    if (p) SUBMCONV_TRY(check_strided("a gradient", strided(p, 1, 1, dim, dim, dim), 1, 1, dim));
  if (nq > 0 && !lse) return set_error(SUBMCONV_ERR_INVALID_ARG, "lse is NULL");
  if (!grad_q && !grad_k && !grad_v) return SUBMCONV_OK;
  if (nq == 0 && nk == 0) return SUBMCONV_OK;
  g.out = out;
  g.lse = lse;
  g.dq = grad_q;
  g.dk = grad_k;
  g.dv = grad_v;
  const bool bf16 = dtype == SUBMCONV_DTYPE_BF16;
  Arena need, ws{false, static_cast<char*>(workspace)};
  SUBMCONV_TRY(attention_backward(a, g, bf16, need, stream));
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, need.used));
  return attention_backward(a, g, bf16, ws, stream);
}
