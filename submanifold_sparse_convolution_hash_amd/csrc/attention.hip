// Attention among the rows of packed items, forward. Per query i of an item and
// head, over the keys j that it sees (all of the item's, or with the causal mask
// those up to its own place counted from the end, j <= i + Lk - Lq):
//
//   s_j = scale q_i . k_j,  lse_i = log sum_j exp s_j,  o_i = sum_j exp(s_j - lse_i) v_j
//
// A query that sees no key has o = 0 and lse = -inf.
//
// One pass over the keys with a running maximum and sum. The `group` query heads
// that share a key head are rows of one matrix, row = token group + head, so that
// a few tokens still fill a tile and keys are read once for all of them. A wave
// owns 32 such rows; it forms scores^T = K Q^T, so that a lane holds all of its
// scores of one row: the maximum and the sum need one exchange between the halves
// of the wave, and the rounded weights are at once the operand of O^T = V^T P^T.
// Products, maximum, sum and O are fp32; weights are rounded to 16 bits for the
// second product, as its operands have to be.
//
// 8192 rows of 8 heads of 128 bf16 255-268 us, 1030-1080 TFLOP/s; 20011 rows of two
// items, 12 heads of 64 fp16 734-760 us, 810-840; 8192 causal rows of four items, 16 / 4
// heads of 128 86-89 us, 830-860. Bound by the vector units (68 % busy at 64 columns, where
// exp2 takes half of what the matrix units take) and by power: the clock falls to
// 1.7-1.9 GHz, and zeros in place of random numbers take a quarter less time (a
// library product of 8192^3 reaches 1240 TFLOP/s here). So what counts is the work
// per score: scale and maximum go into one multiply-add, the sums are scaled only
// when the maximum rises (kSlack), masks are applied in tiles that need them. 64
// rows a wave, which read LDS half as often, took 735 us in place of 760 at 64
// columns and left small inputs half the workgroups; priorities around the products
// (s_setprio) and more chains in maximum and sum changed nothing.
#include <algorithm>

#include "attention_tile.h"

namespace submconv {
namespace {

struct AttnOut {
  uint16_t* out;    // [nq][heads][D]
  float* lse;       // [nq][heads] or null
  float* part;      // [splits][nq][heads][D], where the keys are split
  float* part_lse;  // [splits][nq][heads]
  int32_t splits;
  int64_t slots;  // tiles, times the splits
  bool by_slot;   // see place_of
};

// The maximum is raised, and what was summed scaled down, only once a score
// passes it by this many powers of two: weights stay below 2^8, which bf16
// holds as exactly as any other, and the sums' 32 bits have room. In fp16 they are
// taken times 2^7, up to 2^15 of its range, so that small ones beside a large one
// keep their digits: a weight loses at most 2^-32 of the row's largest. (As they
// are it is 2^-25: beside one key of value 0 whose score leads by 17, the output of
// all others was 0.)
constexpr float kSlack = 8.0f;
template <bool BF16>
constexpr float kUp = BF16 ? 0.0f : 7.0f;

// KG = 2: two groups of NW waves have the same rows and take every other tile of
// keys, each with its own buffers; what they have is joined through LDS. For the
// same waves on a unit this halves the walk of a workgroup that would be alone on
// it: 2048 causal rows of 16 heads of 128 48.5 -> 40.5 us.
template <bool BF16, int DP, int NW, int KG>
__global__ __launch_bounds__(NW * KG * 64, NW == 1 ? 1 : 2) void k_attention(Attention a, AttnOut o) {
  constexpr int T = 32 * NW, SHIFT = NW == 1 ? 5 : 7;
  static_assert(T == 1 << SHIFT, "rows");
  using H = HeadTile<DP>;
  using L = TileLoad<DP, NW>;
  constexpr int KS = DP / 16, DB = DP / 32;
  __shared__ __attribute__((aligned(16))) char tiles_of[KG][2][2][H::BYTES];
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5;
  const int wave_of = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = wave_of % NW, kg = wave_of / NW;
  char(&smem)[2][2][H::BYTES] = tiles_of[kg];
  const Place at = place_of(blockIdx.x, o.slots, a.kv_heads, a.causal, KG == 1, o.by_slot);
  const Walk w = walk_of(a.qi, a.group, SHIFT, o.slots, o.splits, at.slot, a.causal, false);
  const ItemTile t = w.t;
  const int split = w.split;
  const Extent x = extent_of(a, t, false);
  const int64_t rows = static_cast<int64_t>(x.q_rows) * a.group, r_first = t.tile * T;
  if (t.tile < 0 || r_first >= rows) return;

  // this lane's row
  const TileRows at_row(r_first, rows, T, a.group);
  const int i = wave * 32 + (lane & 31);
  const bool live = i < at_row.count;
  const int32_t token = at_row.token(i);
  const int head = at.head * a.group + at_row.head(i);
  const int32_t see = keys_of(a, x, token);
  const int32_t see_least = keys_of(a, x, at_row.token(wave * 32));  // of the wave's rows: the first's
  const int32_t see_most = keys_of(a, x, at_row.token(T - 1));
  const int tiles = (see_most + kTileKeys - 1) / kTileKeys;
  const int first = static_cast<int>(static_cast<int64_t>(tiles) * split / o.splits);
  const int last = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / o.splits);

  const HeadRows kr{a.k.p + x.k0 * a.k.ld + at.head * a.k.hs, a.k.ld, x.Lk};
  const HeadRows vr{a.v.p + x.k0 * a.v.ld + at.head * a.v.hs, a.v.ld, x.Lk};
  L lk, lv;
  lk.init(a.k.ld, a.D, wave, lane);
  lv.init(a.v.ld, a.D, wave, lane);
  const uint32_t lds = lds_addr(&smem[0][0][0]);
  auto issue = [&](int tile, int buf) {
    const uint32_t to = lds + buf * 2 * H::BYTES;
    lk.issue(kr, static_cast<int64_t>(tile) * kTileKeys, a.D, to, wave);
    lv.issue(vr, static_cast<int64_t>(tile) * kTileKeys, a.D, to + H::BYTES, wave);
  };

  if (first + kg < last) issue(first + kg, 0);  // on its way beside the queries
  half8 q[KS];
  {
    const uint16_t* p = a.q.p + (x.q0 + token) * a.q.ld + head * a.q.hs;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int c = kk * 16 + h * 8;
      q[kk] = half8{};
      if (c < a.D) q[kk] = *reinterpret_cast<const half8*>(p + c);
    }
  }
  settle(q);
  const float c = a.scale * kLog2e;
  float m = -kInf, mc = 0.0f, sum = 0.0f;  // mc = m c - kUp, 0 while m is -inf
  float16v acc[DB];
#pragma unroll
  for (int j = 0; j < DB; ++j) acc[j] = float16v{};
  // One tile, of the buffer whose number is a constant: its addresses are then
  // offsets in the reads.
  auto step = [&](int tile, auto buf) {
    // this tile has landed and all waves are past the last one
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (tile + KG < last) issue(tile + KG, buf ^ 1);
    if (KG > 1 && tile >= last) return;  // (the other group has one more)
    const char* tk = smem[buf][0];
    const char* tv = smem[buf][1];
    float16v s[2] = {};
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
      for (int b = 0; b < 2; ++b) s[b] = mfma32<BF16>(H::rows(tk, b * 32, kk, lane), q[kk], s[b]);
    const int j0 = tile * kTileKeys;
    if (j0 + kTileKeys > see_least) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + b * 32 + 8 * (i / 4) + 4 * h + i % 4 >= see) s[b][i] = -kInf;
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = b == 0 ? 1 : 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = halves_max(top);
    const bool raise = top * c > mc + (kUp<BF16> + kSlack) || (m == -kInf && top > -kInf);
    if (__ballot(raise)) {
      const float next = raise ? top : m;
      const float nc = next == -kInf ? 0.0f : next * c - kUp<BF16>;
      const float f = m == -kInf ? 0.0f : __builtin_amdgcn_exp2f(mc - nc);
      m = next;
      mc = nc;
      sum *= f;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] *= f;
    }
    half8 p[4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[b][i] = __builtin_amdgcn_exp2f(s[b][i] * c - mc);
        sum += s[b][i];
      }
      p[2 * b] = operand_of<BF16>(s[b], 0);
      p[2 * b + 1] = operand_of<BF16>(s[b], 8);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < DB; ++j) acc[j] = mfma32<BF16>(H::columns(tv, k * 16, j, lane), p[k], acc[j]);
  };
  for (int tile = first; tile < last; tile += 2 * KG) {
    step(tile + kg, std::integral_constant<int, 0>{});
    if (tile + KG < last) step(tile + KG + kg, std::integral_constant<int, 1>{});
  }
  if constexpr (KG > 1) {
    static_assert(KG == 2 && NW * DB * 16 * 64 * 4 <= sizeof(smem), "sums fit the tiles");
    __shared__ float tops[2][NW * 64];
    float* const sums = reinterpret_cast<float*>(&tiles_of[1][0][0][0]);
    __syncthreads();
    if (kg == 1) {
      tops[0][wave * 64 + lane] = m == -kInf ? -kInf : mc;
      tops[1][wave * 64 + lane] = sum;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) sums[((wave * DB + j) * 16 + i) * 64 + lane] = acc[j][i];
    }
    __syncthreads();
    if (kg == 1) return;
    const float other = tops[0][wave * 64 + lane], mine = m == -kInf ? -kInf : mc;
    const float top = fmaxf(mine, other), base = top == -kInf ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(mine - base), g = __builtin_amdgcn_exp2f(other - base);
    mc = base;
    sum = sum * f + tops[1][wave * 64 + lane] * g;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] = acc[j][i] * f + sums[((wave * DB + j) * 16 + i) * 64 + lane] * g;
  }
  sum = halves_sum(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // (a NaN stays one)
  const float lse = sum == 0.0f ? -kInf : (mc + __log2f(sum)) * kLn2;
  if (!live) return;
  const int64_t heads = static_cast<int64_t>(a.kv_heads) * a.group;
  int64_t to = (x.q0 + token) * heads + head;
  if (o.splits == 1) {
    if (o.lse && h == 0) o.lse[to] = lse;
    uint16_t* out = o.out + to * a.D;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        float4v u, w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = acc[j][i + e] * inv;
          w[e] = acc[j][i + 4 + e] * inv;
        }
        const u32x4 v = eight_rows<BF16>(u, w);
        const int d = j * 32 + i * 2 + h * 8;
        if (d < a.D) *reinterpret_cast<u32x4*>(out + d) = v;
      }
    return;
  }
  to += split * a.qi.n * heads;
  if (h == 0) o.part_lse[to] = lse;
  float* part = o.part + to * a.D;
#pragma unroll
  for (int j = 0; j < DB; ++j)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = j * 32 + i * 2 + h * 4;
      float4v u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = acc[j][i + e] * inv;
      if (d < a.D) *reinterpret_cast<float4v*>(part + d) = u;
    }
}

// Joins the splits: o = sum_s w_s o_s, w_s = exp(lse_s - lse). A wave has one row
// of [nq heads]: its lanes the weights of the splits, then pieces of four columns,
// the splits shared among up to eight groups of lanes, whose first loads are on
// their way before the weights are known. 128 rows of 64 columns, 32 splits: 4.6 us
// (16 splits joined by a thread per four columns: 7.2).
constexpr int kJoinGroups = 8;
template <bool BF16>
__global__ __launch_bounds__(256) void k_attention_join(const float* __restrict__ part,
                                                        const float* __restrict__ part_lse, int64_t rows, int D,
                                                        int splits, uint16_t* __restrict__ out,
                                                        float* __restrict__ lse) {
  constexpr int AHEAD = 8, PER = kMostSplits / 64;
  __shared__ float weights[4][kMostSplits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (row >= rows) return;
  const int pieces = D / 4, groups = min(64 / pieces, kJoinGroups);
  const int piece = lane % pieces, group = lane / pieces;
  const bool on = group < groups;
  float l[PER], top = -kInf, total = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    l[i] = lane + i * 64 < splits ? part_lse[(lane + i * 64) * rows + row] : -kInf;
    top = fmaxf(top, l[i]);
  }
  auto load = [&](int s) {
    return on && s < splits ? *reinterpret_cast<const float4v*>(part + (s * rows + row) * D + piece * 4) : float4v{};
  };
  float4v u[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) u[i] = load(group + i * groups);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float w = __builtin_amdgcn_exp2f((l[i] - (top == -kInf ? 0.0f : top)) * kLog2e);
    weights[wave][lane + i * 64] = w;  // read by this wave alone
    total += w;
  }
  total = lanes_sum<64>(total);
  float4v v = {};
  for (int i = 0; i * groups < splits; i += AHEAD) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int s = group + (i + k) * groups;
      const float f = s < splits ? weights[wave][s] : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += s < splits ? f * u[k][e] : 0.0f;
    }
    if ((i + AHEAD) * groups < splits) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) u[k] = load(group + (i + AHEAD + k) * groups);
    }
  }
  const float inv = total > 0.0f ? 1.0f / total : total == 0.0f ? 0.0f : total;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float sum = v[e];
    for (int g = 1; g < groups; ++g) sum += __shfl(v[e], (lane + g * pieces) & 63, 64);
    v[e] = sum * inv;
  }
  if (lane < pieces) *reinterpret_cast<u32x2*>(out + row * D + lane * 4) = pack4<BF16>(v);
  if (lse && lane == 0) lse[row] = total == 0.0f ? -kInf : top + __log2f(total) * kLn2;
}

// ---- dispatch ----

struct Plan {
  int waves, groups, splits;
  int64_t slots;
};

// One wave a workgroup where the items have at most 32 rows on average, else four,
// two workgroups a unit: a step of 64 keys takes them 0.9 us at 64 columns and 1.4
// at 128. Or twice four, one workgroup a unit, where that is faster: their start and
// join take 6 us, their steps 1.45 times as long, and they walk half as far. A single
// wave waits for its loads, 1.3 to 1.6 us a step; as many workgroups of one run on
// a unit at once as its LDS holds their tiles.
Plan plan_of(const Attention& a) {
  Plan p;
  const int64_t mean_rows = (a.qi.n * a.group + a.qi.items - 1) / a.qi.items;
  p.waves = mean_rows <= 32 ? 1 : 4;
  const int64_t tile = p.waves * 32;
  const int64_t tiles = std::max<int64_t>(1, (mean_rows + tile - 1) / tile * a.qi.items * a.kv_heads);
  const int64_t steps = (a.ki.n / a.qi.items + kTileKeys - 1) / kTileKeys;
  const int64_t floats = a.qi.n * a.group * a.kv_heads * a.D;
  const double seen = seen_share(a), step = 0.46 + 0.007 * a.D;
  Splits s;
  if (p.waves == 1) {
    s = splits_of(tiles, steps, 4.0, 1.0 + 0.005 * a.D, 1.0, seen, a.D > 64 ? 512 : a.D > 32 ? 1280 : 2560, floats);
    p.groups = 1;
  } else {
    s = splits_of(tiles, steps, 4.0, step, 1.4, seen, 512, floats);
    const Splits two = splits_of(tiles, (steps + 1) / 2, 6.0, 1.45 * step, 1.15, seen, 256, floats);
    p.groups = two.us < s.us ? 2 : 1;
    if (p.groups == 2) s = two;
  }
  p.splits = s.splits;
  p.slots = item_slots(a.qi, a.group, p.waves == 1 ? 5 : 7) * p.splits;
  return p;
}

int attention_forward(const Attention& a, bool bf16, uint16_t* out, float* lse, Arena& ws, hipStream_t stream) {
  const Plan p = plan_of(a);
  const int64_t rows = a.qi.n * a.group * a.kv_heads;
  AttnOut o{out, lse, nullptr, nullptr, p.splits, p.slots, few_keys(a)};
  if (p.splits > 1) {
    o.part = static_cast<float*>(ws.take(rows * p.splits * a.D * 4));
    o.part_lse = static_cast<float*>(ws.take(rows * p.splits * 4));
  }
  if (ws.counting) return SUBMCONV_OK;
  const int64_t blocks = p.slots * a.kv_heads;
  if (!launch_fits(blocks, p.waves * p.groups * 64))
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "too many tiles: %lld", (long long)blocks);
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  auto go = [&](auto dp, auto nw, auto kg) {
    const unsigned grid = static_cast<unsigned>(blocks);
    if (bf16) k_attention<true, dp, nw, kg><<<grid, nw * kg * 64, 0, stream>>>(a, o);
    else k_attention<false, dp, nw, kg><<<grid, nw * kg * 64, 0, stream>>>(a, o);
  };
  auto by_width = [&](auto nw, auto kg) {
    if (a.D <= 32) go(std::integral_constant<int, 32>{}, nw, kg);
    else if (a.D <= 64) go(std::integral_constant<int, 64>{}, nw, kg);
    else if (a.D <= 96) go(std::integral_constant<int, 96>{}, nw, kg);
    else go(std::integral_constant<int, 128>{}, nw, kg);
  };
  if (p.waves == 1) by_width(One{}, One{});
  else if (p.groups == 1) by_width(Four{}, One{});
  else by_width(Four{}, Two{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  if (p.splits > 1) {
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    if (bf16) k_attention_join<true><<<grid, 256, 0, stream>>>(o.part, o.part_lse, rows, a.D, p.splits, out, lse);
    else k_attention_join<false><<<grid, 256, 0, stream>>>(o.part, o.part_lse, rows, a.D, p.splits, out, lse);
    SUBMCONV_HIP_CHECK(hipGetLastError());
  }
  return SUBMCONV_OK;
}

}  // namespace

int check_strided(const char* name, const Strided& s, int64_t n, int32_t heads, int32_t D) {
  if (n > 0 && !s.p) return set_error(SUBMCONV_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(s.p) & 15)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s does not start on 16 bytes", name);
  if ((n > 1 && s.ld % 8) || (heads > 1 && s.hs % 8))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: strides %lld, %lld are not multiples of 8", name,
                     (long long)s.ld, (long long)s.hs);
  if ((heads > 1 && s.hs < D) || (n > 1 && s.ld < D))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%s: strides %lld, %lld below %d columns", name, (long long)s.ld,
                     (long long)s.hs, D);
  if (n > 1 && s.ld > kMaxLd)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%s: row stride %lld above %lld", name, (long long)s.ld,
                     (long long)kMaxLd);
  return SUBMCONV_OK;
}

// (a tile's row numbers past the last one stay within 32 bits)
constexpr int64_t kMostRows = INT32_MAX - 1024;

int check_attention(const Attention& a, int64_t nq, int64_t nk, int32_t heads, int32_t dtype) {
  if (dtype != SUBMCONV_DTYPE_F16 && dtype != SUBMCONV_DTYPE_BF16)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "dtype = %d", dtype);
  if (nq < 0 || nk < 0 || nq > kMostRows || nk > kMostRows)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%lld queries, %lld keys", (long long)nq, (long long)nk);
  if (a.kv_heads < 1 || heads < a.kv_heads || heads % a.kv_heads || heads > 65536)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d heads on %d key heads", heads, a.kv_heads);
  if (a.D < 8 || a.D > 128 || a.D % 8)
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "%d columns a head, multiples of 8 up to 128 are supported", a.D);
  if (a.qi.items < 1 || a.qi.items > 65535)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items, 1 to 65535 are supported", a.qi.items);
  if ((!a.qi.offsets || !a.ki.offsets) && a.qi.items != 1)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items without offsets", a.qi.items);
  if (!(a.scale > 0.0f) || a.scale > 2e38f) return set_error(SUBMCONV_ERR_INVALID_ARG, "scale = %g", a.scale);
  return SUBMCONV_OK;
}

}  // namespace submconv

using namespace submconv;

extern "C" int64_t submconv_attention_workspace_bytes(int64_t nq, int64_t nk, int32_t heads, int32_t kv_heads,
                                                      int32_t dim, int32_t items, int32_t causal) {
  clear_error();
  const Attention a{{}, {}, {}, {reinterpret_cast<const int32_t*>(4), items, nq},
                    {reinterpret_cast<const int32_t*>(4), items, nk}, nullptr,
                    kv_heads > 0 ? heads / kv_heads : 0, kv_heads, dim, 1.0f, causal};
  SUBMCONV_TRY(check_attention(a, nq, nk, heads, SUBMCONV_DTYPE_F16));
  Arena ws;
  SUBMCONV_TRY(attention_forward(a, false, nullptr, nullptr, ws, nullptr));
  return ws.used;
}

extern "C" int submconv_attention(const uint16_t* q, int64_t ldq, int64_t hq, int64_t nq, const uint16_t* k,
                                  int64_t ldk, int64_t hk, const uint16_t* v, int64_t ldv, int64_t hv, int64_t nk,
                                  int32_t heads, int32_t kv_heads, int32_t dim, const int32_t* q_offsets,
                                  const int32_t* k_offsets, const int32_t* k_lengths, int32_t items, float scale,
                                  int32_t causal, uint16_t* out, float* lse, int32_t dtype, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const Attention a{strided(q, nq, heads, dim, ldq, hq), strided(k, nk, kv_heads, dim, ldk, hk),
                    strided(v, nk, kv_heads, dim, ldv, hv), Items{q_offsets, items, nq}, Items{k_offsets, items, nk},
                    k_lengths, kv_heads > 0 ? heads / kv_heads : 0, kv_heads, dim, scale, causal};
  SUBMCONV_TRY(check_attention(a, nq, nk, heads, dtype));
  SUBMCONV_TRY(check_strided("q", a.q, nq, heads, dim));
  SUBMCONV_TRY(check_strided("k", a.k, nk, kv_heads, dim));
  SUBMCONV_TRY(check_strided("v", a.v, nk, kv_heads, dim));
  SUBMCONV_TRY(check_strided("out", strided(out, nq, 1, dim, dim, dim), nq, 1, dim));
  if (nq == 0) return SUBMCONV_OK;
  const bool bf16 = dtype == SUBMCONV_DTYPE_BF16;
  Arena need, ws{false, static_cast<char*>(workspace)};
  SUBMCONV_TRY(attention_forward(a, bf16, out, lse, need, stream));
  SUBMCONV_TRY(check_workspace(workspace, workspace_bytes, need.used));
  return attention_forward(a, bf16, out, lse, ws, stream);
}
