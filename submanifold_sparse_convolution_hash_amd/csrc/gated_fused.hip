// The whole gated feed-forward block of a layer with at most 128 input and 128
// output channels in one kernel:
//
//   [g | u] = x W_in + b_in,  h = act(g) u,  out = h W_out + b_out + residual
//
// At these widths the hidden rows are the traffic: at 209715 x 128 / 512 they
// are 215 MB written and read between two kernels, four times x and out. Here
// they never leave the registers. A wave owns 32 rows (16 where
// there are few): their x is read once into MFMA operands, their out stays in
// accumulators, and the hidden channels pass by in chunks of 32. A chunk's columns of W_in and rows of W_out go
// through LDS, shared by the workgroup's waves; the chunk's g and u accumulate
// on b_in, and h, rounded to 16 bits, is at once the operand of the second
// product: an accumulator holds 4 consecutive hidden channels of one row per
// lane, two of them the 8 values of k of one operand, and W_out is read from
// LDS in that same order of k.
//
// 209715 x 128 / 512 with silu and a residual: 123-131 us, 650 TFLOP/s (two
// kernels: 207 us). The matrix units are busy 27 % and the vector units, with exp
// and reciprocal at a quarter of their rate, 35 % of the time; two waves a SIMD
// (the registers allow no more) overlap them only in part, and the last of 3.2
// rounds of workgroups is mostly empty (given to a launch of its own with half
// the rows a wave, it cost as much again: 131 -> 135 us on new rows). Chunks of
// 64, one buffer, eight waves, and reads or activations interleaved by hand
// measured the same or slower (126 to 144 us).
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "linear_epilogue.h"

namespace submconv {
namespace {

constexpr int kHidden = 32;      // hidden channels of a chunk
constexpr int kWaves = 4;        // of a workgroup; two workgroups fit a compute unit
constexpr int kFusedHidden = 2048;  // most hidden channels (their biases sit in LDS)

// A chunk's k rows of W_out, OC columns: the transposed reads take k rows 4 g ..
// + 3 (g = lane / 16) of two 16-row blocks, so the swizzle goes by k % 8.
template <int OC, int NT>
struct LoadOut {
  static constexpr int CH = OC / 8;
  static constexpr int SL = kHidden * CH / NT > 0 ? kHidden * CH / NT : 1;
  static_assert(kHidden * CH % NT == 0, "slots");
  uint32_t voff[SL];
  static __device__ __forceinline__ int swz(int k) { return ((k & 7) << 1) & (CH - 1); }
  __device__ __forceinline__ void init(const Operand& o, int tid) {
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int s = tid + i * NT, k = s / CH, c = (s % CH ^ swz(k)) * 8;
      voff[i] = c < o.rows ? static_cast<uint32_t>(k * o.ld + c) * 2u : kOobOff;
    }
  }
  __device__ __forceinline__ void issue(const Operand& o, uint32_t lds, int64_t k0, int wave) const {
    const int64_t left = o.k - k0;
    rsrc4 r = load_rsrc(o.p + k0 * o.ld,
                        left > 0 ? static_cast<uint32_t>(((left < kHidden ? left : kHidden) - 1) * o.ld + o.rows) * 2u : 0u);
    settle_rsrc(r);
#pragma unroll
    for (int i = 0; i < SL; ++i) load_to_lds(r, voff[i], lds + (i * NT + wave * 64) * 16);
  }
  // the operand of out block j over the chunk's two hidden blocks
  static __device__ __forceinline__ half8 frag(const char* tile, int j, int lane) {
    const int g = lane >> 4, s = lane & 15;
    const int k = g * 4 + (s >> 2);  // and 16 further on
    const int c = (j * 2 + ((s & 3) >> 1)) ^ swz(k);
    const char* q = tile + k * (OC * 2) + c * 16 + (s & 1) * 8;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)q);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(q + 16 * OC * 2));
    return __builtin_bit_cast(half8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// x [M][<= KC], W_in [C][2 F] as a pair operand, W_out [F][<= OC], out as in
// LinearEpi.
template <bool BF16, int KC, int OC, int FM>
__global__ __launch_bounds__(kWaves * 64, 2) void k_gated_ffn(Operand X, Operand Wi, Operand Wo,
                                                          int64_t half, const float* __restrict__ b_in,
                                                          int64_t F, int64_t cout, int act, LinearEpi e) {
  constexpr int NT = kWaves * 64, kWaveRows = 16 * FM, KS = KC / 32, OB = OC / 16;
  using LI = LoadKRow<2 * kHidden, NT, true, false>;
  using LO = LoadOut<OC, NT>;
  using T = Tile<BF16, false, true, true, 128, 2 * kHidden, 1, 1, 2>;  // its operand reads
  constexpr int IN_BYTES = kStepK * 2 * kHidden * 2, TILE = KC / kStepK * IN_BYTES + kHidden * OC * 2;
  constexpr int ROWS = kWaves * kWaveRows, PH = 2;
  using R = LdsRows<ROWS / PH, OC, NT>;  // of the out rows, half of them at a time
  static_assert(R::PH_ROWS * OC * 4 <= 2 * TILE, "the rows fit the weights' buffers");
  __shared__ __attribute__((aligned(16))) char smem[2 * TILE];
  __shared__ __attribute__((aligned(16))) float bias[2][kFusedHidden];  // b_in, zeros past F
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, s = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * ROWS;

  // x of the wave's rows: k pieces past the width and rows past the last are
  // zeros
  half8 xf[KS][FM];
  {
    const int64_t left = X.rows - m0 - wave * kWaveRows;
    const __amdgpu_buffer_rsrc_t r =
        tile_rsrc(X.p + (m0 + wave * kWaveRows) * X.ld,
                  left > 0 ? static_cast<uint32_t>(((left < kWaveRows ? left : kWaveRows) - 1) * X.ld + X.k) * 2u : 0u);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int k = kk * 32 + g * 8;
        const uint32_t off = static_cast<uint32_t>((i * 16 + s) * X.ld + k) * 2u;
        xf[kk][i] = __builtin_bit_cast(half8, __builtin_amdgcn_raw_buffer_load_b128(r, k < X.k ? off : kOobOff, 0, 0));
      }
  }
  LO lo;
  lo.init(Wo, tid);
  const uint32_t lds = lds_addr(smem);
  const int chunks = static_cast<int>((F + kHidden - 1) / kHidden);
  LI li;
  li.init(Wi, 0, half, tid);
  auto issue = [&](int c, int buf) {
    if (c > 0) li.next(kHidden, Wi.rows);
#pragma unroll
    for (int q = 0; q < KC / kStepK; ++q)
      li.issue(lds + buf * TILE + q * IN_BYTES, q * kStepK, X.k, wave);  // zeros past x's width
    lo.issue(Wo, lds + buf * TILE + KC / kStepK * IN_BYTES, static_cast<int64_t>(c) * kHidden, wave);
  };

  float4v out[OB][FM];
#pragma unroll
  for (int j = 0; j < OB; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i) out[j][i] = float4v{};
  for (int n = tid; n < chunks * kHidden; n += NT)
#pragma unroll
    for (int q = 0; q < 2; ++q) bias[q][n] = b_in && n < F ? b_in[q * F + n] : 0.0f;
  // (the first chunk's barrier makes them every wave's)
  issue(0, 0);
  with_act(act, [&](auto a) {
    for (int c = 0; c < chunks; ++c) {
      // this chunk's weights have landed and all waves are past the last one
      wait_loads<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (c + 1 < chunks) issue(c + 1, (c + 1) & 1);
      const char* ti = smem + (c & 1) * TILE;
      const char* to = ti + KC / kStepK * IN_BYTES;
      // Accumulators 0, 1: the gate's two blocks of 16 channels, 2, 3: the up
      // projection's. LDS reads are issued a group of operands ahead of the
      // products that take them (the scheduling barriers keep them there).
      half8 w[2][4], wo[OB];
      auto read_in = [&](int kk, half8 (&r)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[j] = T::template frag<2 * kHidden, true>(ti + kk / 2 * IN_BYTES, j * 16, kk & 1, lane);
      };
      read_in(0, w[0]);
      float4v acc[4][FM];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4v b = *reinterpret_cast<const float4v*>(&bias[j >> 1][c * kHidden + (j & 1) * 16 + g * 4]);
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = b;
      }
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        if (kk + 1 < KS) {
          read_in(kk + 1, w[(kk + 1) & 1]);
        } else {
#pragma unroll
          for (int j = 0; j < OB; ++j) wo[j] = LO::frag(to, j, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < FM; ++i) acc[j][i] = mfma16<BF16>(w[kk & 1][j], xf[kk][i], acc[j][i]);
      }
      half8 h[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          v[q] = act_value<decltype(a)::value>(acc[q / 4][i][q % 4]) * acc[2 + q / 4][i][q % 4];
        h[i] = __builtin_bit_cast(half8, pack8<BF16>(v));
      }
#pragma unroll
      for (int j = 0; j < OB; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) out[j][i] = mfma16<BF16>(wo[j], h[i], out[j][i]);
    }
  });

  // hidden channels past F are zeros in W_out's rows (and g = u = 0 there)
#pragma unroll 1
  for (int ph = 0; ph < PH; ++ph) {
    __syncthreads();
    if (wave / (kWaves / PH) == ph) {
      const int r0 = wave % (kWaves / PH) * kWaveRows;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < OB; ++j)
          *reinterpret_cast<float4v*>(smem + R::row_byte(r0 + i * 16 + s, j * 4 + g)) = out[j][i];
    }
    __syncthreads();
    linear_epilogue<BF16, kActNone, R>(e, X.rows, cout, m0 + ph * R::PH_ROWS, 0, smem);
  }
}

}  // namespace

// A workgroup walks all hidden channels, 32 at a time, whatever the rows: 0.5 us a
// chunk at 64 channels, 0.65 at 128, against 0.3 for the two kernels, which start
// from one launch more and spread the hidden channels until they run out of
// units. So the one kernel is taken for short walks, and for any from as many rows
// as fill the units; without those the two are even near hidden 850 and 450. One
// kernel against two, fp16, us:
//   64 channels, hidden 64 / 512 / 1024 / 2048: 256 rows 4.5 / 11.2 / 19.1 / 34 against 9.3 / 13.5 /
//   18.3 / 28, 4000 rows 4.6 / 11.4 / 19.1 / 34.3 against 9.5 / 14.1 / 20.3 / 34.5, 33000 rows 7.2 /
//   20 / 35 / 65 against 12.4 / 37 / 60 / 106;
//   128 channels, hidden 64 / 256 / 512 / 2048: 256 rows 5.5 / 9.4 / 14.8 / 46 against 10.0 / 12.0 /
//   14.1 / 28, 8000 rows 5.8 / 9.9 / 15.2 / 47.1 against 10.4 / 12.8 / 17.1 / 47.6, 33000 rows 10 / 18 /
//   29 / 95 against 13 / 25 / 43 / 129.
bool fused_ffn_takes(int64_t rows, int64_t cin, int64_t hidden, int64_t cout) {
  const int64_t most = std::max(cin, cout);
  if (hidden > kFusedHidden || most > 128) return false;
  return most <= 64 ? hidden <= 768 || rows >= 4096 : hidden <= 384 || rows >= 8192;
}

int fused_ffn(const Mat16& x, const Mat16& W_in, int64_t F, const float* b_in, const Mat16& W_out,
              const float* b_out, int act, bool bf16, const uint16_t* residual, int64_t ldr,
              uint16_t* out, int64_t cout, hipStream_t stream) {
  const int64_t half = W_in.cols / 2;
  const Operand X{x.p, x.ld, x.rows, x.cols}, Wi{W_in.p, W_in.ld, half, W_in.rows};
  const Operand Wo{W_out.p, W_out.ld, W_out.cols, W_out.rows};
  const LinearEpi e{b_out, residual, ldr, out, cout, nullptr, kActNone,
                    cout % 8 == 0 && ldr % 8 == 0 && aligned16(residual),
                    cout % 8 == 0 && aligned16(out), false};
  if (!launch_fits(div_up(x.rows, kWaves * 32), kWaves * 64))  // of 32 rows a wave
    return set_error(SUBMCONV_ERR_UNSUPPORTED_SHAPE, "too many rows: %lld", (long long)x.rows);
  auto go = [&](auto width, auto fm) {
    const dim3 grid(static_cast<unsigned>(div_up(x.rows, kWaves * 16 * fm)));
    if (bf16)
      k_gated_ffn<true, width, width, fm><<<grid, kWaves * 64, 0, stream>>>(X, Wi, Wo, half, b_in, F, cout, act, e);
    else
      k_gated_ffn<false, width, width, fm><<<grid, kWaves * 64, 0, stream>>>(X, Wi, Wo, half, b_in, F, cout, act, e);
  };
  auto by_rows = [&](auto width) {
    // 16 rows a wave where those fill at most every place once (two workgroups
    // a compute unit), else 32, which read the weights half as often. 32 against
    // 16: 128 / 512, 20000 rows 27.1 us against 22.2, 30000 rows 27.6 against 24.5;
    // 64 / 256, 1000 rows 11.2 against 8.8, 20000 rows 11.9 against 10.4.
    if (x.rows <= 512 * kWaves * 16) go(width, std::integral_constant<int, 1>{});
    else go(width, std::integral_constant<int, 2>{});
  };
  if (x.cols <= 64 && cout <= 64) by_rows(std::integral_constant<int, 64>{});
  else by_rows(std::integral_constant<int, 128>{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

}  // namespace submconv
