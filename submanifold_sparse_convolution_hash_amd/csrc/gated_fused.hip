// The whole gated feed-forward block of a layer with at most 128 input and 128
// output channels in one kernel:
//
//   [g | u] = x W_in + b_in,  h = act(g) u,  out = h W_out + b_out + residual
//
// At these widths the hidden rows are the traffic: at 209715 x 128 / 512 they
// are 215 MB written and read between two kernels, four times x and out. Here
// they never leave the registers. A wave owns 32 rows: their x is read once
// into MFMA operands, their out stays in accumulators, and the hidden channels
// pass by in chunks of 64. A chunk's columns of W_in and rows of W_out go
// through LDS, shared by the workgroup's waves; the chunk's g and u accumulate
// on b_in, and h, rounded to 16 bits, is at once the operand of the second
// product: an accumulator holds 4 consecutive hidden channels of one row per
// lane, two of them the 8 values of k of one operand, and W_out is read from
// LDS in that same order of k.
#include <algorithm>

#include "dense_common.h"
#include "dense_tile.h"
#include "linear_epilogue.h"

namespace submconv {
namespace {

constexpr int kHidden = 64;      // hidden channels of a chunk
constexpr int kWaveRows = 32;

// 64 k rows of W_out, OC columns: the transposed reads take k rows 4 g .. + 3
// (g = lane / 16) of two 16-row blocks, so the swizzle goes by k % 8.
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
  // the operand of out block j over the chunk's hidden blocks 2 t and 2 t + 1
  static __device__ __forceinline__ half8 frag(const char* tile, int j, int t, int lane) {
    const int g = lane >> 4, s = lane & 15;
    const int k = t * 32 + g * 4 + (s >> 2);
    const int c = (j * 2 + ((s & 3) >> 1)) ^ swz(k);
    const char* q = tile + k * (OC * 2) + c * 16 + (s & 1) * 8;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)q);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(q + 16 * OC * 2));
    return __builtin_bit_cast(half8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// x [M][<= KC], W_in [C][2 F] as a pair operand, W_out [F][<= OC], out as in
// LinearEpi. NW waves, NBUF chunks of weights in LDS.
template <bool BF16, int KC, int OC, int NW, int NBUF>
__global__ __launch_bounds__(NW * 64, 2) void k_gated_ffn(Operand X, Operand Wi, Operand Wo,
                                                          int64_t half, const float* __restrict__ b_in,
                                                          int64_t F, int64_t cout, int act, LinearEpi e) {
  constexpr int NT = NW * 64, FM = kWaveRows / 16, KS = KC / 32, OB = OC / 16, HB = kHidden / 16;
  using LI = LoadKRow<2 * kHidden, NT, true, false>;
  using LO = LoadOut<OC, NT>;
  using T = Tile<BF16, false, true, true, 128, 2 * kHidden, 1, 1, 2>;  // its operand reads
  constexpr int IN_BYTES = kStepK * 2 * kHidden * 2, TILE = KC / kStepK * IN_BYTES + kHidden * OC * 2;
  constexpr int ROWS = NW * kWaveRows, PH = ROWS * OC * 4 <= NBUF * TILE ? 1 : 2;
  using R = LdsRows<ROWS / PH, OC, NT>;
  constexpr int ROW_BYTES = R::PH_ROWS * OC * 4;
  __shared__ __attribute__((aligned(16))) char smem[NBUF * TILE > ROW_BYTES ? NBUF * TILE : ROW_BYTES];
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
  auto issue = [&](int c, int buf) {
    LI li;
    li.init(Wi, static_cast<int64_t>(c) * kHidden, half, tid);
#pragma unroll
    for (int q = 0; q < KC / kStepK; ++q)
      if (q * kStepK < X.k) li.issue(lds + buf * TILE + q * IN_BYTES, q * kStepK, X.k, wave);
    lo.issue(Wo, lds + buf * TILE + KC / kStepK * IN_BYTES, static_cast<int64_t>(c) * kHidden, wave);
  };

  float4v out[OB][FM];
#pragma unroll
  for (int j = 0; j < OB; ++j)
#pragma unroll
    for (int i = 0; i < FM; ++i) out[j][i] = float4v{};
  const uint32_t bias_bytes = b_in ? static_cast<uint32_t>(F) * 4u : 0u;
  const __amdgpu_buffer_rsrc_t rb[2] = {tile_rsrc(b_in, bias_bytes), tile_rsrc(b_in ? b_in + F : nullptr, bias_bytes)};
  if (NBUF == 2) issue(0, 0);
  with_act(act, [&](auto a) {
    for (int c = 0; c < chunks; ++c) {
      const int buf = NBUF == 2 ? c & 1 : 0;
      if constexpr (NBUF == 2) {
        // this chunk's weights have landed and all waves are past the last one
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (c + 1 < chunks) issue(c + 1, buf ^ 1);
      } else {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();  // all waves are past the last chunk
        asm volatile("" ::: "memory");
        issue(c, 0);
        wait_loads<0>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      const char* ti = smem + buf * TILE;
      const char* to = ti + KC / kStepK * IN_BYTES;
      // 32 hidden channels at a time: blocks 2 t, 2 t + 1 of gate and up
#pragma unroll
      for (int t = 0; t < HB / 2; ++t) {
        float4v acc[4][FM];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t n = c * kHidden + (2 * t + (j & 1)) * 16 + g * 4;
#pragma unroll
          for (uint32_t q = 0; q < 4; ++q) {
            const float b = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rb[j >> 1], (n + q) * 4u, 0, 0));
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[j][i][q] = b;
          }
        }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          if (kk * 32 >= X.k) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const half8 w = T::template frag<2 * kHidden, true>(
                ti + kk / 2 * IN_BYTES, (j >> 1) * kHidden + (2 * t + (j & 1)) * 16, kk & 1, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[j][i] = mfma16<BF16>(w, xf[kk][i], acc[j][i]);
          }
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
        for (int j = 0; j < OB; ++j) {
          const half8 w = LO::frag(to, j, t, lane);
#pragma unroll
          for (int i = 0; i < FM; ++i) out[j][i] = mfma16<BF16>(w, h[i], out[j][i]);
        }
      }
    }
  });

  // hidden channels past F are zeros in W_out's rows (and g = u = 0 there)
#pragma unroll 1
  for (int ph = 0; ph < PH; ++ph) {
    __syncthreads();
    if (PH == 1 || wave / (NW / PH) == ph) {
      const int r0 = wave % (NW / PH) * kWaveRows;
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

bool fused_ffn_takes(int64_t rows, int64_t cin, int64_t cout) {
  return cin <= 128 && cout <= 128 && rows >= 1;
}

int fused_ffn(const Mat16& x, const Mat16& W_in, int64_t F, const float* b_in, const Mat16& W_out,
              const float* b_out, int act, bool bf16, const uint16_t* residual, int64_t ldr,
              uint16_t* out, int64_t cout, hipStream_t stream) {
  constexpr int NW = 8, NBUF = 2, ROWS = NW * kWaveRows;
  const LinearEpi e{b_out, residual, ldr, out, cout, nullptr, kActNone,
                    cout % 8 == 0 && ldr % 8 == 0 && aligned16(residual),
                    cout % 8 == 0 && aligned16(out), false};
  const int64_t half = W_in.cols / 2;
  const Operand X{x.p, x.ld, x.rows, x.cols}, Wi{W_in.p, W_in.ld, half, W_in.rows};
  const Operand Wo{W_out.p, W_out.ld, W_out.cols, W_out.rows};
  const dim3 grid(static_cast<unsigned>(div_up(x.rows, ROWS)));
  auto go = [&](auto kc, auto oc) {
    if (bf16)
      k_gated_ffn<true, kc, oc, NW, NBUF><<<grid, NW * 64, 0, stream>>>(X, Wi, Wo, half, b_in, F, cout, act, e);
    else
      k_gated_ffn<false, kc, oc, NW, NBUF><<<grid, NW * 64, 0, stream>>>(X, Wi, Wo, half, b_in, F, cout, act, e);
  };
  using C64 = std::integral_constant<int, 64>;
  using C128 = std::integral_constant<int, 128>;
  if (x.cols <= 64 && cout <= 64) go(C64{}, C64{});
  else go(C128{}, C128{});
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}

}  // namespace submconv
