// Dense projection with packed group-32 weights: y = x W^T + bias.
//
// One wave per (output row, tile of kTok tokens): a lane takes every 64th
// group of the row, dequantises its 32 weights to fp32 and multiplies them
// with each token's activations; the lanes' sums meet in a wave reduction.
#include "moe_device.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kTok = 4;

template <int QF>
__device__ __forceinline__ void dequant32(const LinearArgs& a, int64_t row, int g, float (&w)[32]) {
  const int G = a.K / kGroup;
  const uint8_t* c = a.codes + (row * G + g) * (4 * code_bits(QF));
  const float s = f16_to_f32(a.scales[row * G + g]);
  const float m = QF == MOE_Q2_ASYM_G32 ? f16_to_f32(a.mins[row * G + g]) : 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if constexpr (QF == MOE_Q4_SYM_G32) {
      w[i] = s * (float)((int)((c[i / 2] >> (4 * (i & 1))) & 15) - 8);
    } else if constexpr (QF == MOE_Q3_SYM_G32) {
      const int u = ((c[i / 4] >> (2 * (i & 3))) & 3) | (((c[8 + i / 8] >> (i & 7)) & 1) << 2);
      w[i] = s * (float)(u - 4);
    } else {
      w[i] = fmaf(s, (float)((c[i / 4] >> (2 * (i & 3))) & 3), m);
    }
  }
}

template <int QF, int ACT>
__global__ __launch_bounds__(256) void k_linear(LinearArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= a.N) return;  // whole waves
  const int t0 = blockIdx.y * kTok, nt = min(kTok, a.T - t0);
  float acc[kTok] = {};
  for (int g = lane; g < a.K / kGroup; g += 64) {
    float w[32];
    dequant32<QF>(a, row, g, w);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      if (t < nt) {
        const size_t at = (size_t)(t0 + t) * a.ldx + g * kGroup;
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[t] = fmaf(w[i], load_act<ACT>(a.x, at + i), acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    const float v = wave_sum(acc[t]) + (a.bias ? a.bias[row] : 0.f);
    if (lane == 0 && t < nt) {
      const size_t at = (size_t)(t0 + t) * a.ldy + row;
      if (a.out == MOE_ACT_BF16) store_act<1>(a.y, at, v);
      else store_act<0>(a.y, at, v);
    }
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 3) / 4), 1);
  return by_qfmt(a.qfmt, [&](auto qf) {
    constexpr int QF = decltype(qf)::value;
    constexpr int kMaxY = 65535;
    for (int t0 = 0; t0 < a.T; t0 += kMaxY * kTok) {
      LinearArgs b = a;
      b.T = a.T - t0 < kMaxY * kTok ? a.T - t0 : kMaxY * kTok;
      b.x = reinterpret_cast<const char*>(a.x) + (size_t)t0 * a.ldx * (a.act == MOE_ACT_BF16 ? 2 : 4);
      b.y = reinterpret_cast<char*>(a.y) + (size_t)t0 * a.ldy * (a.out == MOE_ACT_BF16 ? 2 : 4);
      const dim3 gr(grid.x, (unsigned)((b.T + kTok - 1) / kTok));
      if (a.act == MOE_ACT_BF16) k_linear<QF, MOE_ACT_BF16><<<gr, 256, 0, s>>>(b);
      else k_linear<QF, MOE_ACT_F32><<<gr, 256, 0, s>>>(b);
    }
    return hipGetLastError();
  });
}

}  // namespace moe
