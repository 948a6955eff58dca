// Dense projection with packed group-32 weights, y = x W^T + bias, on the matrix
// cores (fragments and arithmetic: linear_frag.h).
//
// Few tokens read every weight once and do little with it, so both kernels keep
// the weights out of LDS: a lane loads the whole group (16, 12 or 8 bytes) that
// it unpacks, 16 output rows x 4 groups a wave and load.
//
// k_linear_few (T <= 4).  The 64 lanes hold 4 DIFFERENT groups of 16 rows, and a
// product sums over all four: so the A operand is block diagonal, row 4 q + t =
// token t in the lanes of group q and zero elsewhere.  The four products of the
// four fragments then add up to D[4 q + t] = the sum of group q for token t, in
// the very lane that loaded the group and its scale: no lane exchange, one scale
// a lane and 4 scale FMAs for 32 codes.
//
// k_linear_mid (more tokens).  Tokens fill the 16 rows of A, so the four lanes of
// a row must hold the same group: the fragments' words are transposed over the
// four lane rows (4 swaps for 32 codes), the scales gathered (3 swaps).
//
// The waves of a block split the groups of the same rows and join in LDS, in wave
// order.
#include "linear_frag.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 8;

template <int QF> struct Weights {  // what a lane loads of one row tile: its group's codes and scale
  typename CodeOf<QF>::T c;
  uint16_t s, m;
};

template <int QF>
__device__ __forceinline__ void load_w(const LinearArgs& a, int64_t group, Weights<QF>& w) {
  using T = typename CodeOf<QF>::T;
  typedef T Loose __attribute__((aligned(4)));
  w.c = __builtin_nontemporal_load(reinterpret_cast<const Loose*>(a.codes + group * CodeOf<QF>::kBytes));
  w.s = __builtin_nontemporal_load(a.scales + group);
  if constexpr (QF == MOE_Q2_ASYM_G32) w.m = __builtin_nontemporal_load(a.mins + group);
}

__device__ __forceinline__ void store_y(const LinearArgs& a, int t, int row, float v) {
  if (a.bias) v += a.bias[row];
  const size_t at = (size_t)t * a.ldy + row;
  if (a.out == MOE_ACT_BF16) store_act<1>(a.y, at, v);
  else store_act<0>(a.y, at, v);
}

template <int QF, int ACT, int R>
__global__ __launch_bounds__(64 * kMaxWaves) void k_linear_few(LinearArgs a) {
  extern __shared__ float part[];  // [waves][16 R][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int col = lane & 15, q = lane >> 4;
  const int row0 = blockIdx.x * 16 * R;
  const int G = a.K / kGroup;
  const int steps = (G + 3) >> 2;  // of 4 groups
  const int j0 = steps * wave / waves, j1 = steps * (wave + 1) / waves;
  const int t = col & 3;
  const bool mine = (col >> 2) == q && t < a.T;  // this lane of A is not zero

  int64_t base[R];  // first group of the lane's row in each tile (clamped: such rows are not stored)
#pragma unroll
  for (int r = 0; r < R; ++r) base[r] = (int64_t)min(row0 + 16 * r + col, a.N - 1) * G;

  f32x4_v acc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const Frag off = offset_frag<QF>();

#pragma unroll 2
  for (int j = j0; j < j1; ++j) {
    const int g = 4 * j + q;
    const bool in = g < G;
    const int gc = in ? g : G - 1;
    XRaw<ACT> xr[4] = {};
    if (mine && in) {
#pragma unroll
      for (int f = 0; f < 4; ++f) load_x<QF>(a.x, (size_t)t * a.ldx + g * kGroup + frag_first<QF>(f), xr[f]);
    }
    Weights<QF> w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) load_w<QF>(a, base[r] + gc, w[r]);
    Frag x[4][kParts<ACT>];
#pragma unroll
    for (int f = 0; f < 4; ++f) x_frags(xr[f], x[f]);
    f32x4_v c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int p = 0; p < kParts<ACT>; ++p) c0 = mfma_frag(x[f][p], off, c0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint32_t words[4];
      frag_words<QF>(w[r].c, words);
      f32x4_v d = c0;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const Frag b = unpack_frag<QF>(words[f]);
#pragma unroll
        for (int p = 0; p < kParts<ACT>; ++p) d = mfma_frag(x[f][p], b, d);
      }
      const float s = in ? f16_to_f32(w[r].s) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(s, d[i], acc[r][i]);
      if constexpr (QF == MOE_Q2_ASYM_G32) {
        const float m = in ? -0.25f * f16_to_f32(w[r].m) : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(m, c0[i], acc[r][i]);
      }
    }
  }

  // the four groups of a step meet: sum over the lane rows
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u, v;
      swap16(__float_as_uint(acc[r][i]), &u, &v);
      const float h = __uint_as_float(u) + __uint_as_float(v);
      swap32(__float_as_uint(h), &u, &v);
      acc[r][i] = __uint_as_float(u) + __uint_as_float(v);
    }
  if (q == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[((wave * R + r) * 4 + i) * 16 + col] = acc[r][i];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < R * 64; o += blockDim.x) {  // o = (tile, token, row of the tile)
    const int r = o >> 6, tok = (o >> 4) & 3, row = row0 + 16 * r + (o & 15);
    if (tok >= a.T || row >= a.N) continue;
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w * R * 64 + o];
    store_y(a, tok, row, kOutFactor<QF> * v);
  }
}

// 4 x 4 transpose over (lane row of 16, register): p[g] of lane row q becomes p[q] of lane row g.
__device__ __forceinline__ void transpose4(uint32_t (&p)[4]) {
  auto s16 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = r[0]; y = r[1];
  };
  auto s32 = [](uint32_t& x, uint32_t& y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = r[0]; y = r[1];
  };
  s16(p[0], p[1]);
  s16(p[2], p[3]);
  s32(p[0], p[2]);
  s32(p[1], p[3]);
}
// o[g] = v of lane row g, in every lane row.
__device__ __forceinline__ void gather4(float v, float (&o)[4]) {
  uint32_t a, b, c, d, e, f;
  swap16(__float_as_uint(v), &a, &b);  // a = rows 0 0 2 2, b = rows 1 1 3 3
  swap32(a, &c, &d);
  swap32(b, &e, &f);
  o[0] = __uint_as_float(c); o[1] = __uint_as_float(e); o[2] = __uint_as_float(d); o[3] = __uint_as_float(f);
}

template <int QF, int ACT, int R, int TT>
__global__ __launch_bounds__(64 * kMaxWaves) void k_linear_mid(LinearArgs a) {
  extern __shared__ float part[];  // [waves][16 TT tokens][16 R rows]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int col = lane & 15, q = lane >> 4;
  const int row0 = blockIdx.x * 16 * R, tok0 = blockIdx.y * 16 * TT;
  const int G = a.K / kGroup;
  const int steps = (G + 3) >> 2;
  const int j0 = steps * wave / waves, j1 = steps * (wave + 1) / waves;

  int64_t base[R];
#pragma unroll
  for (int r = 0; r < R; ++r) base[r] = (int64_t)min(row0 + 16 * r + col, a.N - 1) * G;
  size_t xat[TT];  // tokens past the last read the last one's row and are not stored
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
    xat[tt] = (size_t)min(tok0 + 16 * tt + col, a.T - 1) * a.ldx + frag_first<QF>(q);

  f32x4_v acc[R][TT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[r][tt] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const Frag off = offset_frag<QF>();

  for (int j = j0; j < j1; ++j) {
    const int gq = min(4 * j + q, G - 1);
    Weights<QF> w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) load_w<QF>(a, base[r] + gq, w[r]);
    uint32_t words[R][4];
    float s[R][4], m[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      frag_words<QF>(w[r].c, words[r]);
      transpose4(words[r]);
      gather4(f16_to_f32(w[r].s), s[r]);
      if constexpr (QF == MOE_Q2_ASYM_G32) gather4(-0.25f * f16_to_f32(w[r].m), m[r]);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (4 * j + g < G) {  // the same for the whole wave
        Frag b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) b[r] = unpack_frag<QF>(words[r][g]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          XRaw<ACT> xr;
          load_x<QF>(a.x, xat[tt] + (4 * j + g) * kGroup, xr);
          Frag x[kParts<ACT>];
          x_frags(xr, x);
          f32x4_v c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < kParts<ACT>; ++p) c0 = mfma_frag(x[p], off, c0);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            f32x4_v d = c0;
#pragma unroll
            for (int p = 0; p < kParts<ACT>; ++p) d = mfma_frag(x[p], b[r], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][tt][i] = fmaf(s[r][g], d[i], acc[r][tt][i]);
            if constexpr (QF == MOE_Q2_ASYM_G32) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[r][tt][i] = fmaf(m[r][g], c0[i], acc[r][tt][i]);
            }
          }
        }
      }
    }
  }

  constexpr int kOut = 256 * R * TT;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave * kOut + (16 * tt + 4 * q + i) * 16 * R + 16 * r + col] = acc[r][tt][i];
  __syncthreads();
  for (int o = threadIdx.x; o < kOut; o += blockDim.x) {
    const int tok = tok0 + o / (16 * R), row = row0 + o % (16 * R);
    if (tok >= a.T || row >= a.N) continue;
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w * kOut + o];
    store_y(a, tok, row, kOutFactor<QF> * v);
  }
}

// Waves per block: enough waves on the chip, at least one step (4 groups) each.
int split_waves(int64_t blocks, int G, int most) {
  int w = 1;
  while (w < most && blocks * w < 4096 && 2 * w <= (G + 3) / 4) w *= 2;
  return w;
}

template <int QF, int ACT, int R>
hipError_t run_few(const LinearArgs& a, hipStream_t s) {
  const int64_t blocks = (a.N + 16 * R - 1) / (16 * R);
  const int waves = split_waves(blocks, a.K / kGroup, kMaxWaves);
  k_linear_few<QF, ACT, R><<<(unsigned)blocks, 64 * waves, waves * R * 64 * 4, s>>>(a);
  return hipGetLastError();
}

template <int QF, int ACT, int R, int TT>
hipError_t run_mid(const LinearArgs& a, hipStream_t s) {
  const int64_t bx = (a.N + 16 * R - 1) / (16 * R), by = (a.T + 16 * TT - 1) / (16 * TT);
  constexpr int most = 65536 / (1024 * R * TT) < kMaxWaves ? 65536 / (1024 * R * TT) : kMaxWaves;  // 64 KiB of LDS
  const int waves = split_waves(bx * by, a.K / kGroup, most);
  k_linear_mid<QF, ACT, R, TT><<<dim3((unsigned)bx, (unsigned)by), 64 * waves, waves * R * TT * 1024, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  return by_qfmt(a.qfmt, [&](auto qf) {
    constexpr int QF = decltype(qf)::value;
    auto go = [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if (a.T <= 4) return a.N > 16384 ? run_few<QF, ACT, 2>(a, s) : run_few<QF, ACT, 1>(a, s);
      if (a.T <= 16) return a.N > 16384 ? run_mid<QF, ACT, 4, 1>(a, s) : run_mid<QF, ACT, 1, 1>(a, s);
      if (a.T <= 32) return a.N > 8192 ? run_mid<QF, ACT, 4, 2>(a, s) : run_mid<QF, ACT, 2, 2>(a, s);
      return run_mid<QF, ACT, 4, 4>(a, s);
    };
    if (a.act == MOE_ACT_BF16) return go(std::integral_constant<int, MOE_ACT_BF16>{});
    return go(std::integral_constant<int, MOE_ACT_F32>{});
  });
}

}  // namespace moe
