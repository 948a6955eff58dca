// Dense projection with packed group-32 weights, y = x W^T + bias (fragments and
// arithmetic: linear_frag.h).  Five kernels by the number of tokens T, all with
// whole cache lines of the weights per row and load, past the caches except for tiles:
//
// k_linear_one (T = 1, and a few tokens of a small matrix, token by token).  A lane
// is a group: it unpacks 32 codes and multiplies them with its 32 activations by
// v_dot2, 64 groups of a row a load.  Memory bounds it where the matrix is large:
// 131072 x 2048 4-bit 24.5 us, 6.2 TB/s (a plain read of as many bytes 6.4); 2048 x
// 2048 2.9 us, a launch and one trip to memory.
//
// k_linear_few (T = 2..4).  Matrix cores.  Products sum over the four lane rows,
// which hold four DIFFERENT groups: so the A operand is block diagonal, row
// 4 q + t = token t in the lanes of group q and zero elsewhere.  The products of
// the four fragments then add up to D[4 q + t] = the sum of group q for token t,
// in the very lane that has the group's scale: one scale and 4 scale FMAs for 32
// codes a lane.  x stays in LDS for the whole launch.  131072 x 2048 4-bit, T = 4: 30 us,
// 5 TB/s (16 rows of A with a token in each, zeros behind them: 71 us, the scale FMAs).
//
// k_linear_some (T = 5..16).  The tokens fill the 16 rows of A and the four lane
// rows hold one group: 4 scale FMAs for 8 codes a lane.  Up to 8 tokens the rows are
// the tokens twice, for two groups of two lane rows each, block diagonal as above: 4
// scale FMAs for 16 codes (16384 x 4096, T = 8 13.3 -> 11.9 us).  x stays in LDS.  Bound
// by the vector instructions of a wave's chain (unpack, scales, LDS) and by the start, x
// and the first weights: 65536 x 2048 2-bit, T = 5 17.9 us (2.9 TB/s); 50021 x 2016
// 3-bit, T = 13 24.3 us (1.9 TB/s).
//
// k_linear_tile (more tokens).  Tiles of 16 R rows a wave and 16 TT tokens, x
// staged chunk by chunk; S parts of the waves split K and join in LDS.  Four scale FMAs
// and three instructions of unpacking go with each MFMA, so the vector unit has more to
// issue than the matrix cores: 1000 x 2048 x 8192 4-bit 61 us, 0.55 PFLOP/s, 63 % of it
// in the products.  With one block a CU the loads, x's staging and the products follow
// each other: 64 x 4096 x 16384 24 us.  Tiles of 32 x 128 a wave 62 against 64 us at T =
// 1000, of 64 x 64 the same: no gain.
//
// k_linear_mid: as k_linear_some with x read from the caches, the block's waves
// splitting K: few rows, or x too large for LDS.  2048 x 2048 4-bit, T = 16 5.7 us: the
// waves' start, one trip to memory and the join.
#include "linear_frag.h"

namespace moe {
namespace {

constexpr int kChunk = 16;             // groups staged at once by the kernels with x in LDS
constexpr size_t kLds = 160 * 1024;    // of a CU
constexpr int kCus = 256;

__device__ __forceinline__ void store_y(const LinearArgs& a, int t, int row, float v) {
  if (a.bias) v += a.bias[row];
  const size_t at = (size_t)t * a.ldy + row;
  if (a.out == MOE_ACT_BF16) store_act<1>(a.y, at, v);
  else store_act<0>(a.y, at, v);
}

// ---------------------------------------------------------------- one token
// LR lanes a row (64 / LR rows a load), NR loads in flight.
template <int QF, int ACT, int LR, int NR>
__global__ __launch_bounds__(256) void k_linear_one(LinearArgs a) {
  constexpr int RPI = 64 / LR, kB = CodeOf<QF>::kBytes;
  constexpr int kPlanes = QF == MOE_Q2_ASYM_G32 ? 2 : 1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane / LR, gl = lane % LR;
  const int G = a.K / kGroup;
  const int row0 = (blockIdx.x * 4 + wave) * (NR * RPI);
  if (row0 >= a.N) return;
  const int t = blockIdx.y;
  const size_t x0 = (size_t)t * a.ldx;
  const int64_t at = (int64_t)row0 * G, all = (int64_t)a.N * G;
  const uint32_t left = (uint32_t)min(all - at, (int64_t)1 << 26);
  const auto rc = rsrc(a.codes + at * kB, left * kB);
  const auto rs = rsrc(a.scales + at, left * 2);
  const auto rm = rsrc(kPlanes == 2 ? a.mins + at : a.scales, kPlanes == 2 ? left * 2 : 0);
  const Unpack<QF> unpack;
  float acc[NR] = {};
  for (int g0 = 0; g0 < G; g0 += LR) {
    const bool in = g0 + gl < G;
    const int g = in ? g0 + gl : G - 1;
    XHalf<ACT> xr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) xr[h] = load_half<ACT>(a.x, x0 + (size_t)g * kGroup + 16 * h);
    typename CodeOf<QF>::T c[NR];
    uint16_t s[NR], m[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint32_t o = (uint32_t)((r * RPI + sub) * G + g);
      c[r] = buf_codes<QF>(rc, o * kB);
      s[r] = __builtin_amdgcn_raw_buffer_load_b16(rs, o * 2, 0, 0);
      if constexpr (kPlanes == 2) m[r] = __builtin_amdgcn_raw_buffer_load_b16(rm, o * 2, 0, 0);
    }
    const float sx = half_sum(xr[0]) + half_sum(xr[1]);
    Frag x[2][2][1];
    if constexpr (ACT == MOE_ACT_BF16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) half_frags<QF>(xr[h], x[h]);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      uint32_t words[4];
      frag_words<QF>(c[r], words);
      // bf16 x: the offset first; fp32 x: off every code, which is exact and keeps fp32's last bits
      constexpr float kOff = QF == MOE_Q2_ASYM_G32 ? 1.f : 1.5f;
      float d = ACT == MOE_ACT_BF16 ? -kOff * sx : 0.f;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const Frag b = unpack(words[f]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (ACT == MOE_ACT_BF16) {
            d = dot2_bf16(b.d[j], x[f >> 1][f & 1][0].d[j], d);
          } else {
            const u32x4& xa = QF == MOE_Q4_SYM_G32 ? xr[f >> 1].v[2 * (f & 1)] : xr[f >> 1].v[f & 1];
            const u32x4& xb = QF == MOE_Q4_SYM_G32 ? xr[f >> 1].v[2 * (f & 1) + 1] : xr[f >> 1].v[2 + (f & 1)];
            d = fmaf(__uint_as_float(b.d[j] << 16) - kOff, __uint_as_float(xa[j]), d);
            d = fmaf(__uint_as_float(b.d[j] & 0xffff0000u) - kOff, __uint_as_float(xb[j]), d);
          }
        }
      }
      acc[r] = fmaf(in ? f16_to_f32(s[r]) : 0.f, d, acc[r]);
      if constexpr (kPlanes == 2) acc[r] = fmaf(in ? 0.25f * f16_to_f32(m[r]) : 0.f, sx, acc[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = row0 + r * RPI + sub;
    const float v = seg_sum(acc[r], LR);
    if (gl == 0 && row < a.N) store_y(a, t, row, kOutFactor<QF> * v);
  }
}

template <int QF, int ACT, int LR>
hipError_t run_one(const LinearArgs& a, hipStream_t s) {
  constexpr int RPI = 64 / LR;
  auto go = [&](auto nr) {
    constexpr int NR = decltype(nr)::value, rows = 4 * NR * RPI;
    k_linear_one<QF, ACT, LR, NR><<<dim3((unsigned)((a.N + rows - 1) / rows), (unsigned)a.T), 256, 0, s>>>(a);
    return hipGetLastError();
  };
  // rows a wave: few while the chip is not full, many once it is
  if ((int64_t)a.N * a.T <= 4096 * RPI) return go(std::integral_constant<int, 1>{});
  if ((int64_t)a.N * a.T <= 65536 * RPI) return go(std::integral_constant<int, 4>{});
  return go(std::integral_constant<int, 8>{});
}

// ---------------------------------------------------------------- two to four tokens
// Blocks of 4 waves; a unit is 16 rows; S waves share a unit and split K.
template <int QF, int ACT>
struct FewLds {
  static constexpr int P = kParts<ACT>;
  int Tp, kQ, x, zero, c0, part, total;  // byte offsets behind the waves' weights
  __host__ __device__ FewLds(int T, int chunks, int S) {
    Tp = T == 3 ? 4 : T;
    kQ = 17 * Tp * 16;  // 4 groups x 4 fragments x Tp tokens, padded
    x = 4 * Stage<QF, 1, kChunk>::kBytes;
    zero = x + P * chunks * 4 * kQ;
    c0 = zero + 64;
    part = c0 + chunks * kChunk * 16;
    total = part + (S > 1 ? 1024 : 0);
  }
};

template <int QF, int ACT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void k_linear_few(LinearArgs a, int S, int units) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using St = Stage<QF, 1, kChunk>;
  constexpr int P = kParts<ACT>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int G = a.K / kGroup, chunks = (G + kChunk - 1) / kChunk;
  const FewLds<QF, ACT> L(a.T, chunks, S);
  char* wl = lds + wave * St::kBytes;
  char* xl = lds + L.x;
  float* c0l = reinterpret_cast<float*>(lds + L.c0);
  float* part = reinterpret_cast<float*>(lds + L.part);
  const int tiles = 4 / S;  // units a block takes at a time
  const int first_c = chunks * (wave % S) / S, nc = chunks * (wave % S + 1) / S - first_c;
  const int first = blockIdx.x * tiles + wave / S, stride = gridDim.x * tiles;
  const int rounds = (units - 1 - (int)blockIdx.x * tiles) / stride + 1;  // the same for every wave of the block

  // x first, then the first weights: loads return in order, and x is wanted first
  St w;
  const int nx = a.T * chunks * kChunk * 2;
  auto x_at = [&](int o, int* t, int* g) { *g = (o >> 1) % (chunks * kChunk); *t = (o >> 1) / (chunks * kChunk); };
  auto x_load = [&](int o) {
    int t, g;
    x_at(o, &t, &g);
    XHalf<ACT> r = {};
    if (o < nx && g < G) r = load_half<ACT>(a.x, (size_t)t * a.ldx + g * kGroup + 16 * (o & 1));
    return r;
  };
  constexpr int B = 2;
  XHalf<ACT> xb[B];
#pragma unroll
  for (int b = 0; b < B; ++b) xb[b] = x_load(threadIdx.x + b * 256);
  w.load(a, (int64_t)min(first, units - 1) * 16 * G + first_c * kChunk, true, lane);
  for (int o0 = threadIdx.x; o0 < nx; o0 += B * 256) {
    if (o0 >= B * 256) {
#pragma unroll
      for (int b = 0; b < B; ++b) xb[b] = x_load(o0 + b * 256);
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int o = o0 + b * 256;
      if (o >= nx) break;
      int t, g;
      x_at(o, &t, &g);
      Frag x[2][P];
      half_frags<QF>(xb[b], x);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<Frag*>(xl + (p * (chunks * 4) + (g >> 2)) * L.kQ + (((g & 3) * 4 + 2 * (o & 1) + k) * L.Tp + t) * 16) = x[k][p];
      const float sum = seg_sum(half_sum(xb[b]), 2);  // the two halves are neighbours
      if ((o & 1) == 0) c0l[g * 4 + t] = (QF == MOE_Q2_ASYM_G32 ? -1.f : -1.5f) * sum;
    }
  }
  for (int o = threadIdx.x; o < chunks * kChunk * 4; o += 256)
    if ((o & 3) >= a.T) c0l[o] = 0.f;
  if (threadIdx.x < 16) reinterpret_cast<uint32_t*>(lds + L.zero)[threadIdx.x] = 0;
  __syncthreads();
  const bool mine = (col >> 2) == q && (col & 3) < a.T;  // this lane of A is not zero
  const char* xr = mine ? xl + q * L.kQ + (col & 3) * 16 : lds + L.zero;
  const int xf = mine ? L.Tp * 16 : 16, xu = mine ? 4 * xf : 0, xc = mine ? 4 * L.kQ : 0, xp = mine ? chunks * 4 * L.kQ : 0;
  const Unpack<QF> unpack;

  for (int rd = 0; rd < rounds; ++rd) {
    const int unit = first + rd * stride;
    f32x4_v acc = {0.f, 0.f, 0.f, 0.f};
    for (int cc = 0; cc < nc; ++cc) {
      const int c = first_c + cc;
      w.put(wl, G - c * kChunk, lane);
      const bool end = cc + 1 == nc;
      if (!end || rd + 1 < rounds) {
        const int un = min(end ? unit + stride : unit, units - 1), cn = end ? first_c : c + 1;
        w.load(a, (int64_t)un * 16 * G + cn * kChunk, true, lane);
      }
      // step u: lane row q works on group 4 q + u of the chunk, whose four scales lie together
      const uint2 sc = *reinterpret_cast<const uint2*>(St::scale(wl, col, 4 * q));
      const uint2 mn = St::kPlanes == 2 ? *reinterpret_cast<const uint2*>(St::scale(wl, col, 4 * q, 1)) : uint2{0, 0};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        __builtin_amdgcn_sched_barrier(0);  // (reads of all four steps at once would cost an occupancy step of registers)
        Frag x[4][P];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int f = 0; f < 4; ++f) x[f][p] = *reinterpret_cast<const Frag*>(xr + c * xc + p * xp + u * xu + f * xf);
        const f32x4_v c0 = *reinterpret_cast<const f32x4_v*>(c0l + (c * kChunk + 4 * q + u) * 4);
        const auto codes = *reinterpret_cast<const typename CodeOf<QF>::T*>(St::codes(wl, col, 4 * q + u));
        uint32_t words[4];
        frag_words<QF>(codes, words);
        f32x4_v d = c0;
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const Frag b = unpack(words[f]);
#pragma unroll
          for (int p = 0; p < P; ++p) d = mfma_frag(x[f][p], b, d);
        }
        const uint32_t sw = u < 2 ? sc.x : sc.y;
        const float s = f16_to_f32((uint16_t)(u & 1 ? sw >> 16 : sw));
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, d[i], acc[i]);
        if constexpr (St::kPlanes == 2) {
          const uint32_t mw = u < 2 ? mn.x : mn.y;
          const float m = -0.25f * f16_to_f32((uint16_t)(u & 1 ? mw >> 16 : mw));
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(m, c0[i], acc[i]);
        }
      }
    }
    // the four groups of a step meet: sum over the lane rows; lane row t keeps token t
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u, v;
      swap16(__float_as_uint(acc[i]), &u, &v);
      const float h = __uint_as_float(u) + __uint_as_float(v);
      swap32(__float_as_uint(h), &u, &v);
      acc[i] = __uint_as_float(u) + __uint_as_float(v);
    }
    const float v = q == 0 ? acc[0] : q == 1 ? acc[1] : q == 2 ? acc[2] : acc[3];
    if (S == 1) {
      const int row = unit * 16 + col;
      if (q < a.T && row < a.N) store_y(a, q, row, kOutFactor<QF> * v);
    } else {
      __syncthreads();
      part[wave * 64 + lane] = v;
      __syncthreads();
      if ((int)threadIdx.x < tiles * 64) {
        const int row = ((int)blockIdx.x * tiles + wave + rd * stride) * 16 + col;
        float t = 0.f;
        for (int p = 0; p < S; ++p) t += part[(wave * S + p) * 64 + lane];
        if (q < a.T && row < a.N) store_y(a, q, row, kOutFactor<QF> * t);
      }
    }
  }
}

template <int QF, int ACT>
bool few_fits(const LinearArgs& a) {
  const int64_t chunks = (a.K / kGroup + kChunk - 1) / kChunk;
  return FewLds<QF, ACT>(a.T, (int)chunks, 4).total <= (int)kLds;
}
template <int QF, int ACT>
hipError_t run_few(const LinearArgs& a, hipStream_t s) {
  const int units = (a.N + 15) / 16, chunks = (a.K / kGroup + kChunk - 1) / kChunk;
  int S = 1;
  while (S < 4 && units * S < 2048 && 2 * S <= chunks) S *= 2;
  const int tiles = 4 / S, blocks = (units + tiles - 1) / tiles;
  k_linear_few<QF, ACT><<<blocks < 4 * kCus ? blocks : 4 * kCus, 256, FewLds<QF, ACT>(a.T, chunks, S).total, s>>>(a, S, units);
  return hipGetLastError();
}

// ---------------------------------------------------------------- five to sixteen tokens
// TB = 8 or 16 tokens at most.  A fragment of a group has TB + 1 slots of 16 bytes:
// the tokens', zero from token T on, and one that stays zero, which the rows of A past
// TB read.
template <int QF, int ACT, int W, int TB>
struct SomeLds {
  static constexpr int ts = (TB + 1) * 16;
  static constexpr int x = W * Stage<QF, 1, kChunk>::kBytes;
  static size_t total(int K) {
    const size_t nc = (K / kGroup + kChunk - 1) / kChunk;
    return x + kParts<ACT> * nc * kChunk * 4 * ts;
  }
};

template <int QF, int ACT, int W, int TB>
__global__ __launch_bounds__(64 * W) void k_linear_some(LinearArgs a, int units) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using St = Stage<QF, 1, kChunk>;
  using L = SomeLds<QF, ACT, W, TB>;
  constexpr int P = kParts<ACT>, ts = L::ts;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int G = a.K / kGroup, nc = (G + kChunk - 1) / kChunk;
  char* wl = lds + wave * St::kBytes;
  char* xl = lds + L::x;  // [part][group][fragment][slot]
  const int xpart = nc * kChunk * 4 * ts;
  const int first = blockIdx.x + wave * gridDim.x, stride = gridDim.x * W;  // (every CU the same number of waves)
  const int halves = nc * kChunk * 2;  // half groups of a token
  for (int o0 = threadIdx.x; o0 < a.T * halves; o0 += 4 * 64 * W) {
    XHalf<ACT> xb[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int o = o0 + b * 64 * W, t = o / halves, g = (o % halves) >> 1;
      xb[b] = XHalf<ACT>{};
      if (t < a.T && g < G) xb[b] = load_half<ACT>(a.x, (size_t)t * a.ldx + g * kGroup + 16 * (o & 1));
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int o = o0 + b * 64 * W, t = o / halves, g = (o % halves) >> 1;
      if (t >= a.T) break;
      Frag x[2][P];
      half_frags<QF>(xb[b], x);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<Frag*>(xl + p * xpart + (g * 4 + 2 * (o & 1) + k) * ts + t * 16) = x[k][p];
    }
  }
  for (int o = threadIdx.x; o < P * nc * kChunk * 4; o += 64 * W)
    for (int t = a.T; t <= TB; ++t) *reinterpret_cast<Frag*>(xl + o * ts + t * 16) = Frag{{0, 0, 0, 0}};
  St w;
  if (first < units) w.load(a, (int64_t)first * 16 * G, true, lane);
  __syncthreads();
  // kPair: lane rows 0, 1 hold one group, 2, 3 the next, two fragments each; else one group, a fragment each
  constexpr bool kPair = TB == 8;
  constexpr int kStep = kPair ? 2 : 1;  // groups (and fragments of a lane) a step
  const int gq = kPair ? q >> 1 : 0, f0 = kPair ? 2 * (q & 1) : q;
  const int slot = !kPair ? col : (col >> 3) == gq ? col & 7 : TB;
  const char* xr = xl + (gq * 4 + f0) * ts + slot * 16;
  const Frag off = offset_frag<QF>();
  const Unpack<QF> unpack;

  for (int unit = first; unit < units; unit += stride) {
    f32x4_v acc = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < nc; ++c) {
      w.put(wl, G - c * kChunk, lane);
      const bool end = c + 1 == nc;
      if (!end || unit + stride < units)
        w.load(a, (int64_t)(end ? unit + stride : unit) * 16 * G + (end ? 0 : c + 1) * kChunk, true, lane);
      const char* xc = xr + c * (kChunk * 4 * ts);
#pragma unroll
      for (int g4 = 0; g4 < kChunk; g4 += 4) {
        const uint2 sc = *reinterpret_cast<const uint2*>(St::scale(wl, col, g4));
        const uint2 mn = St::kPlanes == 2 ? *reinterpret_cast<const uint2*>(St::scale(wl, col, g4, 1)) : uint2{0, 0};
#pragma unroll
        for (int u = 0; u < 4; u += kStep) {
          Frag x[P][kStep];
          f32x4_v c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int f = 0; f < kStep; ++f) {
              x[p][f] = *reinterpret_cast<const Frag*>(xc + p * xpart + ((g4 + u) * 4 + f) * ts);
              c0 = mfma_frag(x[p][f], off, c0);
            }
          f32x4_v d = c0;
#pragma unroll
          for (int f = 0; f < kStep; ++f) {
            const Frag b = unpack(lds_frag_word<QF>(St::codes(wl, col, g4 + u + gq), f0 + f));
#pragma unroll
            for (int p = 0; p < P; ++p) d = mfma_frag(x[p][f], b, d);
          }
          auto plane = [&](const uint2& v) {  // of the lane's group
            const uint32_t w = u < 2 ? v.x : v.y;
            return f16_to_f32((uint16_t)(kPair ? w >> (16 * gq) : u & 1 ? w >> 16 : w));
          };
          const float s = plane(sc);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, d[i], acc[i]);
          if constexpr (St::kPlanes == 2) {
            const float m = -0.25f * plane(mn);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(m, c0[i], acc[i]);
          }
        }
      }
    }
    const int row = unit * 16 + col;
#pragma unroll
    for (int i = 0; i < 4; ++i)
    {
      float v = acc[i];
      if constexpr (kPair) {  // the other groups' sum
        uint32_t lo, hi;
        swap32(__float_as_uint(v), &lo, &hi);
        v = __uint_as_float(lo) + __uint_as_float(hi);
      }
      if (4 * q + i < a.T && row < a.N) store_y(a, 4 * q + i, row, kOutFactor<QF> * v);
    }
  }
}

template <int QF, int ACT, int W, int TB>
bool some_fits(const LinearArgs& a) { return SomeLds<QF, ACT, W, TB>::total(a.K) <= kLds; }
template <int QF, int ACT, int W, int TB>
hipError_t run_some(const LinearArgs& a, hipStream_t s) {
  const size_t lds = SomeLds<QF, ACT, W, TB>::total(a.K);
  const int units = (a.N + 15) / 16;
  int per = (int)(kLds / lds);  // blocks a CU holds
  if (per > 16 / W) per = 16 / W;
  k_linear_some<QF, ACT, W, TB><<<units < per * kCus ? units : per * kCus, 64 * W, lds, s>>>(a, units);
  return hipGetLastError();
}

// ---------------------------------------------------------------- token tiles
constexpr int kRowWaves = 4, kTileChunk = 8;  // waves of a part, groups of a chunk

template <int QF, int ACT, int R, int TT, int S>
struct TileLds {
  static constexpr int RW = kRowWaves, C = kTileChunk;
  static constexpr int kX = kParts<ACT> * C * TT * 1024;  // x of a chunk
  static constexpr int need = S * kX + RW * S * Stage<QF, R, C, 0>::kBytes;
  static constexpr int join = (S - 1) * RW * R * TT * 1024;
  static constexpr int total = need > join ? need : join;
  static_assert(total <= (int)kLds, "LDS");
};

template <int QF, int ACT, int R, int TT, int S, int OCC>
__global__ __launch_bounds__(64 * kRowWaves * S) __attribute__((amdgpu_waves_per_eu(OCC))) void k_linear_tile(LinearArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using L = TileLds<QF, ACT, R, TT, S>;
  constexpr int RW = kRowWaves, C = kTileChunk;
  using St = Stage<QF, R, C, 0>;  // (cached: other token tiles read the same rows)
  constexpr int P = kParts<ACT>, kXS = ACT == MOE_ACT_BF16 ? 2 : 4;
  constexpr int XF = TT * C / (2 * RW);    // half groups a thread stages
  constexpr int kTokStep = 32 * RW / C;    // tokens a pass of a part's threads covers
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave / RW, rw = wave % RW, col = lane & 15, q = lane >> 4;
  const int G = a.K / kGroup;
  const int row0 = (blockIdx.x * RW + rw) * (16 * R), tok0 = blockIdx.y * (16 * TT);
  const int chunks = (G + C - 1) / C, pc = (chunks + S - 1) / S, w0 = part * pc;  // chunks w0 .. w0 + pc - 1 are this part's
  char* xl = lds + part * L::kX;
  char* wl = lds + S * L::kX + wave * St::kBytes;

  St w;
  auto load_w = [&](int c) { w.load(a, (int64_t)row0 * G + (int64_t)(w0 + c) * C, c < pc && w0 + c < chunks, lane); };
  const int pt = threadIdx.x % (64 * RW), xh = pt & 1, xg = (pt >> 1) % C, xt = (pt >> 1) / C;
  uint32_t xo[XF];  // byte offsets, past the end for tokens that are not there
#pragma unroll
  for (int i = 0; i < XF; ++i) {
    const int t = xt + i * kTokStep;
    xo[i] = tok0 + t < a.T ? (uint32_t)((t * a.ldx + xg * kGroup + 16 * xh) * kXS) : 0x80000000u;
  }
  const auto xrs = rsrc(reinterpret_cast<const char*>(a.x) + (int64_t)tok0 * a.ldx * kXS,
                        (uint32_t)(((int64_t)(min(a.T - tok0, 16 * TT) - 1) * a.ldx + a.K) * kXS));
  XHalf<ACT> xr[XF];
  auto load_x = [&](int c, int i) {
    const bool in = c < pc && (w0 + c) * C + xg < G;
    const uint32_t o = in ? xo[i] + (uint32_t)(w0 + c) * (C * kGroup * kXS) : 0x80000000u;
#pragma unroll
    for (int k = 0; k < (int)(sizeof(xr[i].v) / 16); ++k) xr[i].v[k] = __builtin_amdgcn_raw_buffer_load_b128(xrs, o + 16 * k, 0, 0);
  };
  // a fragment's 16 tokens are rotated by a key of its half and group: writes (lanes
  // of many groups, one token) and reads (lanes of many tokens, one group) both
  // spread over the banks
  auto put_x = [&]() {
#pragma unroll
    for (int i = 0; i < XF; ++i) {
      const int t = xt + i * kTokStep;
      Frag x[2][P];
      half_frags<QF>(xr[i], x);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<Frag*>(xl + (((p * C + xg) * TT + (t >> 4)) * 64 + (2 * xh + k) * 16 + ((t & 15) ^ (xh * 8 + xg))) * 16) = x[k][p];
    }
  };

  f32x4_v acc[R][TT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) acc[r][tt] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const Frag off = offset_frag<QF>();
  const Unpack<QF> unpack;

#pragma unroll
  for (int i = 0; i < XF; ++i) load_x(0, i);
  load_w(0);
  for (int c = 0; c < pc; ++c) {
    if (c) __syncthreads();
    put_x();
    w.put(wl, G - (w0 + c) * C, lane);
    __syncthreads();
    load_w(c + 1);
#pragma unroll
    for (int g = 0; g < C; ++g) {
      // the next chunk's loads between the products (chunks past the last load nothing)
#pragma unroll
      for (int i = (g * XF + C - 1) / C; i < ((g + 1) * XF + C - 1) / C; ++i) load_x(c + 1, i);
      Frag x[TT][P];
      f32x4_v c0[TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        c0[tt] = f32x4_v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
          x[tt][p] = *reinterpret_cast<const Frag*>(xl + (((p * C + g) * TT + tt) * 64 + q * 16 + (col ^ ((q >> 1) * 8 + g))) * 16);
          c0[tt] = mfma_frag(x[tt][p], off, c0[tt]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const Frag b = unpack(lds_frag_word<QF>(St::codes(wl, 16 * r + col, g), q));
        const float s = f16_to_f32(*reinterpret_cast<const uint16_t*>(St::scale(wl, 16 * r + col, g)));
        float m = 0.f;
        if constexpr (St::kPlanes == 2) m = -0.25f * f16_to_f32(*reinterpret_cast<const uint16_t*>(St::scale(wl, 16 * r + col, g, 1)));
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          f32x4_v d = c0[tt];
#pragma unroll
          for (int p = 0; p < P; ++p) d = mfma_frag(x[tt][p], b, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][tt][i] = fmaf(s, d[i], acc[r][tt][i]);
          if constexpr (St::kPlanes == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][tt][i] = fmaf(m, c0[tt][i], acc[r][tt][i]);
          }
        }
      }
    }
  }
  if constexpr (S > 1) {  // parts meet: part 0 adds the others' sums, in order
    float* j = reinterpret_cast<float*>(lds);
    __syncthreads();
    if (part > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
          *reinterpret_cast<f32x4_v*>(j + ((((part - 1) * RW + rw) * R + r) * TT + tt) * 256 + lane * 4) = acc[r][tt];
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int p = 0; p < S - 1; ++p)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
          acc[r][tt] += *reinterpret_cast<const f32x4_v*>(j + (((p * RW + rw) * R + r) * TT + tt) * 256 + lane * 4);
  }
  auto write = [&](auto out) {
    constexpr int OUT = decltype(out)::value;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + 16 * r + col;
      const float bias = a.bias && row < a.N ? a.bias[row] : 0.f;
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = tok0 + 16 * tt + 4 * q + i;
          if (t < a.T && row < a.N) store_act<OUT>(a.y, (size_t)t * a.ldy + row, fmaf(kOutFactor<QF>, acc[r][tt][i], bias));
        }
    }
  };
  if (a.out == MOE_ACT_BF16) write(std::integral_constant<int, MOE_ACT_BF16>{});
  else write(std::integral_constant<int, MOE_ACT_F32>{});
}

template <int QF, int ACT, int R, int TT, int S, int OCC>
hipError_t run_tile(const LinearArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 16 * kRowWaves * R - 1) / (16 * kRowWaves * R)), (unsigned)((a.T + 16 * TT - 1) / (16 * TT)));
  k_linear_tile<QF, ACT, R, TT, S, OCC><<<grid, 64 * kRowWaves * S, TileLds<QF, ACT, R, TT, S>::total, s>>>(a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- few rows
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

constexpr int kMidWaves = 8;

template <int QF, int ACT>
__global__ __launch_bounds__(64 * kMidWaves) void k_linear_mid(LinearArgs a) {
  constexpr int kPlanes = QF == MOE_Q2_ASYM_G32 ? 2 : 1;
  __shared__ float part[kMidWaves * 256];  // [wave][16 tokens][16 rows]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int col = lane & 15, q = lane >> 4;
  const int row0 = blockIdx.x * 16, tok0 = blockIdx.y * 16;
  const int G = a.K / kGroup;
  const int steps = (G + 3) >> 2;  // of 4 groups
  const int j0 = steps * wave / waves, j1 = steps * (wave + 1) / waves;
  // rows past the last and tokens past the last are computed from the last and not stored
  const int64_t base = (int64_t)min(row0 + col, a.N - 1) * G;
  const size_t xat = (size_t)min(tok0 + col, a.T - 1) * a.ldx + frag_first<QF>(q);
  f32x4_v acc = {0.f, 0.f, 0.f, 0.f};
  const Frag off = offset_frag<QF>();
  const Unpack<QF> unpack;

  for (int j = j0; j < j1; ++j) {
    const int64_t g0 = base + min(4 * j + q, G - 1);  // a lane row loads one group of the four
    typedef typename CodeOf<QF>::T Code;
    typedef Code Loose __attribute__((aligned(4)));
    const Code c = *reinterpret_cast<const Loose*>(a.codes + g0 * CodeOf<QF>::kBytes);
    uint32_t words[4];
    float s[4], m[4];
    frag_words<QF>(c, words);
    transpose4(words);
    gather4(f16_to_f32(a.scales[g0]), s);
    if constexpr (kPlanes == 2) gather4(-0.25f * f16_to_f32(a.mins[g0]), m);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (4 * j + g < G) {  // the same for the whole wave
        Frag x[kParts<ACT>];
        load_frag<QF>(a.x, xat + (size_t)(4 * j + g) * kGroup, x);
        const Frag b = unpack(words[g]);
        f32x4_v c0 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p < kParts<ACT>; ++p) c0 = mfma_frag(x[p], off, c0);
        f32x4_v d = c0;
#pragma unroll
        for (int p = 0; p < kParts<ACT>; ++p) d = mfma_frag(x[p], b, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(s[g], d[i], acc[i]);
        if constexpr (kPlanes == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = fmaf(m[g], c0[i], acc[i]);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave * 256 + (4 * q + i) * 16 + col] = acc[i];
  __syncthreads();
  for (int o = threadIdx.x; o < 256; o += blockDim.x) {
    const int tok = tok0 + (o >> 4), row = row0 + (o & 15);
    if (tok >= a.T || row >= a.N) continue;
    float v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w * 256 + o];
    store_y(a, tok, row, kOutFactor<QF> * v);
  }
}

template <int QF, int ACT>
hipError_t run_mid(const LinearArgs& a, hipStream_t s) {
  constexpr int kMaxY = 65535;
  const int64_t bx = (a.N + 15) / 16;
  for (int t0 = 0; t0 < a.T; t0 += 16 * kMaxY) {
    LinearArgs b = a;
    b.T = a.T - t0 < 16 * kMaxY ? a.T - t0 : 16 * kMaxY;
    b.x = reinterpret_cast<const char*>(a.x) + (size_t)t0 * a.ldx * (ACT == MOE_ACT_BF16 ? 2 : 4);
    b.y = reinterpret_cast<char*>(a.y) + (size_t)t0 * a.ldy * (a.out == MOE_ACT_BF16 ? 2 : 4);
    const int64_t by = (b.T + 15) / 16;
    int waves = 1;  // enough on the chip, at least one step (4 groups) each
    while (waves < kMidWaves && bx * by * waves < 4096 && 2 * waves <= (a.K / kGroup + 3) / 4) waves *= 2;
    k_linear_mid<QF, ACT><<<dim3((unsigned)bx, (unsigned)by), 64 * waves, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  return by_qfmt(a.qfmt, [&](auto qf) {
    constexpr int QF = decltype(qf)::value;
    auto one = [&](auto act, const LinearArgs& b) {
      constexpr int ACT = decltype(act)::value;
      const int G = b.K / kGroup;
      if (G <= 8) return run_one<QF, ACT, 8>(b, s);
      if (G <= 32) return run_one<QF, ACT, 32>(b, s);
      return run_one<QF, ACT, 64>(b, s);
    };
    auto go = [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      // small enough that one trip to memory is all there is: token by token, every wave its own rows
      // (2048 x 2048: T = 4 4.8 -> 3.8 us, T = 8 5.4 -> 4.9; 4096 x 4096 at T = 4 8.0 against 6.9 the other way)
      if (a.T == 1 || (a.T <= (ACT == MOE_ACT_BF16 ? 16 : 4) && (int64_t)a.N * a.K * a.T <= (int64_t)1 << 25))
        return one(act, a);
      if (a.T <= 4) {
        if (few_fits<QF, ACT>(a)) return run_few<QF, ACT>(a, s);
        return one(act, a);  // x too large for LDS
      }
      if (a.T <= 16) {
        auto some = [&](auto tb) {
          constexpr int TB = decltype(tb)::value;
          if constexpr (TB == 16 && ACT == MOE_ACT_BF16) {  // one large block a CU (T = 13 3-bit 27.0 -> 24.4 us)
            if (some_fits<QF, ACT, 16, TB>(a)) return run_some<QF, ACT, 16, TB>(a, s);
          }
          if (some_fits<QF, ACT, 8, TB>(a)) return run_some<QF, ACT, 8, TB>(a, s);
          if (some_fits<QF, ACT, 4, TB>(a)) return run_some<QF, ACT, 4, TB>(a, s);
          return run_mid<QF, ACT>(a, s);
        };
        if (a.N >= 8192) return a.T <= 8 ? some(std::integral_constant<int, 8>{}) : some(std::integral_constant<int, 16>{});
        return run_mid<QF, ACT>(a, s);
      }
      if (64 * a.ldx * (ACT == MOE_ACT_BF16 ? 2 : 4) >= (int64_t)1 << 31) return run_mid<QF, ACT>(a, s);
      // By the number of tiles of 64 rows x 64 tokens.  More than one a CU: two row groups a wave, so that a block's
      // x serves 128 rows (64 x 50021 x 2592: 85.8 -> 52.7 us, 24576 rows 44.4 -> 40.5), with 48 tokens a tile where
      // that leaves fewer of them empty (T = 70, 44846 x 2592: 65.8 -> 56.1).  About one a CU: 128 rows x 32 tokens,
      // K split over two groups of waves (64 x 16384 x 4096: 28.3 us, of 64 x 64 30.6, without the split 52).  Fewer:
      // 16 tokens a tile, and K over four groups while those tiles leave the chip idle too (T = 64, 2048 x 2048: 6.5
      // us, over two 7.4; T = 128, 4096 x 4096: 20.5 against 17.6).
      const int64_t r64 = (a.N + 63) / 64, t64 = (a.T + 63) / 64, t48 = (a.T + 47) / 48;
      if constexpr (ACT == MOE_ACT_BF16) {
        if (r64 * ((a.T + 15) / 16) <= 320) return run_tile<QF, ACT, 1, 1, 4, 4>(a, s);
        if (r64 * t64 < 192) return run_tile<QF, ACT, 1, 1, 2, 4>(a, s);
        if (a.T <= 32) {  // (many rows: T = 20, 100000 x 2592 76.7 -> 66.1 us, 24576 24.5 against 25.7)
          return r64 <= 2 * kCus ? run_tile<QF, ACT, 1, 2, 2, 4>(a, s) : run_tile<QF, ACT, 1, 2, 1, 4>(a, s);
        }
        if (r64 * t64 <= kCus) return run_tile<QF, ACT, 2, 2, 2, 2>(a, s);
        if (48 * t48 * 8 <= 64 * t64 * 7) return run_tile<QF, ACT, 2, 3, 1, 2>(a, s);
        return run_tile<QF, ACT, 2, 4, 1, 2>(a, s);
      } else {
        // three parts of x a token: tiles of 128 x 32 (T = 500, 8192 x 2048: 78 us, of 64 x 32 with K split in two
        // 135), of 128 x 16 with K split in two (T = 39, 10122 x 3296: 51 -> 28), few: of 64 x 16, in four (T = 17,
        // 4974 x 7264: 60 -> 34)
        const int64_t tiles = r64 * ((a.T + 31) / 32);
        if (tiles < 192) return run_tile<QF, ACT, 1, 1, 4, 2>(a, s);
        if (tiles < 512) return run_tile<QF, ACT, 2, 1, 2, 2>(a, s);
        return run_tile<QF, ACT, 2, 2, 1, 2>(a, s);
      }
    };
    if (a.act == MOE_ACT_BF16) return go(std::integral_constant<int, MOE_ACT_BF16>{});
    return go(std::integral_constant<int, MOE_ACT_F32>{});
  });
}

}  // namespace moe
