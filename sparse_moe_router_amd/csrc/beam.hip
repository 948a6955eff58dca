// Beam search: the n best continuations of each sequence over beams and
// vocabulary, and the move of the beams' states to follow their parents.
//
// Selection, two kernels.  A row's vocabulary is cut into segments of 256
// consecutive tokens.
//
// k_beam_scan reads every logit once: a wave takes 2 U segments of a row and writes
// each segment's maximum and, over all of them, (m, sum exp(l - m)).  No
// selection happens here: the n best candidates of a sequence lie in the n
// segments whose maxima are best (in the order of the totals, equal ones by
// index: if n other segments come before a candidate's, each holds an element
// that comes before the candidate).  The sum is held, and exp evaluated, in 64
// bits: totals of different beams lie within 1e-7 of each other now and then, and
// a logarithm good to 1e-10 keeps them in order.  256 rows of 131072 fp32 logits (134
// MB): 29.5 us, 4.5 TB/s, bound by memory and the 64-bit exp about equally.  Segments of 512
// cost the pick more (24 beams, V 6035, 42 best 28 -> 22 us with 256).
//
// k_beam_pick, one block per sequence: top and sum of every beam, the n best segments,
// then the n best elements of those (read again, from the caches).  Latency bounds it:
// 1 sequence x 4 beams x 32768 8.4 us, 32 x 8 x 131072 12.4 us.  In cycles, of 21 000 at
// the former: start 1000, the beams' sums and logarithms 3200, an edge of the segments
// 1000, held and ranked 4000, the elements' loads 2000, their totals 1900, held and
// ranked 4000.  More blocks a sequence would need a third launch (2 us).
#include "moe_device.h"
#include "moe_internal.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSeg = 256;    // tokens of a segment
constexpr int kPiece = 512;  // tokens a wave reads at once: two segments

// ---------------------------------------------------------------- scan
struct BeamWs {
  double* sum;   // [rows][units]
  float* top;    // [rows][units]
  float* seg;    // [rows][segs] maxima
  int units, segs, pieces;
};

__host__ __device__ inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

__host__ __device__ inline BeamWs beam_ws(void* ws, int rows, int V, int U) {
  BeamWs w;
  w.segs = (V + kSeg - 1) / kSeg;
  w.pieces = (V + kPiece - 1) / kPiece;
  w.units = (w.pieces + U - 1) / U;
  char* p = reinterpret_cast<char*>(ws);
  w.sum = reinterpret_cast<double*>(p);
  p += up256((size_t)rows * w.units * 8);
  w.top = reinterpret_cast<float*>(p);
  p += up256((size_t)rows * w.units * 4);
  w.seg = reinterpret_cast<float*>(p);
  return w;
}

// exp(v - top) to 6e-11 (relative) for v <= top, top finite; what lies more than 700
// below counts e^-700, nothing next to the top's 1.  v - top = n ln 2 + y with |y| <=
// ln 2 / 2; e^y is the polynomial of degree 7 that meets it at the 8 Chebyshev nodes of
// |y| <= 0.34665 (5.6e-11 off at most); n goes into the exponent.  n comes as the low
// bits of n + 1.5 2^52, where the sum rounds to a whole number.  One conversion and 14
// operations in 64 bits: conversions and 32-bit steps between cost more than they save
// (20 operations and two more conversions: 34 us for 134 MB of fp32 logits against 30).
__device__ __forceinline__ double exp_below(float v, float top) {
  constexpr double kWhole = 6755399441055744.0;
  const double d = fmax((double)v - (double)top, -700.0);
  const double m = fma(d, 1.4426950408889634074, kWhole);
  const double y = fma(-(m - kWhole), 0.69314718055994530942, d);
  double p = 0.00019907597155120258;
  p = fma(p, y, 0.001394860471507592);
  p = fma(p, y, 0.008333283498489944);
  p = fma(p, y, 0.04166621792289689);
  p = fma(p, y, 0.16666666786439385);
  p = fma(p, y, 0.5000000107872163);
  p = fma(p, y, 0.9999999999955067);
  p = fma(p, y, 0.9999999999594902);
  return __hiloint2double(__double2hiint(p) + (__double2loint(m) << 20), __double2loint(p));
}

// Maximum over the 32 lanes of a half wave, in each of them.
__device__ __forceinline__ float half_max_f(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  v = fmaxf(v, dpp_f<kDppMirror>(v));
  uint32_t a, b;
  swap16(__float_as_uint(v), &a, &b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float both_halves_max_f(float v) {
  uint32_t a, b;
  swap32(__float_as_uint(v), &a, &b);
  return fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float wave_max_f(float v) { return both_halves_max_f(half_max_f(v)); }

template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  return v + __hiloint2double((int)dpp_u<CTRL>((uint32_t)__double2hiint(v)), (int)dpp_u<CTRL>((uint32_t)__double2loint(v)));
}
// Sum over the wave, the same bits in every lane.
__device__ __forceinline__ double wave_sum_d(double v) {
  v = add_dpp<kDppXor1>(v);
  v = add_dpp<kDppXor2>(v);
  v = add_dpp<kDppHalfMirror>(v);
  v = add_dpp<kDppMirror>(v);
  uint32_t h0, h1, l0, l1;
  swap16((uint32_t)__double2hiint(v), &h0, &h1);
  swap16((uint32_t)__double2loint(v), &l0, &l1);
  v = __hiloint2double((int)h0, (int)l0) + __hiloint2double((int)h1, (int)l1);
  swap32((uint32_t)__double2hiint(v), &h0, &h1);
  swap32((uint32_t)__double2loint(v), &l0, &l1);
  return __hiloint2double((int)h0, (int)l0) + __hiloint2double((int)h1, (int)l1);
}

// Bits of the allowed mask for n (4 or 8) tokens from v on (v a multiple of n).
__device__ __forceinline__ uint32_t allowed_bits(const BeamArgs& a, int row, int v) {
  return a.allowed[(size_t)row * a.ld_allowed + (v >> 5)] >> (v & 31);
}

// 8 logits of one lane of piece s: tokens s 512 + 4 lane + {0..3} and the same + 256
// (fp32) or s 512 + 8 lane + {0..7} (bf16); tokens that are not there or not
// allowed are -inf.  (+ 0 makes a negative zero positive: the two are equal.)
template <int ACT>
__device__ __forceinline__ void load_piece(const BeamArgs& a, int row, int s, int lane, float (&v)[8]) {
  constexpr int N = ACT == MOE_ACT_BF16 ? 8 : 4;
#pragma unroll
  for (int h = 0; h < 8 / N; ++h) {
    const int t = s * kPiece + 256 * h + N * lane;
    const size_t at = (size_t)row * a.ld + t;
    if (t + N <= a.V) {
      if constexpr (ACT == MOE_ACT_BF16) {
        typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
        const u32x4_any r = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_any*>(reinterpret_cast<const uint16_t*>(a.logits) + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(r[i] << 16);
          v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
      } else {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
        const f32x4_any r = __builtin_nontemporal_load(
            reinterpret_cast<const f32x4_any*>(reinterpret_cast<const float*>(a.logits) + at));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = r[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[N * h + i] = t + i < a.V ? load_act<ACT>(a.logits, at + i) : -INFINITY;
    }
    if (a.allowed && t < a.V) {
      const uint32_t bits = allowed_bits(a, row, t);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!((bits >> i) & 1)) v[N * h + i] = -INFINITY;
    }
  }
}

template <int ACT, int U>
__global__ __launch_bounds__(kThreads) void k_beam_scan(BeamArgs a, int64_t work) {
  const int lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (id >= work) return;
  const BeamWs w = beam_ws(a.ws, a.B * a.W, a.V, U);
  const int row = (int)(id / w.units), unit = (int)(id % w.units);
  if (a.finished && a.finished[row]) return;  // its one candidate needs no logits
  float v[U][8], top = -INFINITY;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = -INFINITY;
    if (unit * U + u < w.pieces) load_piece<ACT>(a, row, unit * U + u, lane, v[u]);
  }
  float mine = 0.f;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the maxima of the lane's first and last four (fmaxf passes over a NaN)
    float m0 = fmaxf(fmaxf(v[u][0], v[u][1]), fmaxf(v[u][2], v[u][3]));
    float m1 = fmaxf(fmaxf(v[u][4], v[u][5]), fmaxf(v[u][6], v[u][7]));
#pragma unroll
    for (int i = 0; i < 8; ++i) bad |= v[u][i] != v[u][i];
    // of the first segment in lanes 0..31, of the second in the others
    float m = fmaxf(m0, m1);
    if constexpr (ACT == MOE_ACT_F32) {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(m0), __float_as_uint(m1), false, false);
      m = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    }
    m = half_max_f(m);
    if ((lane & 31) == u) mine = m;
    top = fmaxf(top, m);
  }
  top = both_halves_max_f(top);
  const int seg = 2 * (unit * U + (lane & 31)) + (lane >> 5);
  if ((lane & 31) < U && seg < w.segs) w.seg[(size_t)row * w.segs + seg] = mine + 0.0f;
  double sum = 0.0;
  if (top > -INFINITY && top < INFINITY) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += exp_below(v[u][i], top);
    sum = wave_sum_d(sum);
  }
  bad = __any(bad) || top == INFINITY;
  if (lane == 0) {
    const size_t at = (size_t)row * w.units + unit;
    w.sum[at] = bad ? __longlong_as_double(0x7ff8000000000000ll) : sum;
    w.top[at] = top;
  }
}

// ---------------------------------------------------------------- pick
// Order-preserving map of a double (never NaN here); every real value is > 0.
__device__ __forceinline__ uint64_t order_key64(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key64_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// A candidate: the larger total first, equal totals by the lower index.  key 0: none.
struct Cand { uint64_t key; uint32_t idx; };
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.key > b.key || (a.key == b.key && a.idx < b.idx);
}

constexpr int kPick = 1024;  // threads of k_beam_pick
constexpr int kCap = 2048;  // candidates held between two rankings
struct Ranked {  // in order
  uint64_t key[128];
  uint32_t idx[128];
};
struct PickLds {
  uint64_t key[kCap];
  uint32_t idx[kCap];
  Ranked segments, out;
  uint32_t head[kPick / 4];
  uint32_t count, edge;
};

// The held candidates ranked (16 lanes each, counting those before it), the n first
// into `to`.  Returns how many there are.
__device__ __forceinline__ int rank_held(PickLds& L, Ranked& to, int n) {
  __syncthreads();
  const int m = (int)L.count;
  for (int i0 = 0; i0 < m; i0 += kPick / 16) {
    const int i = i0 + (int)(threadIdx.x >> 4);
    const Cand c{L.key[min(i, m - 1)], L.idx[min(i, m - 1)]};
    int r = 0;
#pragma unroll 2
    for (int j = threadIdx.x & 15; j < m; j += 16) r += before(Cand{L.key[j], L.idx[j]}, c);
    r += (int)dpp_u<kDppXor1>((uint32_t)r);
    r += (int)dpp_u<kDppXor2>((uint32_t)r);
    r += (int)dpp_u<kDppHalfMirror>((uint32_t)r);
    r += (int)dpp_u<kDppMirror>((uint32_t)r);
    if (i < m && r < n && (threadIdx.x & 15) == 0) { to.key[r] = c.key; to.idx[r] = c.idx; }
  }
  __syncthreads();
  return m < n ? m : n;
}

// Above this many candidates from a floor alone a first pass for a better edge costs less than ranking them (4 x 11
// beams, V 520, 18 best: the 18th best of 33 segments lets 8000 through; 178 -> 14 us).
constexpr int kFew = 384;
constexpr int kHeld = 8;  // values a thread holds: 8192 candidates are read once

// The n first of `total` candidates (load(i) the value from memory, cand(i, value)
// the candidate; different indices), in order, in `to`; returns how many there are.
// ready() runs once the first values are on their way.  floor: if not 0, at least n
// candidates are known to have keys with upper halves >= floor.
//   A first pass takes the best of every four threads, and of those a value that n of
// them reach: at least n candidates are as good, so nothing worse is held in the second
// pass (by the upper 32 bits of the key; usually little more than n candidates remain).  When
// the held ones do not fit, as with many equal totals, they are ranked 1024 at a
// time and only what comes before the n-th of them is held from there on.
template <typename Load, typename Ready, typename Make>
__device__ int block_select(PickLds& L, Ranked& to, int n, int total, uint32_t floor, Load&& load, Ready&& ready, Make&& cand) {
  constexpr int kBatch = kPick * kHeld;
  float v[kHeld];
  uint32_t h[kHeld];
  auto read = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      if (i0 + k * kPick >= total) break;  // (the same for the whole block)
      v[k] = load(min(i0 + k * kPick + (int)threadIdx.x, total - 1));
    }
  };
  auto heads = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      h[k] = 0;
      if (i0 + k * kPick >= total) continue;
      const int i = i0 + k * kPick + (int)threadIdx.x;
      if (i < total) h[k] = (uint32_t)(cand(i, v[k]).key >> 32);
    }
  };
  if (threadIdx.x == 0) { L.count = 0; L.edge = floor; }
  uint32_t best = 0;
  Cand last{0, 0xffffffffu};  // the n-th held so far
#pragma unroll 1
  for (int pass = floor ? 1 : 0; pass < 2; ++pass) {
    bool again = false;
    if (pass == 1) __syncthreads();
    const uint32_t edge = pass == 1 ? max(L.edge, 1u) : 0u;  // (key 0 is no candidate)
#pragma unroll 1
    for (int i0 = 0; i0 < total; i0 += kBatch) {
      if (pass == 0 || floor || total > kBatch) {
        read(i0);
        if (i0 == 0 && (pass == 0 || floor)) ready();
        heads(i0);
      }
      if (pass == 0) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) best = max(best, h[k]);
        continue;
      }
      uint32_t todo = 0;  // the values that pass the edge: few
#pragma unroll
      for (int k = 0; k < kHeld; ++k) todo |= (h[k] >= edge ? 1u : 0u) << k;
      auto take = [&](int k) {
        // v[k] by selects: with an index the compiler keeps v in LDS, at an address it works out from the
        // launch's packet in host memory (3000 cycles)
        const float a0 = k & 1 ? v[1] : v[0], a1 = k & 1 ? v[3] : v[2], a2 = k & 1 ? v[5] : v[4], a3 = k & 1 ? v[7] : v[6];
        const float b0 = k & 2 ? a1 : a0, b1 = k & 2 ? a3 : a2, val = k & 4 ? b1 : b0;
        const Cand c = cand(i0 + k * kPick + (int)threadIdx.x, val);
        if (before(c, last)) {
          const uint32_t at = atomicAdd(&L.count, 1u);
          if (at < (uint32_t)kCap) {
            L.key[at] = c.key;
            L.idx[at] = c.idx;
          }
        }
      };
      const uint32_t held = L.count;
      __syncthreads();
#pragma unroll 1
      for (uint32_t t = todo; t; t &= t - 1) take(__ffs((int)t) - 1);
      __syncthreads();
      if (floor && L.count > (uint32_t)kFew) {  // the floor lets too many through: ranking them costs more than a first pass
        again = true;
        break;
      }
      if (L.count <= (uint32_t)kCap) continue;  // (the same for the whole block)
      __syncthreads();
      if (threadIdx.x == 0) L.count = held;
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < kHeld; ++k) {
        if (L.count > kCap - kPick) {  // (the same for the whole block)
          const int k = rank_held(L, to, n);
          for (int i = threadIdx.x; i < k; i += kPick) { L.key[i] = to.key[i]; L.idx[i] = to.idx[i]; }
          if (threadIdx.x == 0) L.count = k;
          if (k == n) last = Cand{to.key[n - 1], to.idx[n - 1]};
        }
        __syncthreads();
        if ((todo >> k) & 1) take(k);
        __syncthreads();
      }
    }
    if (again) {
      __syncthreads();
      if (threadIdx.x == 0) { L.count = 0; L.edge = 0; }
      floor = 0;
      pass = -1;
    }
    if (pass == 0) {
      best = max(best, dpp_u<kDppXor1>(best));
      best = max(best, dpp_u<kDppXor2>(best));
      if ((threadIdx.x & 3) == 0) L.head[threadIdx.x >> 2] = best;
      __syncthreads();
      // the n-th best head or a little less, bit by bit below what all heads share
      if (threadIdx.x < 64) {
        const uint4 o = reinterpret_cast<const uint4*>(L.head)[threadIdx.x];
        const uint32_t hi = wave_max_u32(max(max(o.x, o.y), max(o.z, o.w)));
        auto least = [](uint32_t h) { return h ? h : 0xffffffffu; };  // (0: nothing there)
        const uint32_t lo = ~wave_max_u32(~min(min(least(o.x), least(o.y)), min(least(o.z), least(o.w))));
        auto count = [&](uint32_t t) {
          return __popcll(__ballot(o.x >= t)) + __popcll(__ballot(o.y >= t)) + __popcll(__ballot(o.z >= t)) +
                 __popcll(__ballot(o.w >= t));
        };
        uint32_t at = 0;  // n heads are at or above it
        if (hi == lo) {
          at = count(lo) >= n ? lo : 0;
        } else if (hi > lo && count(lo) >= n) {
          int bit = 31 - __clz((int)(hi ^ lo));
          at = (lo >> bit >> 1) << bit << 1;
#pragma unroll 1
          for (; bit >= 0; --bit) {
            const uint32_t t = at | 1u << bit;
            const int c = count(t);
            if (c >= n) at = t;
            if (c >= n && c <= n + 4) break;
          }
        }
        if (threadIdx.x == 0) L.edge = at;
      }
    }
  }
  return rank_held(L, to, n);
}

template <int ACT, int U>
__global__ __launch_bounds__(kPick) void k_beam_pick(BeamArgs a, uint64_t inv) {
  __shared__ __attribute__((aligned(16))) PickLds L;
  // a candidate's total is score + ((l - top) - ln sum exp(l - top)), in 64 bits: with top + ln sum rounded
  // first, a row of one large value (a mask's lowest value in every place) would lose the logarithm
  __shared__ double lse[64], score[64];  // the logarithm; NaN: the beam has no candidates
  __shared__ float peak[64];             // top
  __shared__ uint8_t over[64];           // finished beams
  const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const BeamWs w = beam_ws(a.ws, a.B * a.W, a.V, U);
  // inv = 2^40 / segs, rounded up: exact for i < 2^24 (i < W segs <= 2^22, segs <= 2^16)
  auto beam_of = [&](int i) { return (int)(((uint64_t)(uint32_t)i * inv) >> 40); };
  const double none = __longlong_as_double(0x7ff8000000000000ll);
  auto beams = [&]() {
    for (int i = wave; i < a.W; i += kPick / 64) {
      const int row = b * a.W + i;
      const float sc = a.scores[row];
      const bool fin = a.finished && a.finished[row];
      float top = -INFINITY;  // of the lane's units so far, and their sum relative to it
      double sum = 0.0;
      for (int u = lane; u < w.units; u += 64) {  // (a finished beam's are not written; its l is set below)
        const float t = w.top[(size_t)row * w.units + u];
        const double su = w.sum[(size_t)row * w.units + u];  // (0 for a unit of -inf, NaN for one with a NaN)
        const float m = fmaxf(top, t);
        sum = sum * exp_below(top, m) + su * exp_below(t, m);
        top = m;
      }
      const float all = wave_max_f(top);
      sum = wave_sum_d(sum * exp_below(top, all));
      double l = all > -INFINITY && all < INFINITY ? log(sum) : none;
      if (fin) l = 0.0;
      if (!(sc > -INFINITY && sc < INFINITY)) l = none;
      if (lane == 0) {
        lse[i] = l;
        peak[i] = fin ? 0.f : all;
        score[i] = (double)sc;
        over[i] = fin;
      }
    }
    __syncthreads();
  };
  auto total_key = [&](int beam, float v) -> uint64_t {
    const double l = lse[beam];
    if (l != l || v == -INFINITY) return 0;
    return order_key64(score[beam] + (((double)v - (double)peak[beam]) - l));
  };
  // the best segments: index beam * 2^16 + segment; a finished beam has its token's segment only
  const int n_seg = block_select(
      L, L.segments, a.n, a.W * w.segs, 0u,
      [&](int i) { return w.seg[(size_t)b * a.W * w.segs + i]; }, beams,
      [&](int i, float v) {
        const int beam = beam_of(i), seg = i - beam * w.segs;
        if (over[beam]) v = seg == a.eos / kSeg ? 0.f : -INFINITY;
        return Cand{total_key(beam, v), (uint32_t)(beam << 16 | seg)};
      });
  // the best of their elements: index beam * V + token (the maxima of n segments are n of them)
  const uint32_t floor = n_seg == a.n ? (uint32_t)(L.segments.key[a.n - 1] >> 32) : 0u;
  auto place = [&](int i) {  // (beam, token)
    const uint32_t g = L.segments.idx[i / kSeg];
    return make_int2((int)(g >> 16), (int)(g & 0xffffu) * kSeg + i % kSeg);
  };
  const int n_out = block_select(
      L, L.out, a.n, n_seg * kSeg, floor,
      [&](int i) {
        const int2 g = place(i);
        const int t = min(g.y, a.V - 1), row = b * a.W + g.x;
        const float v = load_act<ACT>(a.logits, (size_t)row * a.ld + t) + 0.0f;
        return a.allowed && !(allowed_bits(a, row, t) & 1) ? -INFINITY : v;
      },
      []() {},
      [&](int i, float v) {
        const int2 g = place(i);
        if (over[g.x]) v = g.y == a.eos ? 0.f : -INFINITY;
        return Cand{g.y < a.V ? total_key(g.x, v) : 0, (uint32_t)g.x * (uint32_t)a.V + (uint32_t)g.y};
      });
  for (int i = threadIdx.x; i < a.n; i += kPick) {
    const size_t at = (size_t)b * a.n + i;
    const bool have = i < n_out;
    a.out_score[at] = have ? (float)key64_value(L.out.key[i]) : -INFINITY;
    a.out_parent[at] = have ? (int)(L.out.idx[i] / (uint32_t)a.V) : -1;
    a.out_token[at] = have ? (int)(L.out.idx[i] % (uint32_t)a.V) : -1;
  }
}

// ---------------------------------------------------------------- reordering
constexpr int kStates = 32;          // states per launch: the descriptors travel as kernel arguments,
constexpr int kFewStates = 8;        // 2.2 KB of them, 0.6 KB where these are enough (a launch less than 1 us shorter)
constexpr int kMaxBlocks = 1 << 16;  // of one state and sequence

template <int NS>
struct StateArgs {
  moe_state s[NS];
  uint32_t end[NS];  // blocks up to and with this state
  const int32_t* parent;
  int64_t ldp;
  int W, n;
};

// A thread owns a column (the same B bytes of every row) of one sequence: it reads
// the column of all parents before it writes any, and nobody else touches that
// column, so dst may be src, and a row that is its own parent is left alone there.
// Block (x, sequence); x runs over the states' columns.
//   Bound by memory: 2 x the bytes moved (in place only what moves), a beam chosen
// twice read once, by the same thread.  The stores are non-temporal: lines that leave
// the caches early make room for the reads (610 MB into a second buffer 133 -> 125 us,
// 4.9 TB/s, where a copy reaches 5.1; 3 GB in place 600 -> 572, 10 MB 8.6 -> 7.0);
// non-temporal loads as well lose it again (144, 610, 8.2).
template <int B, int WB, int NS>
__global__ __launch_bounds__(kThreads) void k_reorder(StateArgs<NS> a) {
  // (16 bytes at any address: the hardware takes them, and rows of an odd length start anywhere)
  typedef uint32_t Words __attribute__((ext_vector_type(B >= 8 ? B / 4 : 2), aligned(1)));
  using V = std::conditional_t<B >= 8, Words, std::conditional_t<B == 4, uint32_t, std::conditional_t<B == 2, uint16_t, uint8_t>>>;
  int k = 0;
  while (k + 1 < a.n && blockIdx.x >= a.end[k]) ++k;
  const moe_state& s = a.s[k];
  const uint32_t first = k ? a.end[k - 1] : 0u;
  const int b = blockIdx.y;
  const bool same = s.src == s.dst;  // (a rest keeps this: both move by the same bytes)
  const char* src = reinterpret_cast<const char*>(s.src) + (int64_t)b * a.W * s.src_row_stride;
  char* dst = reinterpret_cast<char*>(s.dst) + (int64_t)b * a.W * s.dst_row_stride;
  const int64_t piece = s.chunk_bytes / B, total = s.chunks * piece;
  const int64_t step = (int64_t)(a.end[k] - first) * kThreads;
  const int32_t* parent = a.parent + b * a.ldp;
  for (int64_t c = (int64_t)(blockIdx.x - first) * kThreads + threadIdx.x; c < total; c += step) {
    int64_t pc = 0, off = c;
    if (s.chunks > 1) {
      if (total <= 0x7fffffff) {  // 32-bit division where it does
        pc = (uint32_t)c / (uint32_t)piece;
        off = (uint32_t)c % (uint32_t)piece;
      } else {
        pc = c / piece;
        off = c % piece;
      }
    }
    const char* from = src + pc * s.src_chunk_stride + off * B;
    char* to = dst + pc * s.dst_chunk_stride + off * B;
    V v[WB];
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      if (i < a.W) {
        const int p = parent[i];
        if ((uint32_t)p < (uint32_t)a.W && !(same && p == i)) v[i] = *reinterpret_cast<const V*>(from + p * s.src_row_stride);
      }
    }
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      if (i < a.W) {
        const int p = parent[i];
        if ((uint32_t)p < (uint32_t)a.W && !(same && p == i)) __builtin_nontemporal_store(v[i], reinterpret_cast<V*>(to + i * s.dst_row_stride));
      }
    }
  }
}

}  // namespace

size_t beam_ws_bytes(int B, int W, int V, int n, int act) {
  (void)n; (void)act;
  const size_t rows = (size_t)B * W, segs = (V + kSeg - 1) / kSeg, pieces = (V + kPiece - 1) / kPiece;  // a piece a unit
  return up256(rows * pieces * 8) + up256(rows * pieces * 4) + up256(rows * segs * 4);
}

hipError_t launch_beam_select(const BeamArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.B * a.W, segs = (a.V + kSeg - 1) / kSeg, pieces = (a.V + kPiece - 1) / kPiece;
  auto go = [&](auto act, auto u) {
    constexpr int ACT = decltype(act)::value, U = decltype(u)::value;
    const int64_t work = rows * ((pieces + U - 1) / U), blocks = (work + kThreads / 64 - 1) / (kThreads / 64);
    k_beam_scan<ACT, U><<<(unsigned)blocks, kThreads, 0, s>>>(a, work);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    k_beam_pick<ACT, U><<<(unsigned)a.B, kPick, 0, s>>>(a, (((uint64_t)1 << 40) + segs - 1) / segs);
    return hipGetLastError();
  };
  auto units = [&](auto act) {
    // four pieces a wave read 8 KiB at once; one while that leaves the chip idle
    if (rows * pieces >= 8192) return go(act, std::integral_constant<int, 4>{});
    return go(act, std::integral_constant<int, 1>{});
  };
  if (a.act == MOE_ACT_BF16) return units(std::integral_constant<int, MOE_ACT_BF16>{});
  return units(std::integral_constant<int, MOE_ACT_F32>{});
}

hipError_t launch_beam_reorder(const moe_state* states, int n, const int32_t* parent, int64_t ldp, int B, int W,
                               hipStream_t s) {
  // The widest column that every address, stride and size of a state allows.  A large state takes columns of 16
  // bytes all the same, at any address, and one of those for the rest of its pieces: a launch more (39 states of 213
  // rows of 66 bytes 66 -> 26 us).
  auto width = [&](const moe_state& st) {
    uint64_t all = reinterpret_cast<uintptr_t>(st.src) | reinterpret_cast<uintptr_t>(st.dst) | (uint64_t)st.chunk_bytes |
                   (uint64_t)st.src_row_stride | (uint64_t)st.dst_row_stride | (uint64_t)st.src_chunk_stride |
                   (uint64_t)st.dst_chunk_stride;
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
  };
  auto launch = [&](auto bytes, const auto& a, int blocks, int nb) {
    constexpr int BY = decltype(bytes)::value, NS = (int)(sizeof(a.s) / sizeof(a.s[0]));
    const dim3 grid((unsigned)blocks, (unsigned)nb);
    if (W <= 8) k_reorder<BY, 8, NS><<<grid, kThreads, 0, s>>>(a);
    else if (W <= 16) k_reorder<BY, 16, NS><<<grid, kThreads, 0, s>>>(a);
    else if (W <= 32) k_reorder<BY, 32, NS><<<grid, kThreads, 0, s>>>(a);
    else k_reorder<BY < 16 ? BY : 8, 64, NS><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
  };
  auto run = [&](auto bytes, const StateArgs<kStates>& a, int blocks, int nb) {
    if (a.n > kFewStates) return launch(bytes, a, blocks, nb);
    StateArgs<kFewStates> f{};
    for (int i = 0; i < a.n; ++i) {
      f.s[i] = a.s[i];
      f.end[i] = a.end[i];
    }
    f.parent = a.parent;
    f.ldp = a.ldp;
    f.W = a.W;
    f.n = a.n;
    return launch(bytes, f, blocks, nb);
  };
  for (int b0 = 0; b0 < B; b0 += 65535) {
    const int nb = B - b0 < 65535 ? B - b0 : 65535;
    for (const int bytes : {16, 4, 2, 1}) {  // one launch for up to kStates states of a width
      const int col = bytes == 16 && W > 32 ? 8 : bytes;
      StateArgs<kStates> a{};
      a.parent = parent + b0 * ldp;
      a.ldp = ldp;
      a.W = W;
      int64_t blocks = 0;
      for (int i = 0; i <= n; ++i) {
        if (i < n) {
          moe_state st = states[i];
          if (st.chunk_bytes == 0 || st.chunks == 0) continue;
          if (B * W == 1) st.src_row_stride = st.dst_row_stride = 0;
          if (st.chunks == 1) st.src_chunk_stride = st.dst_chunk_stride = 0;
          const int64_t wide = st.chunks * st.chunk_bytes < 8192 ? 0 : st.chunk_bytes / 16 * 16;
          if (wide == 0) {
            if (width(st) != bytes) continue;
          } else if (bytes == 16) {
            st.chunk_bytes = wide;
          } else {
            st.chunk_bytes -= wide;
            st.src = reinterpret_cast<const char*>(st.src) + wide;
            st.dst = reinterpret_cast<char*>(st.dst) + wide;
          }
          if (st.chunk_bytes == 0 || (wide && bytes < 16 && (width(st) < 4 ? width(st) : 4) != bytes)) continue;
          st.src = reinterpret_cast<const char*>(st.src) + (int64_t)b0 * W * st.src_row_stride;
          st.dst = reinterpret_cast<char*>(st.dst) + (int64_t)b0 * W * st.dst_row_stride;
          const int64_t want = (st.chunks * st.chunk_bytes / col + kThreads - 1) / kThreads;
          blocks += want < kMaxBlocks ? want : kMaxBlocks;
          a.s[a.n] = st;
          a.end[a.n++] = (uint32_t)blocks;
        }
        if (a.n == kStates || (i == n && a.n > 0)) {
          const hipError_t e = bytes == 16  ? run(std::integral_constant<int, 16>{}, a, (int)blocks, nb)
                               : bytes == 4 ? run(std::integral_constant<int, 4>{}, a, (int)blocks, nb)
                               : bytes == 2 ? run(std::integral_constant<int, 2>{}, a, (int)blocks, nb)
                                            : run(std::integral_constant<int, 1>{}, a, (int)blocks, nb);
          if (e != hipSuccess) return e;
          a.n = 0;
          blocks = 0;
        }
      }
    }
  }
  return hipSuccess;
}

}  // namespace moe
