// Matrix-core fragments of packed group-32 rows and of activations, shared by
// the kernels of the dense projection (wave64, gfx950).
//
// v_mfma_f32_16x16x32_bf16: A lane l holds row l % 16, k = 8 (l / 16) .. + 7, B
// lane l column l % 16 at the same k, D lane l rows 4 (l / 16) + i of column
// l % 16.  The activations are A (rows = tokens), the weights B (columns = 16
// output rows), so a lane's four outputs belong to ONE weight row and take one
// scale.
//
// A code u becomes the exact bf16 number 1 + u / 16 (4-bit), 1 + u / 8 (3-bit) or
// 1 + u / 4 (2-bit) by OR-ing it into the top mantissa bits of 1.0; a bf16
// activation times it is exact in fp32.  The offset is taken off through the
// accumulator's input, C = -1.5 sum x (2-bit: -1 sum x), which one more product
// with a constant B makes in the layout in which it is needed:
//   4-bit: D = sum (u - 8) x / 16, 3-bit: D = sum (u - 4) x / 8, 2-bit: D = sum u x / 4
// and w x = F s D (+ m sum x), F = 16, 8, 4.
//
// The 32 codes of a group are four fragments of 8 codes; fragment f holds the
// elements 8f .. 8f + 7 in the pairs (j, j + 4) (4-bit) or 16 (f / 2) + 4 (f % 2)
// + {0..3} and the same + 8 in the pairs (j, j + 8) (3-bit, 2-bit): what a shift
// and a mask of the packed words give.  Activations are put in that order.
#pragma once

#include "gemv_tile.h"

namespace moe {

typedef __bf16 bf16x8_v __attribute__((ext_vector_type(8)));
typedef float f32x4_v __attribute__((ext_vector_type(4)));

template <int QF> constexpr float kOutFactor = QF == MOE_Q4_SYM_G32 ? 16.f : QF == MOE_Q3_SYM_G32 ? 8.f : 4.f;

struct __attribute__((aligned(16))) Frag { uint32_t d[4]; };

__device__ __forceinline__ f32x4_v mfma_frag(const Frag& a, const Frag& b, f32x4_v c) {
  const u32x4 av = {a.d[0], a.d[1], a.d[2], a.d[3]}, bv = {b.d[0], b.d[1], b.d[2], b.d[3]};
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_v, av), __builtin_bit_cast(bf16x8_v, bv), c,
                                                 0, 0, 0);
}

// B whose product with a fragment of x is the offset term: -1.5 (2-bit: -1) everywhere.
template <int QF>
__device__ __forceinline__ Frag offset_frag() {
  constexpr uint32_t v = QF == MOE_Q2_ASYM_G32 ? 0xBF80BF80u : 0xBFC0BFC0u;
  return Frag{{v, v, v, v}};
}

// The packed codes of one group, one word per fragment.
template <int QF>
__device__ __forceinline__ void frag_words(const typename CodeOf<QF>::T& c, uint32_t (&p)[4]) {
  if constexpr (QF == MOE_Q4_SYM_G32) {
#pragma unroll
    for (int f = 0; f < 4; ++f) p[f] = c[f];
  } else if constexpr (QF == MOE_Q2_ASYM_G32) {  // codes at bits 2j and 16 + 2j
#pragma unroll
    for (int f = 0; f < 4; ++f) p[f] = c[f >> 1] >> (8 * (f & 1));
  } else {  // low bits at 2j and 16 + 2j, third bits at 8 + j and 24 + j
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t t = __builtin_amdgcn_perm(0, c[2], d == 0 ? 0x0c010c00u : 0x0c030c02u);
      p[2 * d] = (c[d] & 0x00ff00ffu) | ((t << 8) & 0x0f000f00u);
      p[2 * d + 1] = ((c[d] >> 8) & 0x00ff00ffu) | ((t << 4) & 0x0f000f00u);
    }
  }
}

__device__ __forceinline__ uint32_t shift_to(uint32_t v, int by) { return by >= 0 ? v << by : v >> -by; }

// The unpacking's constants in registers: from literals the compiler makes a shift,
// an and and an or of every pair, from registers a shift and one v_and_or_b32.
template <int QF>
struct Unpack {
  uint32_t m0, m1, one;
  __device__ __forceinline__ Unpack() {
    constexpr uint32_t a = QF == MOE_Q4_SYM_G32 ? 0x00780078u : QF == MOE_Q2_ASYM_G32 ? 0x00600060u : 0x00300030u;
    asm("s_mov_b32 %0, %1" : "=s"(m0) : "i"(a));
    if constexpr (QF == MOE_Q3_SYM_G32) asm("s_mov_b32 %0, 0x00400040" : "=s"(m1));
    asm("v_mov_b32 %0, 0x3f803f80" : "=v"(one));
  }
  // One fragment's word to the bf16 numbers 1 + u / 2^bits.
  __device__ __forceinline__ Frag operator()(uint32_t p) const {
    Frag b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (QF == MOE_Q4_SYM_G32) b.d[j] = (shift_to(p, 3 - 4 * j) & m0) | one;
      else if constexpr (QF == MOE_Q2_ASYM_G32) b.d[j] = (shift_to(p, 5 - 2 * j) & m0) | one;
      else b.d[j] = (shift_to(p, -2 - j) & m1) | ((shift_to(p, 4 - 2 * j) & m0) | one);
    }
    return b;
  }
};

__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Parts of an activation: bf16 is one; fp32 is three bf16 numbers whose sum it
// is exactly (8 of the 24 significant bits each).
template <int ACT> constexpr int kParts = ACT == MOE_ACT_BF16 ? 1 : 3;

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2_v __attribute__((ext_vector_type(2)));
  const f32x2_v v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// The three bf16 parts of a pair of fp32 activations.
__device__ __forceinline__ void split3(float a, float b, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  p0 = bf16_pair(a, b);
  a -= __uint_as_float(p0 << 16);
  b -= __uint_as_float(p0 & 0xffff0000u);
  p1 = bf16_pair(a, b);
  a -= __uint_as_float(p1 << 16);
  b -= __uint_as_float(p1 & 0xffff0000u);
  p2 = bf16_pair(a, b);
}

// Half a group (16 elements) of one token, loaded as it lies, and its two
// fragments 2 h and 2 h + 1 in pair order (h = 0, 1 the half).
template <int ACT> struct XHalf { u32x4 v[ACT == MOE_ACT_BF16 ? 2 : 4]; };

template <int ACT>
__device__ __forceinline__ XHalf<ACT> load_half(const void* x, size_t at) {
  XHalf<ACT> r;
  const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(x) + at * (ACT == MOE_ACT_BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.v) / sizeof(r.v[0])); ++i) r.v[i] = p[i];
  return r;
}

// Runs of four elements i and i + gap (gap 1 run for 4-bit, 2 runs otherwise) pair up.
template <int QF>
__device__ __forceinline__ void half_frags(const XHalf<MOE_ACT_BF16>& r, Frag (&o)[2][1]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t a0, a1, b0, b1;  // the run's two words, its partner's
    if constexpr (QF == MOE_Q4_SYM_G32) {
      a0 = r.v[k][0]; a1 = r.v[k][1]; b0 = r.v[k][2]; b1 = r.v[k][3];
    } else {
      a0 = r.v[0][2 * k]; a1 = r.v[0][2 * k + 1]; b0 = r.v[1][2 * k]; b1 = r.v[1][2 * k + 1];
    }
    o[k][0].d[0] = pair_lo(a0, b0);
    o[k][0].d[1] = pair_hi(a0, b0);
    o[k][0].d[2] = pair_lo(a1, b1);
    o[k][0].d[3] = pair_hi(a1, b1);
  }
}
template <int QF>
__device__ __forceinline__ void half_frags(const XHalf<MOE_ACT_F32>& r, Frag (&o)[2][3]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const u32x4& ra = QF == MOE_Q4_SYM_G32 ? r.v[2 * k] : r.v[k];
    const u32x4& rb = QF == MOE_Q4_SYM_G32 ? r.v[2 * k + 1] : r.v[2 + k];
#pragma unroll
    for (int j = 0; j < 4; ++j) split3(__uint_as_float(ra[j]), __uint_as_float(rb[j]), o[k][0].d[j], o[k][1].d[j], o[k][2].d[j]);
  }
}

// Sum of the 16 elements.
__device__ __forceinline__ float half_sum(const XHalf<MOE_ACT_BF16>& r) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s = dot2_bf16(r.v[i][j], 0x3F803F80u, s);
  return s;
}
__device__ __forceinline__ float half_sum(const XHalf<MOE_ACT_F32>& r) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s += __uint_as_float(r.v[i][j]);
  return s;
}

// One fragment of one token: two runs of four elements, gap apart, the first at
// element frag_first of the group.
template <int QF> __device__ __forceinline__ int frag_first(int f) {
  return QF == MOE_Q4_SYM_G32 ? 8 * f : 16 * (f >> 1) + 4 * (f & 1);
}
template <int QF> constexpr int kFragGap = QF == MOE_Q4_SYM_G32 ? 4 : 8;

template <int QF>
__device__ __forceinline__ void load_frag(const void* x, size_t at, Frag (&o)[1]) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + at;
  const u32x2 a = *reinterpret_cast<const u32x2*>(p), b = *reinterpret_cast<const u32x2*>(p + kFragGap<QF>);
  o[0] = Frag{{pair_lo(a[0], b[0]), pair_hi(a[0], b[0]), pair_lo(a[1], b[1]), pair_hi(a[1], b[1])}};
}
template <int QF>
__device__ __forceinline__ void load_frag(const void* x, size_t at, Frag (&o)[3]) {
  const float* p = reinterpret_cast<const float*>(x) + at;
  const u32x4 ra = *reinterpret_cast<const u32x4*>(p), rb = *reinterpret_cast<const u32x4*>(p + kFragGap<QF>);
#pragma unroll
  for (int j = 0; j < 4; ++j) split3(__uint_as_float(ra[j]), __uint_as_float(rb[j]), o[0].d[j], o[1].d[j], o[2].d[j]);
}

// ---- weights

// Buffer descriptor of `bytes` bytes from p on: loads past the end give zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
constexpr int kNt = 2;  // cache policy of weights that are read once: past the caches

template <int QF, int NT = kNt>
__device__ __forceinline__ typename CodeOf<QF>::T buf_codes(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  if constexpr (QF == MOE_Q4_SYM_G32) return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, NT);
  else if constexpr (QF == MOE_Q3_SYM_G32) return __builtin_amdgcn_raw_buffer_load_b96(r, at, 0, NT);
  else return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, NT);
}

// 16 R rows x C groups of packed weights on their way from memory to the wave's
// own LDS.  A load takes 64 / C rows, C consecutive groups of each (whole cache
// lines); read back, a lane finds any group of its row.  LDS rows are padded so
// that 16 rows at the same group lie in different banks.
template <int QF, int R, int C, int NT = kNt>
struct Stage {
  using T = typename CodeOf<QF>::T;
  static constexpr int kB = CodeOf<QF>::kBytes;
  static constexpr int kSlot = QF == MOE_Q2_ASYM_G32 ? 8 : 16;  // bytes of a group
  static constexpr int kRow = C * kSlot + 16, kScale = 2 * C;
  static constexpr int kPlanes = QF == MOE_Q2_ASYM_G32 ? 2 : 1;
  static constexpr int kLoads = C / 4;                          // per 16 rows
  static constexpr int kBytes = 16 * R * (kRow + kPlanes * kScale);
  T c[R][kLoads];
  uint16_t s[R][kLoads], m[R][kLoads];

  // Groups [first, first + C) of the 16 R rows that start at group `at` of the matrix.
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t at, bool any, int lane) {
    const int G = a.K / kGroup;
    const int64_t all = (int64_t)a.N * G;
    const uint32_t left = any && at < all ? (uint32_t)min(all - at, (int64_t)1 << 26) : 0u;
    const auto rc = rsrc(a.codes + at * kB, left * kB);
    const auto rs = rsrc(a.scales + at, left * 2);
    const auto rm = rsrc(kPlanes == 2 ? a.mins + at : a.scales, kPlanes == 2 ? left * 2 : 0);
    const uint32_t mine = (uint32_t)((lane / C) * G + lane % C);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t g = mine + (uint32_t)((16 * r + (64 / C) * i) * G);
        c[r][i] = buf_codes<QF, NT>(rc, g * kB);
        s[r][i] = __builtin_amdgcn_raw_buffer_load_b16(rs, g * 2, 0, 0);
        if constexpr (kPlanes == 2) m[r][i] = __builtin_amdgcn_raw_buffer_load_b16(rm, g * 2, 0, 0);
      }
  }
  // `left` groups of the chunk are inside the row; the others get scale zero.
  __device__ __forceinline__ void put(char* lds, int left, int lane) const {
    const int lr = lane / C, lg = lane % C;
    const bool in = lg < left;
    char* sl = lds + 16 * R * kRow;
    wave_sync();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int row = 16 * r + (64 / C) * i + lr;
        *reinterpret_cast<T*>(lds + row * kRow + lg * kSlot) = c[r][i];
        *reinterpret_cast<uint16_t*>(sl + row * kScale + lg * 2) = in ? s[r][i] : 0;
        if constexpr (kPlanes == 2) *reinterpret_cast<uint16_t*>(sl + (16 * R + row) * kScale + lg * 2) = in ? m[r][i] : 0;
      }
    wave_sync();
  }
  // The lanes of a wave hand values over through LDS: the hardware keeps one
  // wave's LDS accesses in order, this keeps the compiler from reordering them.
  static __device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  static __device__ __forceinline__ const char* codes(const char* lds, int row, int g) { return lds + row * kRow + g * kSlot; }
  static __device__ __forceinline__ const char* scale(const char* lds, int row, int g, int plane = 0) {
    return lds + 16 * R * kRow + (plane * 16 * R + row) * kScale + 2 * g;
  }
};

// The word of fragment q of the group whose packed codes lie at p in LDS.
template <int QF>
__device__ __forceinline__ uint32_t lds_frag_word(const char* p, int q) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
  if constexpr (QF == MOE_Q4_SYM_G32) {
    return w[q];
  } else if constexpr (QF == MOE_Q2_ASYM_G32) {
    return w[q >> 1] >> (8 * (q & 1));
  } else {
    const uint32_t t = __builtin_amdgcn_perm(0, w[2], (q >> 1) ? 0x0c030c02u : 0x0c010c00u);
    return ((w[q >> 1] >> (8 * (q & 1))) & 0x00ff00ffu) | ((t << (8 - 4 * (q & 1))) & 0x0f000f00u);
  }
}

}  // namespace moe
