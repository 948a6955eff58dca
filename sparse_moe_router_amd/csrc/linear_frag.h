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

struct Frag { uint32_t d[4]; };

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

// One fragment's word to the bf16 numbers 1 + u / 2^bits.
template <int QF>
__device__ __forceinline__ Frag unpack_frag(uint32_t p) {
  constexpr uint32_t one = 0x3F803F80u;
  Frag b;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (QF == MOE_Q4_SYM_G32) b.d[j] = (shift_to(p, 3 - 4 * j) & 0x00780078u) | one;
    else if constexpr (QF == MOE_Q2_ASYM_G32) b.d[j] = (shift_to(p, 5 - 2 * j) & 0x00600060u) | one;
    else b.d[j] = (shift_to(p, -2 - j) & 0x00400040u) | ((shift_to(p, 4 - 2 * j) & 0x00300030u) | one);
  }
  return b;
}

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

// Fragment f of one token's group in pair order; x at the group's first element.
// The two runs of four elements it takes start at first(f) and second(f).
template <int QF> __device__ __forceinline__ int frag_first(int f) {
  return QF == MOE_Q4_SYM_G32 ? 8 * f : 16 * (f >> 1) + 4 * (f & 1);
}
template <int QF> constexpr int kFragGap = QF == MOE_Q4_SYM_G32 ? 4 : 8;

template <int ACT> struct XRaw;
template <> struct XRaw<MOE_ACT_BF16> { u32x2 a, b; };
template <> struct XRaw<MOE_ACT_F32> { u32x4 a, b; };

template <int QF>
__device__ __forceinline__ void load_x(const void* x, size_t at, XRaw<MOE_ACT_BF16>& r) {
  const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + at;
  r.a = *reinterpret_cast<const u32x2*>(p);
  r.b = *reinterpret_cast<const u32x2*>(p + kFragGap<QF>);
}
template <int QF>
__device__ __forceinline__ void load_x(const void* x, size_t at, XRaw<MOE_ACT_F32>& r) {
  const float* p = reinterpret_cast<const float*>(x) + at;
  r.a = *reinterpret_cast<const u32x4*>(p);
  r.b = *reinterpret_cast<const u32x4*>(p + kFragGap<QF>);
}

__device__ __forceinline__ void x_frags(const XRaw<MOE_ACT_BF16>& r, Frag (&o)[1]) {
  o[0].d[0] = pair_lo(r.a[0], r.b[0]);
  o[0].d[1] = pair_hi(r.a[0], r.b[0]);
  o[0].d[2] = pair_lo(r.a[1], r.b[1]);
  o[0].d[3] = pair_hi(r.a[1], r.b[1]);
}
__device__ __forceinline__ void x_frags(const XRaw<MOE_ACT_F32>& r, Frag (&o)[3]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = __uint_as_float(r.a[j]), b = __uint_as_float(r.b[j]);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const uint32_t v = bf16_pair(a, b);
      o[p].d[j] = v;
      a -= __uint_as_float(v << 16);
      b -= __uint_as_float(v & 0xffff0000u);
    }
  }
}

}  // namespace moe
