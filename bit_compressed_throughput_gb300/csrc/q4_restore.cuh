// Values of the 4-bit format restored to fp16 as the format defines them, fp16(a + q ((b - a) / 15))
// with one binary32 rounding per operation, eight at a time (sm_103a).
#pragma once
#include <math.h>

#include "fg_common.cuh"

namespace fg {

__device__ __forceinline__ uint64_t q4_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// w / 15 rounded once (w finite and normal): the product with the rounded reciprocal, corrected by
// its remainder, which is exact (Markstein, 1990).  It equals the quotient for each of the 2^23
// mantissas of w (scaling by powers of two changes nothing).
__device__ __forceinline__ float div15(float w) {
  const float r = 1.0f / 15.0f, q = __fmul_rn(w, r);
  return __fmaf_rn(__fmaf_rn(-15.0f, q, w), r, q);
}
// The same values by the format's operations one by one (infinite or NaN statistics).
static __device__ __noinline__ uint4 restore8_exact(uint32_t codes, float af, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_h2(__fadd_rn(af, __fmul_rn((float)((codes >> (8 * i)) & 0xFu), s)),
                   __fadd_rn(af, __fmul_rn((float)((codes >> (8 * i + 4)) & 0xFu), s)));
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// The 8 values fp16(a + fl(q s)), s = fl((b - a) / 15), of a code word.  A code's bits under the
// exponent of 2^23 are the binary32 number 2^23 + q, and (2^23 + q) s - 2^23 s = q s exactly, so
// one fused multiply-add with the exact -2^23 s gives fl(q s); two values per instruction.
__device__ __forceinline__ uint4 restore8_fp16(uint32_t codes, uint32_t abw) {
  const float2 ab = unpack_h2(abw);
  const float s = div15(__fsub_rn(ab.y, ab.x)), c = -8388608.0f * s;
  if (!(s < INFINITY))                     // fp16 infinities or NaN
    return restore8_exact(codes, ab.x, __fdiv_rn(__fsub_rn(ab.y, ab.x), 15.0f));
  const uint32_t ev = codes & 0x0F0F0F0Fu, od = (codes >> 4) & 0x0F0F0F0Fu;
  const uint64_t a2 = q4_pack2(ab.x, ab.x), s2 = q4_pack2(s, s), c2 = q4_pack2(c, c);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(__byte_perm(ev, 0x4B000000u, 0x7440 + i));
    const float hi = __uint_as_float(__byte_perm(od, 0x4B000000u, 0x7440 + i));
    float x, y;
    q4_unpack2(q4_add2(a2, q4_fma2(q4_pack2(lo, hi), s2, c2)), x, y);
    o[i] = pack_h2(x, y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same with a group's constants computed once for many code words; `plain`: its statistics are
// finite (elsewhere the words take restore8_fp16).
struct GroupFp16 {
  uint64_t a2, s2, c2;
  bool plain;
  __device__ __forceinline__ explicit GroupFp16(uint32_t abw) {
    const float2 ab = unpack_h2(abw);
    const float s = div15(__fsub_rn(ab.y, ab.x)), c = -8388608.0f * s;
    a2 = q4_pack2(ab.x, ab.x);
    s2 = q4_pack2(s, s);
    c2 = q4_pack2(c, c);
    plain = s < INFINITY;
  }
  __device__ __forceinline__ uint4 restore(uint32_t codes) const {
    const uint32_t ev = codes & 0x0F0F0F0Fu, od = (codes >> 4) & 0x0F0F0F0Fu;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(__byte_perm(ev, 0x4B000000u, 0x7440 + i));
      const float hi = __uint_as_float(__byte_perm(od, 0x4B000000u, 0x7440 + i));
      float x, y;
      q4_unpack2(q4_add2(a2, q4_fma2(q4_pack2(lo, hi), s2, c2)), x, y);
      o[i] = pack_h2(x, y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// Two positions' values side by side: a word whose halves hold four codes of either position, as a
// transposition of 8 positions' code words leaves them, gives four pairs (of channel i: both
// positions).
static __device__ __noinline__ uint4 restore_pairs_exact(uint32_t codes, uint32_t ab0, uint32_t ab1) {
  const float2 x = unpack_h2(ab0), y = unpack_h2(ab1);
  const float sx = __fdiv_rn(__fsub_rn(x.y, x.x), 15.0f), sy = __fdiv_rn(__fsub_rn(y.y, y.x), 15.0f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_h2(__fadd_rn(x.x, __fmul_rn((float)((codes >> (4 * i)) & 0xFu), sx)),
                   __fadd_rn(y.x, __fmul_rn((float)((codes >> (16 + 4 * i)) & 0xFu), sy)));
  return make_uint4(o[0], o[1], o[2], o[3]);
}
struct PairsFp16 {
  uint64_t a2, s2, c2;
  bool plain;                              // the statistics are finite
  __device__ __forceinline__ PairsFp16(uint32_t ab0, uint32_t ab1) {
    const float2 x = unpack_h2(ab0), y = unpack_h2(ab1);
    const float sx = div15(__fsub_rn(x.y, x.x)), sy = div15(__fsub_rn(y.y, y.x));
    a2 = q4_pack2(x.x, y.x);
    s2 = q4_pack2(sx, sy);
    c2 = q4_pack2(-8388608.0f * sx, -8388608.0f * sy);
    plain = sx < INFINITY && sy < INFINITY;
  }
  __device__ __forceinline__ uint4 restore(uint32_t codes) const {
    const uint32_t ev = codes & 0x0F0F0F0Fu, od = (codes >> 4) & 0x0F0F0F0Fu;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i & 1 ? od : ev;
      const float lo = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + (i >> 1)));
      const float hi = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442 + (i >> 1)));
      float x, y;
      q4_unpack2(q4_add2(a2, q4_fma2(q4_pack2(lo, hi), s2, c2)), x, y);
      o[i] = pack_h2(x, y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

}  // namespace fg
