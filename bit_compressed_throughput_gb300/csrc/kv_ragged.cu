// Ragged K/V cache: rows of sequences of different lengths quantised into the 4-bit cache at
// each sequence's own position, and ranges of cached positions restored to fp16 rows (sm_103a).
//
// Rows row_off[b] .. row_off[b+1]-1 belong to sequence b and are positions pos[b], pos[b] + 1, ..
// The format is the cache's (include/fg.h): 64 consecutive channels of a row share (a, b), codes
// q = rint((x - a) 15 / (b - a)) in binary32, restored as fp16(a + q ((b - a) / 15)).
//
// Both are bound by HBM: 2 bytes of fp16 and 0.5625 bytes of codes and statistics per element.
// A CTA takes a tile of rows of K and V and some heads.  For one head the tile's codes are then
// one contiguous run of the head-major cache (per sequence), and its rows d contiguous values.
// The tile's sequences are looked up once (while the first rows load), then the CTA walks its heads
// with the next head's loads in flight.
//
// Measured (GB300, HBM copy 6.78 TB/s; calls one after another on other rows): 36 prompts of 400 ..
// 512 tokens, 96 heads, 1033 MB each: append 162 us (0.94), read-back 162 us (0.94); 16 prompts of
// 300 .. 512, 32 heads, 136 MB each: 28.5 us and 26.0 us (0.70 and 0.77; alone with cold caches,
// launch included, 36 and 30).  The append was bound by instructions before the codes were taken
// in fixed point and near ties fixed one by one (290 us at 96 heads with the packed-pair quantiser
// of the plain append on the same split).
#include <algorithm>

#include "fg_common.cuh"
#include "fg_internal.h"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_ragged_error = 0;

namespace {

constexpr int kThreads = 256;

struct RaggedArgs {
  const int32_t* row_off;
  const int32_t* pos;
  int rows, B, H, cap;
  int heads, hblocks;  // heads per CTA; CTAs per tile of rows
  int64_t stride;      // elements between the fp16 rows
};

// The sequence holding row r, found by a whole warp, 32 offsets at a time (the answers of
// sequence_of_row).
__device__ __forceinline__ int warp_sequence_of_row(const int32_t* off, int n, int r, int lane) {
  if (r < off[0] || r >= off[n]) return -1;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, i < hi && off[i] <= r);
    lo += max(__popc(le) - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Slots (b*H)*cap + position of the tile's ROWS rows from r0 on, -1 for rows that no sequence
// holds or that do not fit.  Every thread of the CTA calls it.
template <int ROWS>
__device__ __forceinline__ void tile_slots(const RaggedArgs& a, int r0, int64_t* slots) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 &&
      !offsets_ok(a.row_off, a.B, a.rows, threadIdx.x, kThreads))
    atomicOr(&g_ragged_error, kErrExtent);
  if (threadIdx.x < ROWS) {
    static_assert(ROWS % 32 == 0 && ROWS <= kThreads, "whole warps look rows up");
    const int row = r0 + threadIdx.x;
    // the warp's first row gives the sequence of most of its rows; the others search from there
    int b = warp_sequence_of_row(a.row_off, a.B, row - lane, lane);
    if (b < 0 || row >= a.row_off[b + 1]) {
      // one row a sequence (single tokens) puts this row `lane` sequences on
      const int c = b < 0 ? -1 : min(b + lane, a.B - 1);
      if (c >= 0 && a.row_off[c] <= row && row < a.row_off[c + 1])
        b = c;
      else
        b = row < a.rows ? sequence_of_row(a.row_off, a.B, row) : -1;
    }
    int64_t slot = -1;
    if (b >= 0 && row < a.rows) {
      const int64_t t = (int64_t)row - a.row_off[b];
      if (t >= 0 && row < a.row_off[b + 1]) {
        const int64_t p = a.pos[b] + t;
        if (a.pos[b] >= 0 && p < a.cap)
          slot = (int64_t)b * a.H * a.cap + p;
        else
          atomicOr(&g_ragged_error, kErrExtent);
      }
    }
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------- append

__device__ __forceinline__ uint32_t hmin2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmax2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t q4_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A group's 16 values per lane (8 words), 4 lanes per group, by the exact formulas: order keys for
// the minimum and maximum (signed zeros, NaN), the division for the codes.  The lanes of a group
// come here together.
__device__ __noinline__ uint2 quantize16_exact(uint4 v0, uint4 v1, unsigned group_lanes,
                                               uint32_t* ab_out) {
  const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
  uint32_t mm = __vminu2(q4_minmax8(w0), q4_minmax8(w1));
  mm = __vminu2(mm, __shfl_xor_sync(group_lanes, mm, 1));
  mm = __vminu2(mm, __shfl_xor_sync(group_lanes, mm, 2));
  *ab_out = q4_ab_word(mm);
  const Q4Group g = q4_group(*ab_out);
  if (g.bma == 0.0f) return make_uint2(0u, 0u);
  return make_uint2(q4_codes8_exact(v0, g.af, g.bma), q4_codes8_exact(v1, g.af, g.bma));
}

// Codes of 8 values in fixed point: with c15 = 15 / (b - a) and K = 192.5 + 2^-15 - a c15 held
// in [128, 256), one fused multiply-add gives x c15 + K = 192.5 + y + 2^-15 with a unit of 2^-16:
// bits 16-19 hold floor(y + 1/2) and the low 16 bits its fraction.  Errors, in that unit: 1/2 for
// rounding K, 1/2 for the fused sum, and 15 * 2^-22 relative (the reciprocal's 2^-23, two roundings
// of 2^-24) = 0.24 for c15, which multiplies x - a exactly; the defined code's own three roundings
// move it by at most 15 * 3 * 2^-24 = 0.18.  So the code is the defined one unless y lies within
// 1.42 units of a half-integer, when the fraction is 2 +- 1.42: below 4.  `frac` gathers the
// smallest fraction (16-bit lanes).
__device__ __forceinline__ void fixed2(uint32_t w, uint64_t c2, uint64_t k2, uint32_t (&t)[2]) {
  const float2 x = unpack_h2(w);
  float lo, hi;
  q4_unpack2(q4_fma2(q4_pack2(x.x, x.y), c2, k2), lo, hi);
  t[0] = __float_as_uint(lo);
  t[1] = __float_as_uint(hi);
}
__device__ __forceinline__ uint32_t codes8_fixed(const uint32_t (&w)[4], uint64_t c2, uint64_t k2,
                                                 uint32_t& frac) {
  uint32_t t[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    fixed2(w[i], c2, k2, t[i]);
    frac = __vminu2(frac, __byte_perm(t[i][0], t[i][1], 0x5410));
  }
  const uint32_t ev = __byte_perm(__byte_perm(t[0][0], t[1][0], 0x0062),
                                  __byte_perm(t[2][0], t[3][0], 0x0062), 0x5410);
  const uint32_t od = __byte_perm(__byte_perm(t[0][1], t[1][1], 0x0062),
                                  __byte_perm(t[2][1], t[3][1], 0x0062), 0x5410);
  return (ev & 0x0F0F0F0Fu) | ((od & 0x0F0F0F0Fu) << 4);
}
// The codes of 8 values with those near a half-integer taken by the division (a called function,
// out of the way of the code that calls it rarely).
__device__ __noinline__ uint32_t codes8_near(uint4 v, float c15, float K, float2 ab,
                                             uint32_t codes) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t c2 = q4_pack2(c15, c15), k2 = q4_pack2(K, K);
  const float width = __fsub_rn(ab.y, ab.x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t t[2];
    fixed2(w[i], c2, k2, t);
    const bool near0 = (t[0] & 0xFFFFu) < 4u, near1 = (t[1] & 0xFFFFu) < 4u;
    if (near0 || near1) {
      const float2 x = unpack_h2(w[i]);
      const int at = near0 ? 8 * i : 8 * i + 4;
      codes = (codes & ~(0xFu << at)) | (q4_code(near0 ? x.x : x.y, ab.x, width) << at);
      if (near0 && near1)
        codes = (codes & ~(0xF0u << at)) | (q4_code(x.y, ab.x, width) << (at + 4));
    }
  }
  return codes;
}

// Quantises the 16 values of this lane (4 lanes per group of 64): codes, and the group's (a, b).
// The fast path takes minimum and maximum as fp16 pairs and the codes in fixed point.  A group with
// a NaN, an infinity, a zero at either end (their order is by sign), a constant one, or one whose K
// leaves [128, 256) (its offset is more than four times its width) goes the exact way as a whole;
// codes near a tie do so alone (1 value in 4000 of normal data, exact ties of fp16 values; a lane
// of 1 warp in 8 has one).
__device__ __forceinline__ uint2 quantize16(const uint4 v0, const uint4 v1, int lane,
                                            uint32_t* ab_out) {
  const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
  uint32_t mn = hmin2_nan(w0[0], w0[1]), mx = hmax2_nan(w0[0], w0[1]);
  mn = hmin2_nan(mn, hmin2_nan(w0[2], w0[3]));
  mx = hmax2_nan(mx, hmax2_nan(w0[2], w0[3]));
  mn = hmin2_nan(mn, hmin2_nan(hmin2_nan(w1[0], w1[1]), hmin2_nan(w1[2], w1[3])));
  mx = hmax2_nan(mx, hmax2_nan(hmax2_nan(w1[0], w1[1]), hmax2_nan(w1[2], w1[3])));
  // (min, -max) in one word: a minimum merges both
  uint32_t mm = hmin2_nan(__byte_perm(mn, mx ^ 0x80008000u, 0x5410),
                          __byte_perm(mn, mx ^ 0x80008000u, 0x7632));
  mm = hmin2_nan(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 1));
  mm = hmin2_nan(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, 2));
  const uint32_t abw = mm ^ 0x80000000u;
  const float2 ab = unpack_h2(abw);
  const float c15 = 15.0f * rcp_approx(__fsub_rn(ab.y, ab.x));
  const float K = fmaf(-ab.x, c15, 192.5f + 0x1p-15f);
  const uint64_t c2 = q4_pack2(c15, c15), k2 = q4_pack2(K, K);
  uint32_t frac = 0xFFFFFFFFu;
  uint2 codes;
  codes.x = codes8_fixed(w0, c2, k2, frac);
  codes.y = codes8_fixed(w1, c2, k2, frac);
  // every comparison is false for NaN; c15 is 0 where b - a is infinite
  const bool plain = K >= 128.0f && K < 256.0f && c15 > 0.0f && c15 < INFINITY && ab.x != 0.0f &&
                     ab.y != 0.0f;
  const bool near = min(frac & 0xFFFFu, frac >> 16) < 4u;
  *ab_out = abw;
  if (__any_sync(0xFFFFFFFFu, !plain || near)) {
    if (!plain) {                          // the group's lanes agree
      codes = quantize16_exact(v0, v1, 0xFu << (lane & ~3), ab_out);
    } else if (near) {
      codes.x = codes8_near(v0, c15, K, ab, codes.x);
      codes.y = codes8_near(v1, c15, K, ab, codes.y);
    }
  }
  return codes;
}

// 4 lanes per group of 64, 16 values each: 16 * 256 / D rows per CTA.
template <int D>
__global__ void __launch_bounds__(kThreads, 4)
append_kernel(const RaggedArgs a, const uint16_t* __restrict__ k_new,
              const uint16_t* __restrict__ v_new, const fg_kvcache kv) {
  constexpr int ROWS = 16 * kThreads / D, LPR = D / 16, NG = D / 64;
  __shared__ int64_t slots[ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, r = threadIdx.x / LPR, c = threadIdx.x % LPR;
  const unsigned tile = blockIdx.x / a.hblocks;
  const int64_t r0 = (int64_t)tile * ROWS;
  const int h0 = (int)(blockIdx.x - tile * a.hblocks) * a.heads, h1 = min(a.H, h0 + a.heads);
  const bool held = r0 + r < a.rows;
  const int64_t at = held ? (r0 + r) * a.stride + c * 16 : 0;
  const uint16_t *ks = k_new + at, *vs = v_new + at;
  uint4 x[4];
  auto load = [&](int head) {
    if (held) {
      x[0] = ldg_nc_v4(ks + head * D);
      x[1] = ldg_nc_v4(ks + head * D + 8);
      x[2] = ldg_nc_v4(vs + head * D);
      x[3] = ldg_nc_v4(vs + head * D + 8);
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
  load(h0);                                // in flight while the rows' sequences are looked up
  tile_slots<ROWS>(a, (int)r0, slots);
  const int64_t slot0 = slots[r];
  const bool live = slot0 >= 0;
  for (int head = h0; head < h1; ++head) {
    const uint4 k0 = x[0], k1 = x[1], v0 = x[2], v1 = x[3];
    if (head + 1 < h1) load(head + 1);
    uint32_t kab, vab;
    const uint2 kc = quantize16(k0, k1, lane, &kab);
    const uint2 vc = quantize16(v0, v1, lane, &vab);
    if (live) {
      const int64_t slot = slot0 + (int64_t)head * a.cap;
      *reinterpret_cast<uint2*>(kv.k_codes + slot * (D / 2) + c * 8) = kc;
      *reinterpret_cast<uint2*>(kv.v_codes + slot * (D / 2) + c * 8) = vc;
      if ((c & 3) == 0) {
        kv.k_ab[slot * NG + (c >> 2)] = kab;
        kv.v_ab[slot * NG + (c >> 2)] = vab;
      }
    }
  }
}

// ---------------------------------------------------------------------------- read-back

// w / 15 rounded once (w finite and normal): the product with the rounded reciprocal, corrected by
// its remainder, which is exact (Markstein, 1990).  It equals the quotient for each of the 2^23
// mantissas of w (scaling by powers of two changes nothing).
__device__ __forceinline__ float div15(float w) {
  const float r = 1.0f / 15.0f, q = __fmul_rn(w, r);
  return __fmaf_rn(__fmaf_rn(-15.0f, q, w), r, q);
}
// The same values by the format's operations one by one (infinite or NaN statistics).
__device__ __noinline__ uint4 restore8_exact(uint32_t codes, float af, float s) {
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
__device__ __forceinline__ uint4 restore8(uint32_t codes, uint32_t abw) {
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

// 8 lanes per group of 64, 8 values each (a warp's stores are whole 32-byte sectors), two rows
// per thread.
template <int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(const RaggedArgs a, const fg_kvcache kv, uint16_t* __restrict__ k_out,
            uint16_t* __restrict__ v_out) {
  constexpr int ROWS = 16 * kThreads / D, LPR = D / 8, NG = D / 64, STEP = kThreads / LPR;
  __shared__ int64_t slots[ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int r = threadIdx.x / LPR, c = threadIdx.x % LPR;
  const unsigned tile = blockIdx.x / a.hblocks;
  const int64_t r0 = (int64_t)tile * ROWS;
  tile_slots<ROWS>(a, (int)r0, slots);
  const int h0 = (int)(blockIdx.x - tile * a.hblocks) * a.heads, h1 = min(a.H, h0 + a.heads);
  for (int head = h0; head < h1; ++head) {
    uint32_t code[2][2], ab[2][2];
    int64_t slot[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      slot[j] = slots[r + j * STEP];
      if (slot[j] < 0) continue;
      slot[j] += (int64_t)head * a.cap;
      if (k_out) {
        code[j][0] = *reinterpret_cast<const uint32_t*>(kv.k_codes + slot[j] * (D / 2) + c * 4);
        ab[j][0] = kv.k_ab[slot[j] * NG + (c >> 3)];
      }
      if (v_out) {
        code[j][1] = *reinterpret_cast<const uint32_t*>(kv.v_codes + slot[j] * (D / 2) + c * 4);
        ab[j][1] = kv.v_ab[slot[j] * NG + (c >> 3)];
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (slot[j] < 0) continue;
      const int64_t at = (r0 + r + j * STEP) * a.stride + (int64_t)head * D + c * 8;
      if (k_out) *reinterpret_cast<uint4*>(k_out + at) = restore8(code[j][0], ab[j][0]);
      if (v_out) *reinterpret_cast<uint4*>(v_out + at) = restore8(code[j][1], ab[j][1]);
    }
  }
}

// Heads per CTA: as many as leave the grid kCtasPerSm CTAs per SM, at most 8, so that the lookup
// of a tile's rows is shared; one when there are few tiles.
constexpr int kCtasPerSm = 16;
template <typename Kernel, typename... Args>
cudaError_t launch(Kernel* kernel, const int32_t* row_off, const int32_t* pos, int32_t rows,
                   int64_t stride, const fg_kvcache& kv, int nsm, cudaStream_t st, Args... args) {
  const int per = 16 * kThreads / (kv.h / kv.H);
  const int64_t tiles = ((int64_t)rows + per - 1) / per;
  const int heads =
      (int)std::max<int64_t>(1, std::min<int64_t>(8, tiles * kv.H / ((int64_t)nsm * kCtasPerSm)));
  const int hblocks = (kv.H + heads - 1) / heads;
  if (tiles * hblocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const RaggedArgs a{row_off, pos, rows, kv.B, kv.H, kv.cap, heads, hblocks, stride};
  return launch_pdl(kernel, dim3((unsigned)(tiles * hblocks)), dim3(kThreads), 0, st, a, args...);
}

}  // namespace

cudaError_t launch_kv_append_ragged(const uint16_t* k_new, const uint16_t* v_new,
                                    int64_t row_stride, int32_t rows, const int32_t* row_off,
                                    const int32_t* pos, const fg_kvcache& kv, int nsm,
                                    cudaStream_t st) {
  return launch(kv.h / kv.H == 128 ? append_kernel<128> : append_kernel<64>, row_off, pos, rows,
                row_stride, kv, nsm, st, k_new, v_new, kv);
}

cudaError_t launch_kv_read_ragged(const fg_kvcache& kv, const int32_t* row_off, const int32_t* pos,
                                  int32_t rows, uint16_t* k_out, uint16_t* v_out,
                                  int64_t row_stride, int nsm, cudaStream_t st) {
  return launch(kv.h / kv.H == 128 ? read_kernel<128> : read_kernel<64>, row_off, pos, rows,
                row_stride, kv, nsm, st, kv, k_out, v_out);
}

cudaError_t ragged_read_error(unsigned int* out) {
  return read_and_clear(g_ragged_error, out);
}

}  // namespace fg
