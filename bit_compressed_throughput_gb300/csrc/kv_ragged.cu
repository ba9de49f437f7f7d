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
#include "paged.cuh"
#include "q4_restore.cuh"
#include "ragged.cuh"
#include "rope.h"

namespace fg {

__device__ unsigned int g_ragged_error = 0;

namespace {

constexpr int kThreads = 256;

struct RaggedArgs {
  const int32_t* row_off;
  const int32_t* pos;
  int rows, B, H;
  int heads, hblocks;  // heads per CTA; CTAs per tile of rows
  int64_t stride;      // elements between the fp16 rows
};

// Where the 4-bit rows of a position lie: slot(b, p) numbers position p of sequence b (-1: it does
// not fit), cell(slot, head) is that head's part of it.
struct Cell {
  uint8_t *k_codes, *v_codes;
  uint32_t *k_ab, *v_ab;
};
struct Regions {                           // one region per (sequence, head)
  fg_kvcache kv;
  __device__ __forceinline__ int64_t slot(int b, int64_t p) const {
    return p < kv.cap ? (int64_t)b * kv.H * kv.cap + p : -1;
  }
  template <int D>
  __device__ __forceinline__ Cell cell(int64_t slot, int head) const {
    const int64_t s = slot + (int64_t)head * kv.cap;
    return Cell{kv.k_codes + s * (D / 2), kv.v_codes + s * (D / 2), kv.k_ab + s * (D / 64),
                kv.v_ab + s * (D / 64)};
  }
};
struct Pages {
  PagedCache pc;
  __device__ __forceinline__ int64_t slot(int b, int64_t p) const {
    return p < pc.cap() ? pc.slot(b, p) : -1;
  }
  template <int D>
  __device__ __forceinline__ Cell cell(int64_t slot, int head) const {
    uint8_t *k = pc.block(slot, head, D), *v = k + pc.half_bytes(D);
    const int64_t at = slot & ((1 << pc.lg) - 1), ab = (int64_t)(D / 2) << pc.lg;
    return Cell{k + at * (D / 2), v + at * (D / 2),
                reinterpret_cast<uint32_t*>(k + ab) + at * (D / 64),
                reinterpret_cast<uint32_t*>(v + ab) + at * (D / 64)};
  }
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

// place(b, t) of the tile's ROWS rows from r0 on, row t of sequence b, into slots; -1 for rows that
// no sequence holds or that do not fit (place < 0).  Every thread of the CTA calls it.
template <int ROWS, typename Place>
__device__ __forceinline__ void tile_slots(const RaggedArgs& a, int r0, int64_t* slots,
                                           Place place) {
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
        slot = place(b, t);
        if (slot < 0) atomicOr(&g_ragged_error, kErrExtent);
      }
    }
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------- rotary positions
//
// A row at position p turns pairs of a head's first `rot` channels, (j, j + rot/2) or (2j, 2j + 1),
// by the angle of (c, s) = angles[p][j]:  y0 = x0 c - x1 s, y1 = x0 s + x1 c, each product and sum
// rounded to binary32, the result to fp16.
struct Turn {
  const float2* angles;
  const int32_t* pos;  // position of each sequence's first row
  int positions, rot;
};
__device__ __forceinline__ float turn0(float x0, float x1, float2 cs) {
  return __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));
}
__device__ __forceinline__ float turn1(float x0, float x1, float2 cs) {
  return __fadd_rn(__fmul_rn(x0, cs.y), __fmul_rn(x1, cs.x));
}
template <int N>
__device__ __forceinline__ void load_angles(const float2* p, float2* cs) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    cs[i] = make_float2(v.x, v.y);
    cs[i + 1] = make_float2(v.z, v.w);
  }
}
// 8 channels with their partners' 8: the lower or the upper half of the pairs.
__device__ __forceinline__ uint4 turn_half(uint4 x, uint4 partner, const float2* cs, bool upper) {
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, pw[4] = {partner.x, partner.y, partner.z, partner.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_h2(xw[i]), b = unpack_h2(pw[i]);
    y[i] = upper ? pack_h2(turn1(b.x, a.x, cs[2 * i]), turn1(b.y, a.y, cs[2 * i + 1]))
                 : pack_h2(turn0(a.x, b.x, cs[2 * i]), turn0(a.y, b.y, cs[2 * i + 1]));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}
// 8 channels as 4 neighbouring pairs.
__device__ __forceinline__ uint4 turn_pairs(uint4 x, const float2* cs) {
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = unpack_h2(xw[i]);
    y[i] = pack_h2(turn0(a.x, a.y, cs[i]), turn1(a.x, a.y, cs[i]));
  }
  return make_uint4(y[0], y[1], y[2], y[3]);
}

// d/16 lanes per row, 16 channels each: 8 of either half of the pairs, or 8 neighbouring pairs;
// channels behind the first `rot` are copied.  A lane's angles serve all heads that its CTA walks.
// Bound by HBM, 4 bytes an element: 16 prompts of 300 .. 512 tokens, 64 heads of 128 channels, 214 MB:
// 39 us, 5.5 TB/s (0.82 of the copy rate); 64 tokens: the launch, 3 us.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const RaggedArgs a, const Turn turn, float sign, const uint16_t* x, uint16_t* y,
            int64_t y_stride) {
  constexpr int ROWS = 16 * kThreads / D, LPR = D / 16;
  __shared__ int64_t slots[ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int r = threadIdx.x / LPR, u = threadIdx.x % LPR;
  const unsigned tile = blockIdx.x / a.hblocks;
  const int64_t r0 = (int64_t)tile * ROWS;
  const int h0 = (int)(blockIdx.x - tile * a.hblocks) * a.heads, h1 = min(a.H, h0 + a.heads);
  const bool turned = 16 * u < turn.rot;
  const int c0 = turned && !PAIRS ? 8 * u : 16 * u;
  const int c1 = turned && !PAIRS ? turn.rot / 2 + 8 * u : 16 * u + 8;
  const bool held = r0 + r < a.rows;
  const uint16_t* xs = x + (held ? (r0 + r) * a.stride : 0);
  uint4 v[2] = {};
  auto load = [&](int head) {
    if (held) {                            // (y may be x: not through the read-only path)
      v[0] = *reinterpret_cast<const uint4*>(xs + (int64_t)head * D + c0);
      v[1] = *reinterpret_cast<const uint4*>(xs + (int64_t)head * D + c1);
    }
  };
  load(h0);
  tile_slots<ROWS>(a, (int)r0, slots, [&](int b, int64_t t) -> int64_t {
    const int64_t p = turn.pos[b] + t;
    return turn.pos[b] >= 0 && p < turn.positions ? p : -1;
  });
  const int64_t p = slots[r];
  if (p < 0) return;
  float2 cs[8];
  if (turned) {
    load_angles<8>(turn.angles + p * (turn.rot / 2) + 8 * u, cs);
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i].y *= sign;
  }
  uint16_t* ys = y + (r0 + r) * y_stride;
  for (int head = h0; head < h1; ++head) {
    uint4 o[2] = {v[0], v[1]};
    if (head + 1 < h1) load(head + 1);
    if (turned) {
      const uint4 w0 = o[0], w1 = o[1];
      o[0] = PAIRS ? turn_pairs(w0, cs) : turn_half(w0, w1, cs, false);
      o[1] = PAIRS ? turn_pairs(w1, cs + 4) : turn_half(w1, w0, cs, true);
    }
    *reinterpret_cast<uint4*>(ys + (int64_t)head * D + c0) = o[0];
    *reinterpret_cast<uint4*>(ys + (int64_t)head * D + c1) = o[1];
  }
}

// angles[p][j] = gain (cos, sin)(p w_j), in 64 bits, rounded once.
__global__ void __launch_bounds__(kThreads)
rope_table_kernel(float2* angles, int32_t positions, int32_t half, RopeScale sc) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t n = (int64_t)positions * half;
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += step) {
    const int j = (int)(i % half);
    double s, c;
    sincos((double)(i / half) * rope_frequency(sc, j, half), &s, &c);
    angles[i] = make_float2((float)(sc.gain * c), (float)(sc.gain * s));
  }
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

// 4 lanes per group of 64, 16 values each: 16 * 256 / D rows per CTA.  ROPE: K is turned first (1:
// pairs in halves, 2: neighbouring pairs), as rope_kernel does.  Pairs in halves lie in other lanes,
// whose chunks come in a second load (from L1): 48 us for 16 prompts of 300 .. 512 tokens, 32 heads,
// 136 MB, where neighbouring pairs take 38 us and K as it is 30 us.
template <int D, typename Cache, int ROPE>
__global__ void __launch_bounds__(kThreads, ROPE == 0 ? 4 : 2)
append_kernel(const RaggedArgs a, const uint16_t* __restrict__ k_new,
              const uint16_t* __restrict__ v_new, const Cache cache, const Turn turn) {
  constexpr int ROWS = 16 * kThreads / D, LPR = D / 16;
  __shared__ int64_t slots[ROWS];
  __shared__ int turn_at[ROPE ? ROWS : 1];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, r = threadIdx.x / LPR, c = threadIdx.x % LPR;
  const unsigned tile = blockIdx.x / a.hblocks;
  const int64_t r0 = (int64_t)tile * ROWS;
  const int h0 = (int)(blockIdx.x - tile * a.hblocks) * a.heads, h1 = min(a.H, h0 + a.heads);
  const bool held = r0 + r < a.rows;
  const int64_t at = held ? (r0 + r) * a.stride + c * 16 : 0;
  const uint16_t *ks = k_new + at, *vs = v_new + at;
  // the lane's two chunks of 8 channels are both turned or neither (rot is a multiple of 16), and
  // their partners lie half of rot before or behind
  const bool turned = ROPE != 0 && 16 * c < turn.rot;
  const int half = turn.rot / 2;
  const bool upper[2] = {16 * c >= half, 16 * c + 8 >= half};
  uint4 x[4], mate[2];
  auto load = [&](int head) {
    if (held) {
      x[0] = ldg_nc_v4(ks + head * D);
      x[1] = ldg_nc_v4(ks + head * D + 8);
      x[2] = ldg_nc_v4(vs + head * D);
      x[3] = ldg_nc_v4(vs + head * D + 8);
      if (ROPE == 1 && turned) {
        mate[0] = ldg_nc_v4(ks + head * D + (upper[0] ? -half : half));
        mate[1] = ldg_nc_v4(ks + head * D + 8 + (upper[1] ? -half : half));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
  mate[0] = mate[1] = make_uint4(0, 0, 0, 0);
  load(h0);                                // in flight while the rows' sequences are looked up
  tile_slots<ROWS>(a, (int)r0, slots, [&](int b, int64_t t) -> int64_t {
    if (a.pos[b] < 0) return -1;
    if constexpr (ROPE != 0) {
      const int64_t p = turn.pos[b] + t;
      if (turn.pos[b] < 0 || p >= turn.positions) return -1;
      turn_at[threadIdx.x] = (int)p;
    }
    return cache.slot(b, a.pos[b] + t);
  });
  const int64_t slot0 = slots[r];
  const bool live = slot0 >= 0;
  float2 cs[ROPE == 1 ? 16 : 8];
  if (ROPE != 0 && turned && live) {
    const float2* row = turn.angles + (int64_t)turn_at[r] * half;
    if constexpr (ROPE == 1) {
      load_angles<8>(row + 16 * c - (upper[0] ? half : 0), cs);
      load_angles<8>(row + 16 * c + 8 - (upper[1] ? half : 0), cs + 8);
    } else {
      load_angles<8>(row + 8 * c, cs);
    }
  }
  for (int head = h0; head < h1; ++head) {
    uint4 k0 = x[0], k1 = x[1];
    const uint4 v0 = x[2], v1 = x[3];
    if constexpr (ROPE != 0) {
      if (turned && live) {
        k0 = ROPE == 1 ? turn_half(k0, mate[0], cs, upper[0]) : turn_pairs(k0, cs);
        k1 = ROPE == 1 ? turn_half(k1, mate[1], cs + 8, upper[1]) : turn_pairs(k1, cs + 4);
      }
    }
    if (head + 1 < h1) load(head + 1);
    uint32_t kab, vab;
    const uint2 kc = quantize16(k0, k1, lane, &kab);
    const uint2 vc = quantize16(v0, v1, lane, &vab);
    if (live) {
      const Cell cell = cache.template cell<D>(slot0, head);
      *reinterpret_cast<uint2*>(cell.k_codes + c * 8) = kc;
      *reinterpret_cast<uint2*>(cell.v_codes + c * 8) = vc;
      if ((c & 3) == 0) {
        cell.k_ab[c >> 2] = kab;
        cell.v_ab[c >> 2] = vab;
      }
    }
  }
}

// ---------------------------------------------------------------------------- read-back

// 8 lanes per group of 64, 8 values each (a warp's stores are whole 32-byte sectors), two rows
// per thread.
template <int D, typename Cache>
__global__ void __launch_bounds__(kThreads)
read_kernel(const RaggedArgs a, const Cache cache, uint16_t* __restrict__ k_out,
            uint16_t* __restrict__ v_out) {
  constexpr int ROWS = 16 * kThreads / D, LPR = D / 8, STEP = kThreads / LPR;
  __shared__ int64_t slots[ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int r = threadIdx.x / LPR, c = threadIdx.x % LPR;
  const unsigned tile = blockIdx.x / a.hblocks;
  const int64_t r0 = (int64_t)tile * ROWS;
  tile_slots<ROWS>(a, (int)r0, slots, [&](int b, int64_t t) -> int64_t {
    return a.pos[b] < 0 ? -1 : cache.slot(b, a.pos[b] + t);
  });
  const int h0 = (int)(blockIdx.x - tile * a.hblocks) * a.heads, h1 = min(a.H, h0 + a.heads);
  for (int head = h0; head < h1; ++head) {
    uint32_t code[2][2], ab[2][2];
    int64_t slot[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      slot[j] = slots[r + j * STEP];
      if (slot[j] < 0) continue;
      const Cell cell = cache.template cell<D>(slot[j], head);
      if (k_out) {
        code[j][0] = *reinterpret_cast<const uint32_t*>(cell.k_codes + c * 4);
        ab[j][0] = cell.k_ab[c >> 3];
      }
      if (v_out) {
        code[j][1] = *reinterpret_cast<const uint32_t*>(cell.v_codes + c * 4);
        ab[j][1] = cell.v_ab[c >> 3];
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (slot[j] < 0) continue;
      const int64_t at = (r0 + r + j * STEP) * a.stride + (int64_t)head * D + c * 8;
      if (k_out) *reinterpret_cast<uint4*>(k_out + at) = restore8_fp16(code[j][0], ab[j][0]);
      if (v_out) *reinterpret_cast<uint4*>(v_out + at) = restore8_fp16(code[j][1], ab[j][1]);
    }
  }
}

// Heads per CTA: as many as leave the grid ctas_per_sm CTAs per SM, at most 8, so that the lookup
// of a tile's rows is shared; one when there are few tiles.
constexpr int kCtasPerSm = 16, kTurnCtasPerSm = 4;
template <typename Kernel, typename... Args>
cudaError_t launch_per_sm(int ctas_per_sm, Kernel* kernel, const int32_t* row_off,
                          const int32_t* pos, int32_t rows, int64_t stride, int B, int H, int d,
                          int nsm, cudaStream_t st, Args... args) {
  const int per = 16 * kThreads / d;
  const int64_t tiles = ((int64_t)rows + per - 1) / per;
  const int heads =
      (int)std::max<int64_t>(1, std::min<int64_t>(8, tiles * H / ((int64_t)nsm * ctas_per_sm)));
  const int hblocks = (H + heads - 1) / heads;
  if (tiles * hblocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const RaggedArgs a{row_off, pos, rows, B, H, heads, hblocks, stride};
  return launch_pdl(kernel, dim3((unsigned)(tiles * hblocks)), dim3(kThreads), 0, st, a, args...);
}
template <typename Kernel, typename... Args>
cudaError_t launch(Kernel* kernel, const int32_t* row_off, const int32_t* pos, int32_t rows,
                   int64_t stride, int B, int H, int d, int nsm, cudaStream_t st, Args... args) {
  return launch_per_sm(kCtasPerSm, kernel, row_off, pos, rows, stride, B, H, d, nsm, st, args...);
}

}  // namespace

cudaError_t launch_kv_append_ragged(const uint16_t* k_new, const uint16_t* v_new,
                                    int64_t row_stride, int32_t rows, const int32_t* row_off,
                                    const int32_t* pos, const fg_kvcache& kv, int nsm,
                                    cudaStream_t st) {
  const int d = kv.h / kv.H;
  return launch(d == 128 ? append_kernel<128, Regions, 0> : append_kernel<64, Regions, 0>, row_off,
                pos, rows, row_stride, kv.B, kv.H, d, nsm, st, k_new, v_new, Regions{kv}, Turn{});
}

cudaError_t launch_kv_read_ragged(const fg_kvcache& kv, const int32_t* row_off, const int32_t* pos,
                                  int32_t rows, uint16_t* k_out, uint16_t* v_out,
                                  int64_t row_stride, int nsm, cudaStream_t st) {
  const int d = kv.h / kv.H;
  return launch(d == 128 ? read_kernel<128, Regions> : read_kernel<64, Regions>, row_off, pos, rows,
                row_stride, kv.B, kv.H, d, nsm, st, Regions{kv}, k_out, v_out);
}

cudaError_t launch_kv_append_paged(const uint16_t* k_new, const uint16_t* v_new,
                                   int64_t row_stride, int32_t rows, const int32_t* row_off,
                                   const int32_t* pos, const PagedCache& pc, int d,
                                   const RopeRows* rope, int nsm, cudaStream_t st) {
  auto* kernel = d == 128 ? append_kernel<128, Pages, 0> : append_kernel<64, Pages, 0>;
  Turn turn{};
  if (rope) {
    turn = Turn{reinterpret_cast<const float2*>(rope->angles), rope->pos ? rope->pos : pos,
                rope->positions, rope->rot};
    if (rope->interleaved)
      kernel = d == 128 ? append_kernel<128, Pages, 2> : append_kernel<64, Pages, 2>;
    else
      kernel = d == 128 ? append_kernel<128, Pages, 1> : append_kernel<64, Pages, 1>;
  }
  // (a CTA's angles serve all of its heads: 85 us with read-back at 16 CTAs per SM, 74 us at 4)
  return launch_per_sm(rope ? kTurnCtasPerSm : kCtasPerSm, kernel, row_off, pos, rows, row_stride,
                       pc.B, pc.H, d, nsm, st, k_new, v_new, Pages{pc}, turn);
}

cudaError_t launch_kv_read_paged(const PagedCache& pc, int d, const int32_t* row_off,
                                 const int32_t* pos, int32_t rows, uint16_t* k_out,
                                 uint16_t* v_out, int64_t row_stride, int nsm, cudaStream_t st) {
  return launch(d == 128 ? read_kernel<128, Pages> : read_kernel<64, Pages>, row_off, pos, rows,
                row_stride, pc.B, pc.H, d, nsm, st, Pages{pc}, k_out, v_out);
}

cudaError_t launch_rope(const uint16_t* x, int64_t x_stride, int32_t rows, int32_t heads, int d,
                        const int32_t* row_off, int32_t nseq, const RopeRows& rope, bool transpose,
                        uint16_t* y, int64_t y_stride, int nsm, cudaStream_t st) {
  auto* kernel = rope.interleaved ? (d == 128 ? rope_kernel<128, true> : rope_kernel<64, true>)
                                  : (d == 128 ? rope_kernel<128, false> : rope_kernel<64, false>);
  const Turn turn{reinterpret_cast<const float2*>(rope.angles), rope.pos, rope.positions, rope.rot};
  return launch(kernel, row_off, rope.pos, rows, x_stride, nseq, heads, d, nsm, st, turn,
                transpose ? -1.0f : 1.0f, x, y, y_stride);
}

cudaError_t launch_rope_table(float* angles, int32_t positions, int32_t rot, const RopeScale& sc,
                              int nsm, cudaStream_t st) {
  const int64_t n = (int64_t)positions * (rot / 2);
  const int64_t ctas = std::min<int64_t>((n + kThreads - 1) / kThreads, (int64_t)nsm * 8);
  return launch_pdl(rope_table_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, st,
                    reinterpret_cast<float2*>(angles), positions, rot / 2, sc);
}

cudaError_t ragged_read_error(unsigned int* out) {
  return read_and_clear(g_ragged_error, out);
}

}  // namespace fg
