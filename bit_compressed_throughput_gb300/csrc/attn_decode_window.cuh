// Decode attention over the 4-bit cache for sequences of different lengths, with a sliding
// window, first positions that stay visible, and query heads that share K/V heads (sm_103a): the
// kernels, for caches of one region per (sequence, head) and of pages.
//
// The query of sequence b is its newest position i = lens[b] - 1:
//   out_hq = sum_t softmax_t(scale * q_hq . k^_t) v^_t   over the t that i sees,
// K/V head hq / G of G = Hq / H query heads each; a sequence of length 0 sees nothing and gets
// zeros.  Per group g of 64 channels (a = min, s = (b - a)/15, c = code)
//   q . k^ = sum_g (s_g sum_j c_j q_j + a_g sum_j q_j),   sum_t p_t v^_tj = sum_t (p_t s_t) c_tj +
//   sum_t p_t a_t,
// so the products run on mma.sync m16n8k16 over the codes (exact fp16 subnormals, attn_q4.cuh) with
// fp32 sums.  The work is bound by reading the visible part of the cache once.  k^ and v^ are not
// rounded to fp16 then; where a cache asks for the format's rounded values (kRestored: the pages,
// whose values the tensor-core kernels restore, too), they are restored before the products
// (RestoredSums), and the work is bound by the instructions for that.
//
// Columns, over codes: the 8 columns of a product are (part, query head, group) with NP parts of HEADS
// = 4 / NP query heads of one K/V head (for d = 64 the second column of a group pair repeats the first), so
// lane (gid, tig) ends up with scores of head tig % HEADS.  A slot of 32 positions has four
// 8-row halves of tiles; part tig / HEADS takes 4 / NP of them, so the softmax and the statistics
// of a position are computed once per head: with one head per K/V head (NP = 4) a lane has one
// position of the slot, with four (NP = 1) all four of its rows.  The weights meet the values as a
// B operand that is zero outside the part's columns, so the parts add up in separate columns,
// summed at the end.  More than 4 heads per K/V head are further row sets over the same positions,
// adjacent in the work order, which find them in L2.
//
// Work split: the visible 16-position tiles of all row sets (sequence, K/V head, HEADS query heads)
// stand in one order, cut evenly among the warps of the grid (one CTA per SM), whatever the
// lengths.  A warp's share crosses row sets; a row set that lies within one share is finished
// there, one that is cut leaves softmax partials (m, l, unnormalised o), merged by a second kernel
// in a fixed order.  So the scratch is two partials per warp, whatever the call, and results do not
// depend on the order in which warps run.
//
// Memory pipeline, as in the dense decode attention: per warp a ring of slots (2 tiles of K and V
// codes and statistics; 4 where they are restored), filled by bulk async copies that run ahead across
// row sets.  Every wait is bounded; on timeout the warp sets the device error word, drains its copies
// and stops.
//
// Measured (GB300, HBM copy 6.78 TB/s; calls one after another, bytes of the visible 4-bit K/V):
//   128 sequences x 56 heads, 512 .. 1055 positions: 135 us, 0.89 of the copy rate.
//   64 x 32 heads, 200 .. 2048 positions, a window of 1024: 52 us, 0.70.  Of that 2 us plan (with
//   64-bit divisions, and one of them per share boundary, 2.7 us), 4 us pass until the first slots
//   are there, 37 us stream the 248 MB, 5 us are uneven ends (warps end up to 12% behind the mean,
//   in no fixed order) and 4 us merge.
//   16 contexts of 9000 .. 32760, 4 heads per K/V head, a window of 16384: 59 us, 0.70.
// A further row set over the same positions costs most of what the first does: 16 contexts of about
// 32,000, 8 K/V heads, window 16384: 73 us with 1 or 2 heads per K/V head, 75 with 4, 118 with 5, 7
// or 8 (caches cold).
#pragma once
#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attn_q4.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "q4_restore.cuh"
#include "ragged.cuh"

namespace fg {
namespace decode_window {

using q4attn::mma16816;
using q4attn::movtrans;

constexpr int kSub = 2;                   // tiles per ring slot (of codes)
constexpr int kRecentre = 8;              // slots between corrections of the sums (a power of 2)
constexpr int kMinTiles = 2;              // per warp of a small call: one slot (32 heads x 260
                                          // positions: 7.0 us; with 4 and 6, when 2
                                          // took 7.8, 9.3 and 8.8)
constexpr long long kWaitCycles = 1ll << 32;
constexpr unsigned int kErrWait = 1u, kErrDrain = 2u;

// The weights p (b - a) / 15 of the values are rounded to fp16, so they are taken times a power of
// two f per (head, group), which leaves the sums again at their end.  t = (b - a) f is at most
// kWide: with p <= 4 a weight is at most 2^15.  A wider position, or a new reference maximum, sets
// f anew, to t of 2^13 .. 2^14 for the widest position of its slot, so that a 7 times wider one
// still fits; f starts where the narrowest group's t is past kWide.  Weights down to 2^-23 of the
// widest position's are then normal numbers.  (Unscaled, the weights of a position 12 nats below
// the largest score, or of values near 0.003, were subnormal or 0, and their codes' part of the
// values lost, all with one sign: 8192 positions 14 nats below a first one, values of 0.05:
// relative error 2.0e-2, now 2.3e-4 with one head, 5.0e-4 with four; 1 to 2% of the time.)
constexpr float kWide = 122880.0f, kFirstF = 0x1p60f;
__device__ __forceinline__ float inverse_f(float f) {    // of a power of two
  return __uint_as_float(0x7F000000u - __float_as_uint(f));
}
// The power of two that brings t into 2^13 .. 2^14; 1 for 0, infinities and NaN.  (Widths of 2^-24
// .. 131008 keep f within 2^-4 .. 2^60, t and the factor within binary32's normal range.)
__device__ __forceinline__ float to_scale(float t) {
  return t > 0.0f && t < INFINITY ? __uint_as_float((267u - (__float_as_uint(t) >> 23)) << 23)
                                  : 1.0f;
}

// One CTA per SM.  Its rings hold about 110 KB, what the memory system needs in flight (152 x 110
// KB = 17 MB, 2.4 us of its rate); with twice as much the SMs advance less evenly and the last ones
// finish later (128 sequences of 784 positions, 56 heads: 173 us with 16 warps x 3 slots, 152 us
// with 12 x 2; 64-channel heads, whose slots are half as large, 72 us with 16 x 3, 81 us with 12 x
// 2).  Restored values take longer than their bytes, and slots of 4 tiles halve what a slot costs
// beside them (16 contexts of 9000 .. 32760, 8 K/V heads: 173 us with 2 tiles, 166 us with 4 at that
// stage).
template <int D, bool RESTORED>
struct Ring {
  static constexpr int WARPS = (D == 128) ? 12 : 16, DEPTH = (D == 128) ? 2 : 3;
  static constexpr int SUB = RESTORED ? 2 * kSub : kSub, POS = SUB * kTilePos;   // of a slot
  static constexpr int NG = D / 64;
  static constexpr int ROW_CODE = D / 2;                // code bytes of one position
  static constexpr int ROW_AB = NG * 4;                 // statistics bytes of one position
  static constexpr int V_OFF = POS * ROW_CODE;          // V codes in a slot
  static constexpr int KAB_OFF = 2 * V_OFF;
  static constexpr int VAB_OFF = KAB_OFF + POS * ROW_AB;
  static constexpr int SLOT = VAB_OFF + POS * ROW_AB;
  static constexpr int CTA_BYTES = WARPS * DEPTH * (SLOT + 8);
};
static_assert(Ring<128, true>::CTA_BYTES + 1024 <= 227 * 1024, "shared memory per CTA");

// What is to be merged at the cut before a warp's share: the pieces of the row set that it begins
// inside of, when the share before holds that row set's first tile.
struct Cut {
  int pieces;          // 0: nothing to merge here
  int b, hq, heads;
  int prev_slot;       // partial slot of the first piece
};

struct Args {
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  int G, nhb;          // query heads per K/V head; row sets per K/V head
  int window, sinks;
  float scale_log2;
  int ncuts;           // the grid's warps
  Cut* cuts;           // [ncuts]
  float* partial;      // [2 * ncuts][HEADS][D + 2]
  float* lse;          // [rows][query heads], may be null (Cache::kLse)
};

template <typename Cache>
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, unsigned int err) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (clock64() - t0 > kWaitCycles) {
      atomicOr(Cache::error_word(), err);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// An output is a mean of values within fp16's range: what the rounding of the weights (at most
// 131008 * 2^-11) carries past its end is put back; infinities stay.
__device__ __forceinline__ float in_range(float y) {
  return fabsf(y) < 66000.0f ? fminf(fmaxf(y, -65504.0f), 65504.0f) : y;
}

// The log-sum-exp of a maximum and a sum in base 2.
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Cache says where a sequence's positions lie (Run, begin, copy), which row of q and out is its
// query, how long it is (0: it takes no part), which sequences see nothing and get zeros, whether a
// log-sum-exp may be asked for (kLse) and whether values are restored (kRestored).

// A place in the work order: tile u of row set rs of sequence b.
struct Cursor {
  int b, rs, u;
  SeqTiles s;
};
// The K/V head of a row set (most calls have one row set each: no division for them).
__device__ __forceinline__ int kv_head(int rs, const Args& a) {
  return a.nhb == 1 ? rs : rs / a.nhb;
}
// Moves to the next sequence that sees something, found by the whole warp 32 at a time (a batch
// may have many empty places).
template <typename Cache>
__device__ __forceinline__ bool next_sequence(Cursor& c, const Args& a, const Cache& kv) {
  const int lane = threadIdx.x & 31;
  for (int b = c.b + 1; b < kv.B; b += 32) {
    const int len = b + lane < kv.B ? kv.length(b + lane) : 0;
    const unsigned busy = __ballot_sync(0xFFFFFFFFu, len > 0);
    if (busy) {
      const int i = __ffs(busy) - 1;
      c.b = b + i;
      c.s = seq_tiles(__shfl_sync(0xFFFFFFFFu, len, i), a.window, a.sinks);
      return true;
    }
  }
  return false;                            // the end of the order: never asked for
}
template <typename Cache>
__device__ __forceinline__ void next_row_set(Cursor& c, const Args& a, const Cache& kv) {
  c.u = 0;
  if (++c.rs < kv.H * a.nhb) return;
  c.rs = 0;
  next_sequence(c, a, kv);
}

// (a called function: groups with infinities or NaN are rare)
static __device__ __noinline__ uint4 restore8_any(uint32_t codes, uint32_t abw) {
  return restore8_fp16(codes, abw);
}

// The query heads of a row set as B fragments (column n = gid: head (gid / 2) % HEADS, group gid &
// 1; indexes permuted as the lanes hold the codes), the group sums of head tig % HEADS, in the
// base-2 score scale.
template <int D>
struct QFrag {
  uint32_t bq[2 * (D / 32)][2];
  float Q[D / 64];
};
template <int D, int HEADS>
__device__ __forceinline__ void load_q(const uint16_t* q_heads, int heads, int lane,
                                       float scale_log2, QFrag<D>& f) {
  constexpr int NW = D / 32, NG = D / 64;
  const int gid = lane >> 2, tig = lane & 3, col_head = (gid >> 1) % HEADS;
  uint32_t qw[NW * 4];
#pragma unroll
  for (int c = 0; c < NW; ++c) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (col_head < heads) u = ldg_nc_v4(q_heads + col_head * D + tig * 8 * NW + 8 * c);
    qw[4 * c] = u.x; qw[4 * c + 1] = u.y; qw[4 * c + 2] = u.z; qw[4 * c + 3] = u.w;
  }
  const bool mine = NG == 1 || (gid & 1) == (tig >> 1);
  float qsum = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the pair of channels (8w + i, 8w + i + 4) of the lane's chunk
      uint32_t v = __byte_perm(qw[4 * w + (i >> 1)], qw[4 * w + 2 + (i >> 1)],
                               (i & 1) ? 0x7632 : 0x5410);
      const float2 x = unpack_h2(v);
      qsum += x.x + x.y;
      if (i & 1) {                          // odd pairs meet codes times 16
        const __half2 h = __hmul2(*reinterpret_cast<__half2*>(&v), __float2half2_rn(0.0625f));
        v = *reinterpret_cast<const uint32_t*>(&h);
      }
      f.bq[2 * w + (i >> 1)][i & 1] = mine ? v : 0u;
    }
  }
  qsum += __shfl_xor_sync(0xFFFFFFFFu, qsum, 1);
  if (NG == 1) qsum += __shfl_xor_sync(0xFFFFFFFFu, qsum, 2);
#pragma unroll
  for (int g = 0; g < NG; ++g)              // lanes gid = 2 head, tig = 2 g
    f.Q[g] = __shfl_sync(0xFFFFFFFFu, qsum, 8 * (tig % HEADS) + 2 * g) * scale_log2;
}

// What a warp keeps of a row set while it goes through its positions, in products over the codes as
// they are: queries, softmax, the values' sums.
template <int D, int HEADS>
struct CodeSums {
  using R = Ring<D, false>;
  static constexpr int NP = 4 / HEADS, NW = D / 32, NG = D / 64, RPL = 4 / NP;   // RPL: rows a lane
  int gid, tig, part, slots;
  float ck;
  QFrag<D> qf;
  // head tig % HEADS: the part's rows (l, asum) and columns (acc)
  float m_run, l_run;
  float acc[2 * NW][4], asum[NG], wsum[NG], f[NG];     // acc and wsum: times f

  __device__ __forceinline__ CodeSums(const uint16_t* q, int heads, int lane, float scale_log2) {
    gid = lane >> 2, tig = lane & 3, part = tig / HEADS;
    ck = (16777216.0f / 15.0f) * scale_log2;
    load_q<D, HEADS>(q, heads, lane, scale_log2, qf);
    m_run = -INFINITY, l_run = 0.0f;
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[u][c] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      asum[g] = wsum[g] = 0.0f;
      f[g] = kFirstF;
    }
    slots = 0;
  }

  // One slot: scores of every tile, one softmax step, the values of every tile.  MASK: positions
  // that are not visible, and tiles the copy left out (whose stale bytes are still codes), get
  // weight 0 by selects on the score and on the statistics.
  template <bool MASK>
  __device__ __forceinline__ void process(const uint8_t* slot, int ts, int cnt, const SeqTiles& s,
                                          const Args& a) {
    float dk[kSub][4];
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
      uint32_t kw[2][NW];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        load_words<NW>(slot + (sub * kTilePos + gid + 8 * r) * R::ROW_CODE + tig * 4 * NW, kw[r]);
#pragma unroll
      for (int c = 0; c < 4; ++c) dk[sub][c] = 0.0f;
#pragma unroll
      for (int wd = 0; wd < NW; ++wd) {
        uint32_t c0[4], c1[4];
        q4attn::code_pairs(kw[0][wd], c0);
        q4attn::code_pairs(kw[1][wd], c1);
        mma16816(dk[sub], c0[0], c1[0], c0[1], c1[1], qf.bq[2 * wd][0], qf.bq[2 * wd][1]);
        mma16816(dk[sub], c0[2], c1[2], c0[3], c1[3], qf.bq[2 * wd + 1][0],
                 qf.bq[2 * wd + 1][1]);
      }
    }
    // dk[sub][2r + g]: row 16 sub + 8r + gid, the lane's head, group g.  The part's rows are
    // 8 rh + gid, rh = part * RPL + j.
    float sc[RPL];
    bool valid[RPL];
#pragma unroll
    for (int j = 0; j < RPL; ++j) {
      const int row = 8 * (part * RPL + j) + gid, t = ts + row;
      valid[j] = !MASK || (row < cnt * kTilePos && t < s.len &&
                           (t >= s.wstart || t < a.sinks));
      uint32_t ka[NG];
      load_words<NG>(slot + R::KAB_OFF + row * R::ROW_AB, ka);
      float dot = 0.0f, off = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float x;
        if (NP == 4)
          x = (part & 2) ? ((part & 1) ? dk[1][2 + g] : dk[1][g])
                         : ((part & 1) ? dk[0][2 + g] : dk[0][g]);
        else if (NP == 2)
          x = part ? dk[1][2 * j + g] : dk[0][2 * j + g];
        else
          x = dk[j >> 1][2 * (j & 1) + g];
        const float2 ab = unpack_h2(ka[g]);
        dot = fmaf(ab.y - ab.x, x, dot);
        off = fmaf(ab.x, qf.Q[g], off);
      }
      const float s = fmaf(dot, ck, off);
      sc[j] = valid[j] ? s : -INFINITY;
    }
    // The reference maximum moves only when a score exceeds it by more than 2^2, so that p <= 4;
    // the weights' scale then and for a position wider than kWide.
    float mloc = sc[0], tloc[NG] = {};
#pragma unroll
    for (int j = 1; j < RPL; ++j) mloc = fmaxf(mloc, sc[j]);
#pragma unroll
    for (int j = 0; j < RPL; ++j) {
      uint32_t va[NG];
      load_words<NG>(slot + R::VAB_OFF + (8 * (part * RPL + j) + gid) * R::ROW_AB, va);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float2 ab = unpack_h2(valid[j] ? va[g] : 0u);
        tloc[g] = fmaxf(tloc[g], (ab.y - ab.x) * f[g]);
      }
    }
    if (__any_sync(0xFFFFFFFFu,
                   mloc > m_run + 2.0f || fmaxf(tloc[0], tloc[NG - 1]) > kWide)) {
      float mx = fmaxf(mloc, m_run), r[NG];
#pragma unroll
      for (int o = HEADS; o < 32; o <<= 1) {          // over parts and gid
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
        for (int g = 0; g < NG; ++g)
          tloc[g] = fmaxf(tloc[g], __shfl_xor_sync(0xFFFFFFFFu, tloc[g], o));
      }
      const float corr = (m_run == -INFINITY) ? 0.0f : ex2(m_run - mx);
      l_run *= corr;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float n = to_scale(tloc[g]);
        f[g] *= n;
        r[g] = corr * n;
        asum[g] *= corr;
        wsum[g] *= r[g];
      }
#pragma unroll
      for (int u = 0; u < 2 * NW; ++u)                // columns 2 tig, 2 tig + 1: the same head
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[u][c] *= r[NG == 2 ? c & 1 : 0];
      m_run = mx;
    }
    const float m_ref = (m_run == -INFINITY) ? 0.0f : m_run;
    // weights p (b - a) / 15 of both groups, times f, transposed: column (part, head, group) x
    // the half's 8 rows; and their second terms
    uint32_t wt[RPL], lt[RPL];
#pragma unroll
    for (int j = 0; j < RPL; ++j) {
      const int row = 8 * (part * RPL + j) + gid;
      uint32_t va[NG];
      load_words<NG>(slot + R::VAB_OFF + row * R::ROW_AB, va);
      const float p = ex2(sc[j] - m_ref);
      l_run += p;
      const float p15 = p * (1.0f / 15.0f);
      float w[2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float2 ab = unpack_h2(valid[j] ? va[g] : 0u);
        w[g] = p15 * ((ab.y - ab.x) * f[g]);
        asum[g] = fmaf(p, ab.x, asum[g]);
        wsum[g] += w[g];
      }
      // Outputs are means, near 0, of values a + s c with a < 0, and show an fp16 weight's error
      // several times over (relative error of the outputs 6.6e-4).  So the weight's remainder
      // goes along: as a second fp16 term in the columns of another part, which are zero in this
      // half's products (3.3e-4); with one part, where it would take products of its own (4%
      // of the call's time), times the codes' middle, in the sums of the minima (5e-4).
      const uint32_t wh = pack_h2(w[0], NG == 2 ? w[NG - 1] : w[0]);
      const float2 wr = unpack_h2(wh);
      if (NP == 1) {
        asum[0] = fmaf(7.5f * inverse_f(f[0]), w[0] - wr.x, asum[0]);
        if (NG == 2)
          asum[NG - 1] = fmaf(7.5f * inverse_f(f[NG - 1]), w[NG - 1] - wr.y, asum[NG - 1]);
      } else {
        const uint32_t wl = pack_h2(w[0] - wr.x, NG == 2 ? w[NG - 1] - wr.y : w[0] - wr.x);
        lt[j] = movtrans(__shfl_xor_sync(0xFFFFFFFFu, wl, 2));
      }
      wt[j] = movtrans(wh);
    }
#pragma unroll
    for (int sub = 0; sub < kSub; ++sub) {
      uint32_t vw[2][NW], bv[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int rh = 2 * sub + r;
        load_words<NW>(slot + R::V_OFF + (8 * rh + gid) * R::ROW_CODE + tig * 4 * NW, vw[r]);
        const int col = (gid >> 1) / HEADS;            // the part of the lane's column
        bv[r] = (NP == 1 || col == rh / RPL)         ? wt[rh % RPL]
                : ((col ^ (NP / 2)) == rh / RPL) ? lt[rh % RPL]
                                                 : 0u;
      }
#pragma unroll
      for (int wd = 0; wd < NW; ++wd) {
        uint32_t c0[4], c1[4];
        q4attn::code_pairs(movtrans(vw[0][wd]), c0);
        q4attn::code_pairs(movtrans(vw[1][wd]), c1);
        mma16816(acc[2 * wd], c0[0], c0[1], c1[0], c1[1], bv[0], bv[1]);
        mma16816(acc[2 * wd + 1], c0[2], c0[3], c1[2], c1[3], bv[0], bv[1]);
      }
    }
  }

  // Codes are not negative: sums of them grow with the positions, while the output, a mean of
  // values of both signs, gets smaller, and the products' additions truncate.  So every kRecentre
  // slots the codes' middle times the weights since then moves from these sums to those of the
  // minima, binary32 additions of a lane's own.  Relative error of outputs over 65536 positions a
  // warp: 3.5e-4 (without it 6e-2); 1% of the time.
  __device__ __forceinline__ void recentre() {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      asum[g] = fmaf(7.5f * inverse_f(f[g]), wsum[g], asum[g]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)               // the rows of the part
        wsum[g] += __shfl_xor_sync(0xFFFFFFFFu, wsum[g], o);
    }
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c)                    // column 2 tig + (c & 1): the lane's head
        acc[u][c] = fmaf(c < 2 ? -7.5f / 16777216.0f : -7.5f / 1048576.0f,
                         wsum[NG == 2 ? c & 1 : 0], acc[u][c]);
#pragma unroll
    for (int g = 0; g < NG; ++g) wsum[g] = 0.0f;
  }
  __device__ __forceinline__ void slot_done() {
    if ((++slots & (kRecentre - 1)) == 0) recentre();
  }

  // Sums over the rows' lanes and the parts, into the outputs of the set's heads (`out`: the first
  // one's) and their log-sum-exp (may be null), or its partial [HEADS][D + 2].
  __device__ __forceinline__ void finish(bool whole, int heads, uint16_t* out, float* lse,
                                         float* partial) {
#pragma unroll
    for (int o = HEADS; o < 32; o <<= 1) {
      l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, o);
#pragma unroll
      for (int g = 0; g < NG; ++g) asum[g] += __shfl_xor_sync(0xFFFFFFFFu, asum[g], o);
    }
    // the lane's channels are those of group gid / 4 (d = 128): pair u holds channels cbase + 8 (u
    // / 2) + 2 (u % 2) and the next
    const int g = (NG == 2) ? (gid >> 2) : 0;
    const float A = (NG == 2 && g) ? asum[NG - 1] : asum[0];
    const int cbase = 8 * NW * (gid >> 1) + 4 * (gid & 1);
    const float unit = inverse_f(g ? f[NG - 1] : f[0]);
    float2 y[2 * NW];
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
      y[u] = make_float2((g ? acc[u][1] : acc[u][0]) * (16777216.0f * unit),
                         (g ? acc[u][3] : acc[u][2]) * (1048576.0f * unit));
    // each halving of the parts leaves half of the pairs to a lane: pairs u0 .. u0 + NY - 1
    constexpr int NY = 2 * NW / NP;
    int u0 = 0;
#pragma unroll
    for (int n = NW, o = 2; o >= HEADS; n >>= 1, o >>= 1) {
      const bool up = tig & o;
#pragma unroll
      for (int u = 0; u < n; ++u) {
        const float2 keep = up ? y[u + n] : y[u], send = up ? y[u] : y[u + n];
        y[u].x = keep.x + __shfl_xor_sync(0xFFFFFFFFu, send.x, o);
        y[u].y = keep.y + __shfl_xor_sync(0xFFFFFFFFu, send.y, o);
      }
      u0 += up ? n : 0;
    }
    const int head = tig % HEADS;
    if (head >= heads) return;
    const float inv = (l_run == 0.0f) ? 0.0f : 1.0f / l_run;
    uint16_t* o = out + head * D;
    float* pp = partial + head * (D + 2);
#pragma unroll
    for (int i = 0; i < NY; ++i) {
      const int ch = cbase + 8 * ((u0 + i) >> 1) + 2 * ((u0 + i) & 1);
      const float y0 = y[i].x + A, y1 = y[i].y + A;
      if (whole)
        *reinterpret_cast<uint32_t*>(o + ch) = pack_h2(in_range(y0 * inv), in_range(y1 * inv));
      else
        *reinterpret_cast<float2*>(pp + ch) = make_float2(y0, y1);
    }
    if (gid != 0 || part != 0) return;
    if (!whole) *reinterpret_cast<float2*>(pp + D) = make_float2(m_run, l_run);
    if (lse && whole) lse[head] = log_sum(m_run, l_run);
  }
};

// The same in products over values restored to fp16 exactly as the format defines them.  Positions are
// the rows of K Q^T and the columns of V^T P^T, up to 8 query heads the columns of both.  A lane (gid,
// tig) has the scores of positions gid and gid + 8 of a tile for heads 2 tig and 2 tig + 1; of the
// values it restores, for positions 2 tig, 2 tig + 1 (and 8 behind), the channels that a transposition
// of the code words gives row gid.  Weights are scaled by 2^7, which lets the reference maximum lag by
// 2^8, and go into the products as two fp16 terms, so that their rounding does not show in the outputs
// (relative error 2.9e-4, and up to 3.2e-4 where few weights count, with one; 2.1e-4, that of the
// outputs' own rounding, with both; 5% of the time).
template <int D, int HEADS>
struct RestoredSums {
  using R = Ring<D, true>;
  static constexpr int NW = D / 32;
  static constexpr float kLag = 8.0f, kPExp = 7.0f;
  static constexpr int kFlush = 32;        // slots between moves of the sums (a power of 2)
  int gid, tig, slots;
  float sl2;
  uint4 q[NW];                             // head gid: 8 channels a word
  float m[2], l[2], acc[2 * NW][4];        // heads 2 tig, 2 tig + 1
  // The products' additions truncate: sums of values of one sign lose 4e-4 over 65536 positions.  So
  // every kFlush slots they move to sums of binary32 additions, in local memory (volatile: with all in
  // registers some are spilled, and 16 contexts of 9000 .. 32760 took 185 us, 171 us as it is, 166 us
  // without), relative to the maximum m_far.
  volatile float far[2 * NW][4];
  float m_far[2];

  __device__ __forceinline__ RestoredSums(const uint16_t* q_heads, int heads, int lane,
                                          float scale_log2) {
    gid = lane >> 2, tig = lane & 3, slots = 0;
    sl2 = scale_log2;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      q[w] = gid < heads ? ldg_nc_v4(q_heads + gid * D + tig * 8 * NW + 8 * w)
                         : make_uint4(0, 0, 0, 0);
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[u][c] = 0.0f;
  }

  // One slot, tile by tile (in a loop, so that its instructions stay near).  MASK: positions that are
  // not visible get weight 0 by selects on the score and on the value's statistics.
  template <bool MASK>
  __device__ __forceinline__ void process(const uint8_t* slot, int ts, int cnt, const SeqTiles& s,
                                          const Args& a) {
#pragma unroll 1
    for (int sub = 0; sub < (MASK ? cnt : R::SUB); ++sub) {
      const int row0 = sub * kTilePos;
      auto sees = [&](int row) {
        const int t = ts + row0 + row;
        return !MASK || (t < s.len && (t >= s.wstart || t < a.sinks));
      };
      // ---- scores
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      {
        const uint8_t* k = slot + (row0 + gid) * R::ROW_CODE + tig * 4 * NW;
        const uint8_t* ab = slot + R::KAB_OFF + (row0 + gid) * R::ROW_AB +
                            (D == 128 ? 4 * (tig >> 1) : 0);
        uint32_t w0[NW], w1[NW], ab0[1], ab1[1];
        load_words<NW>(k, w0);
        load_words<NW>(k + 8 * R::ROW_CODE, w1);
        load_words<1>(ab, ab0);
        load_words<1>(ab + 8 * R::ROW_AB, ab1);
        const GroupFp16 g0(ab0[0]), g1(ab1[0]);
        const bool plain = __all_sync(0xFFFFFFFFu, g0.plain && g1.plain);
#pragma unroll
        for (int w = 0; w < NW; w += 2) {
          uint4 k0[2], k1[2];
          if (plain) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              k0[i] = g0.restore(w0[w + i]);
              k1[i] = g1.restore(w1[w + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              k0[i] = restore8_any(w0[w + i], ab0[0]);
              k1[i] = restore8_any(w1[w + i], ab1[0]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma16816(c, k0[i].x, k1[i].x, k0[i].y, k1[i].y, q[w + i].x, q[w + i].y);
            mma16816(c, k0[i].z, k1[i].z, k0[i].w, k1[i].w, q[w + i].z, q[w + i].w);
          }
        }
      }
      // c[2 r + e]: position gid + 8 r, head 2 tig + e
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (!sees(gid + 8 * r)) c[2 * r] = c[2 * r + 1] = -INFINITY;
      float mx[2] = {fmaxf(c[0], c[2]) * sl2, fmaxf(c[1], c[3]) * sl2};
      if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] + kLag || mx[1] > m[1] + kLag)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(mx[e], m[e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], o));
          const float alpha = m[e] == -INFINITY ? 0.0f : ex2(m[e] - mx[e]);
          l[e] *= alpha;
#pragma unroll
          for (int u = 0; u < 2 * NW; ++u) {
            acc[u][e] *= alpha;
            acc[u][2 + e] *= alpha;
          }
          m[e] = mx[e];
        }
      }
      // ---- weights
      uint32_t b[2], rest[2];
      {
        const float z0 = kPExp - (m[0] == -INFINITY ? 0.0f : m[0]);
        const float z1 = kPExp - (m[1] == -INFINITY ? 0.0f : m[1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float p0 = ex2(fmaf(c[2 * r], sl2, z0)), p1 = ex2(fmaf(c[2 * r + 1], sl2, z1));
          l[0] += p0;
          l[1] += p1;
          const uint32_t h = pack_h2(p0, p1);
          const float2 x = unpack_h2(h);
          b[r] = movtrans(h);
          rest[r] = movtrans(pack_h2(p0 - x.x, p1 - x.y));
        }
      }
      // ---- values
      const uint8_t* v = slot + R::V_OFF + (row0 + gid) * R::ROW_CODE + tig * 4 * NW;
      uint32_t v0[NW], v1[NW], ab[2][2];
      load_words<NW>(v, v0);
      load_words<NW>(v + 8 * R::ROW_CODE, v1);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * r + 2 * tig + i;
          uint32_t word[1];
          load_words<1>(slot + R::VAB_OFF + (row0 + row) * R::ROW_AB + (D == 128 ? 4 * (gid >> 2) : 0),
                        word);
          ab[r][i] = sees(row) ? word[0] : 0u;         // (0, 0): every code is 0
        }
      const PairsFp16 g0(ab[0][0], ab[0][1]), g1(ab[1][0], ab[1][1]);
      const bool plain = __all_sync(0xFFFFFFFFu, g0.plain && g1.plain);
#pragma unroll
      for (int w = 0; w < NW; w += 2) {
        uint4 x[2], y[2];
        const uint32_t t0[2] = {movtrans(v0[w]), movtrans(v0[w + 1])};
        const uint32_t t1[2] = {movtrans(v1[w]), movtrans(v1[w + 1])};
        if (plain) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[i] = g0.restore(t0[i]);
            y[i] = g1.restore(t1[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[i] = restore_pairs_exact(t0[i], ab[0][0], ab[0][1]);
            y[i] = restore_pairs_exact(t1[i], ab[1][0], ab[1][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int u = 2 * (w + i);
          mma16816(acc[u], x[i].x, x[i].y, y[i].x, y[i].y, b[0], b[1]);
          mma16816(acc[u + 1], x[i].z, x[i].w, y[i].z, y[i].w, b[0], b[1]);
          if (plain) {                     // (0 or less times an infinity: NaN)
            mma16816(acc[u], x[i].x, x[i].y, y[i].x, y[i].y, rest[0], rest[1]);
            mma16816(acc[u + 1], x[i].z, x[i].w, y[i].z, y[i].w, rest[0], rest[1]);
          }
        }
      }
    }
  }
  // acc added to the far sums (without any: their start), in the scale of the present maximum.
  __device__ __forceinline__ void add_far(bool any) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float f = any && m_far[e] != -INFINITY ? ex2(m_far[e] - m[e]) : 0.0f;
#pragma unroll
      for (int u = 0; u < 2 * NW; ++u) {
        acc[u][e] = any ? fmaf(far[u][e], f, acc[u][e]) : acc[u][e];
        acc[u][2 + e] = any ? fmaf(far[u][2 + e], f, acc[u][2 + e]) : acc[u][2 + e];
      }
    }
  }
  __device__ __forceinline__ void slot_done() {
    if ((++slots & (kFlush - 1)) != 0) return;
    add_far(slots > kFlush);
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        far[u][c] = acc[u][c];
        acc[u][c] = 0.0f;
      }
    m_far[0] = m[0], m_far[1] = m[1];
  }

  __device__ __forceinline__ void finish(bool whole, int heads, uint16_t* out, float* lse,
                                         float* partial) {
    if (slots >= kFlush) add_far(true);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], o);
      l[1] += __shfl_xor_sync(0xFFFFFFFFu, l[1], o);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int head = 2 * tig + e;
      if (head >= heads) continue;
      const float inv = l[e] == 0.0f ? 0.0f : 1.0f / l[e];
      // acc[2 w + j]: channels 2 j, 2 j + 1 of the four of word w
      const int ch = 8 * NW * (gid >> 1) + 4 * (gid & 1);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 y = make_float4(acc[2 * w][e], acc[2 * w][2 + e], acc[2 * w + 1][e],
                                     acc[2 * w + 1][2 + e]);
        if (whole) {
          *reinterpret_cast<uint2*>(out + head * D + ch + 8 * w) =
              make_uint2(pack_h2(in_range(y.x * inv), in_range(y.y * inv)),
                         pack_h2(in_range(y.z * inv), in_range(y.w * inv)));
        } else {
          float2* pp = reinterpret_cast<float2*>(partial + head * (D + 2) + ch + 8 * w);
          pp[0] = make_float2(y.x, y.y);
          pp[1] = make_float2(y.z, y.w);
        }
      }
      if (gid != 0) continue;
      if (!whole)                          // 2^(score - m + 7): of the maximum m - 7
        *reinterpret_cast<float2*>(partial + head * (D + 2) + D) = make_float2(m[e] - kPExp, l[e]);
      if (lse && whole) lse[head] = log_sum(m[e] - kPExp, l[e]);
    }
  }
};

// Moves a place dx tiles on in the order.
template <typename Cache>
__device__ __forceinline__ void skip_tiles(Cursor& c, int64_t dx, const Args& a,
                                           const Cache& kv) {
  const int rsets = kv.H * a.nhb;
  int64_t at = (int64_t)c.rs * c.s.nt + c.u + dx;        // within sequence b
  while (at >= (int64_t)rsets * c.s.nt) {
    at -= (int64_t)rsets * c.s.nt;
    if (!next_sequence(c, a, kv)) return;
  }
  c.rs = at < 0x7FFFFFFF ? (int)((unsigned)at / (unsigned)c.s.nt) : (int)(at / c.s.nt);
  c.u = (int)(at - (int64_t)c.rs * c.s.nt);
}

template <int D, int HEADS, typename Cache>
__global__ void __launch_bounds__(Ring<D, Cache::kRestored>::WARPS * 32, 1)
decode_window_kernel(const Args a, const Cache kv) {
  using R = Ring<D, Cache::kRestored>;
  using Sums = std::conditional_t<Cache::kRestored, RestoredSums<D, HEADS>, CodeSums<D, HEADS>>;
  constexpr int kWarps = R::WARPS, kRing = R::DEPTH;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned warp_nt[kWarps];
  __shared__ int first_b;                  // the sequence of the CTA's first tile,
  __shared__ int64_t first_before;         // and the tiles of the sequences before it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * kRing * R::SLOT;
  const uint32_t ring0 = smem_u32(ring);
  const uint32_t bar0 = smem_u32(smem + kWarps * kRing * R::SLOT) + warp * kRing * 8;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(bar0 + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the order of the work: how many tiles, and where this CTA's begin
  const int rsets = kv.H * a.nhb;          // row sets of one sequence
  int64_t tiles = 0, before = 0;           // of one row set: all sequences; those of earlier rounds
  unsigned incl = 0, mine = 0;
  auto scan_round = [&](int b0) {          // a sequence per thread: its tiles, those up to it
    const int b = b0 + threadIdx.x;
    mine = b < kv.B ? seq_tiles(kv.length(b), a.window, a.sinks).nt : 0;
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_nt[warp] = incl;
    __syncthreads();
    unsigned round = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const unsigned n = warp_nt[i];
      if (i < warp) incl += n;
      round += n;
    }
    __syncthreads();
    return round;
  };
  for (int b0 = 0; b0 < kv.B; b0 += kWarps * 32) tiles += scan_round(b0);
  const int64_t total = tiles * rsets;
  // Neighbours of the order sit on one SM (they read neighbouring memory); a call with less than
  // kMinTiles for every warp has fewer shares of about that, the same few on every SM.
  const int64_t most_shares = max((int64_t)1, total / kMinTiles);
  const int per_cta = most_shares >= (int64_t)kWarps * gridDim.x
                          ? kWarps
                          : ((int)most_shares - 1) / (int)gridDim.x + 1;
  const int n = (int)min(most_shares, (int64_t)gridDim.x * per_cta);
  const Shares shares(total, n);
  const int w = blockIdx.x * per_cta + warp;
  const bool busy = total > 0 && (int)blockIdx.x * per_cta < n;
  const int64_t cta_x = busy ? shares.first(blockIdx.x * per_cta) : 0;
  if (busy) {
    for (int b0 = 0; b0 < kv.B; b0 += kWarps * 32) {
      const unsigned round = kv.B > kWarps * 32 ? scan_round(b0) : (unsigned)tiles;
      if ((before + round) * rsets > cta_x) {
        if ((before + incl) * rsets > cta_x && (before + incl - mine) * rsets <= cta_x) {
          first_b = b0 + threadIdx.x;
          first_before = before + incl - mine;
        }
        break;
      }
      before += round;
    }
  }
  __syncthreads();

  // ---- issue: fills the ring kRing slots ahead of the computation, one run of positions (the
  // first ones or the window of a row set) after the other
  int ileft = 0, irun = 0, is = 0, issued = 0;         // tiles left, of them in the run; slot
  typename Cache::Run run_at;              // the run's next position
  Cursor ic{};
  const bool has_share = busy && warp < per_cta && w < n;
  if (has_share) {
    const int64_t x0 = shares.first(w);
    ileft = (int)(shares.first(w + 1) - x0);           // the host bounds the call's tiles by 2^40
    ic.b = first_b;
    ic.s = seq_tiles(kv.length(ic.b), a.window, a.sinks);
    skip_tiles(ic, x0 - first_before * rsets, a, kv);
  }
  Cursor cc = ic;                          // the computation's cursor
  int left = ileft;
  auto issue = [&]() {
    if (irun == 0) {
      if (ileft == 0) return;
      if (ic.u == ic.s.nt) {
        next_row_set(ic, a, kv);
        // its queries, needed kRing slots from here
        const int hk = kv_head(ic.rs, a);
        constexpr int LPH = HEADS > 4 ? 4 : 8;         // lanes a head
        const int hq = hk * a.G + (ic.rs - hk * a.nhb) * HEADS + lane / LPH;
        if (lane / LPH < HEADS && hq < hk * a.G + a.G && lane % LPH * (128 / LPH) < D)
          prefetch_l2(a.q + kv.row(ic.b) * a.q_stride + (int64_t)hq * D + lane % LPH * (128 / LPH));
      }
      irun = run_tiles(ic.s, ic.u, min(ic.s.nt, ic.u + ileft));
      kv.begin(run_at, ic.b, kv_head(ic.rs, a), tile_pos(ic.s, ic.u));
      ic.u += irun;
      ileft -= irun;
    }
    const int cnt = min(R::SUB, irun);
    kv.template copy<D>(run_at, cnt, ring0 + is * R::SLOT, bar0 + 8 * is);
    irun -= cnt;
    ++issued;
    if (++is == kRing) is = 0;
  };
  for (int i = 0; i < kRing; ++i) issue();

  // ---- what is to be merged at this warp's cut
  Cut cut{};
  if (has_share && cc.u > 0) {
    const int64_t r0 = shares.first(w) - cc.u, xp = shares.first(w - 1);
    if (xp <= r0) {
      const int hk = kv_head(cc.rs, a), hb = cc.rs - hk * a.nhb;
      cut.pieces = shares.share_of(r0 + cc.s.nt - 1) - (w - 1) + 1;
      cut.b = cc.b;
      cut.hq = hk * a.G + hb * HEADS;
      cut.heads = min(HEADS, a.G - hb * HEADS);
      cut.prev_slot = 2 * (w - 1) + (xp == r0 ? 0 : 1);
    }
  }
  if (has_share && lane == 0) a.cuts[w] = cut;

  // ---- sequences that see nothing, and cuts of warps without a share
  for (int64_t b = (int64_t)blockIdx.x * kWarps + warp; b < kv.B;
       b += (int64_t)gridDim.x * kWarps) {
    if (lane == 0 && kv.misfit((int)b)) atomicOr(Cache::error_word(), kErrExtent);
    if (kv.blind((int)b))
      for (int i = lane; i < kv.H * a.G * (D / 8); i += 32) {
        reinterpret_cast<uint4*>(a.out + kv.row((int)b) * a.out_stride)[i] =
            make_uint4(0, 0, 0, 0);
        if (Cache::kLse && a.lse && i < kv.H * a.G)
          a.lse[kv.row((int)b) * (kv.H * a.G) + i] = -INFINITY;
      }
  }
  for (int c = (total > 0 ? n : 0) + blockIdx.x * kWarps * 32 + threadIdx.x; c < a.ncuts;
       c += gridDim.x * kWarps * 32)
    a.cuts[c].pieces = 0;

  int cs = 0, consumed = 0;
  uint32_t cph = 0;
  bool ok = true;
  for (int seg_no = 0; left > 0 && ok; ++seg_no) {
    const int u1 = min(cc.s.nt, cc.u + left);
    const bool whole = cc.u == 0 && u1 == cc.s.nt;
    const int seg = u1 - cc.u;
    const int hk = kv_head(cc.rs, a), hb = cc.rs - hk * a.nhb;
    const int hq = hk * a.G + hb * HEADS, heads = min(HEADS, a.G - hb * HEADS);
    Sums sums(a.q + kv.row(cc.b) * a.q_stride + (int64_t)hq * D, heads, lane, a.scale_log2);
    while (cc.u < u1 && ok) {
      int run = run_tiles(cc.s, cc.u, u1), ts = tile_pos(cc.s, cc.u);
      cc.u += run;
      for (; run > 0; run -= R::SUB, ts += R::POS) {
        ok = __all_sync(0xFFFFFFFFu, bounded_wait<Cache>(bar0 + 8 * cs, cph, kErrWait));
        if (!ok) break;
        const uint8_t* slot = ring + cs * R::SLOT;
        const int te = ts + R::POS;
        if (run >= R::SUB && te <= cc.s.len && (ts >= cc.s.wstart || te <= a.sinks))
          sums.template process<false>(slot, ts, R::SUB, cc.s, a);
        else
          sums.template process<true>(slot, ts, min(run, R::SUB), cc.s, a);
        __syncwarp();                       // every lane has read the slot: refill it
        issue();
        sums.slot_done();
        ++consumed;
        if (++cs == kRing) {
          cs = 0;
          cph ^= 1u;
        }
      }
    }
    if (!ok) break;
    sums.finish(whole, heads, a.out + kv.row(cc.b) * a.out_stride + (int64_t)hq * D,
                Cache::kLse && a.lse ? a.lse + kv.row(cc.b) * (kv.H * a.G) + hq : nullptr,
                a.partial + (int64_t)(2 * w + (seg_no > 0)) * HEADS * (D + 2));
    __syncwarp();
    left -= seg;
    if (left > 0) next_row_set(cc, a, kv);
  }

  // ---- every issued copy lands before the warp's shared memory is released
  for (int i = consumed; i < issued; ++i)
    bounded_wait<Cache>(bar0 + 8 * (uint32_t)(i % kRing), (uint32_t)((i / kRing) & 1), kErrDrain);
}

// One warp per (cut, head of its row set): merges the pieces (m, l, unnormalised o) in order,
// 32 at a time: a lane takes one piece's m and l, then all lanes that piece's channels.
template <int D, int HEADS, typename Cache>
__global__ void __launch_bounds__(HEADS * 32)
merge_kernel(const Args a, const Cache kv) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int C = D / 32;
  const Cut cut = a.cuts[blockIdx.x];
  const int head = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (cut.pieces == 0 || head >= cut.heads) return;
  auto piece = [&](int i) {
    const int slot = i == 0 ? cut.prev_slot : 2 * ((int)blockIdx.x + i - 1);
    return a.partial + ((int64_t)slot * HEADS + head) * (D + 2);
  };
  float M = -INFINITY, L = 0.0f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.0f;
  // 16 pieces' channels at a time, the first 16 in flight before their weights are known (one
  // sequence of 260 visible positions: 7.0 us; 8 at a time 7.6, 32 7.2)
  constexpr int BATCH = 16;
  float v[BATCH][C];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (i0 + i < cut.pieces) {
        const float* pp = piece(i0 + i);
#pragma unroll
        for (int c = 0; c < C; ++c) v[i][c] = pp[c * 32 + lane];
      }
  };
  for (int i0 = 0; i0 < cut.pieces; i0 += 32) {
    const int n = min(32, cut.pieces - i0);
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < n) ml = *reinterpret_cast<const float2*>(piece(i0 + lane) + D);
    load(i0);
    float mx = ml.x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
    mx = fmaxf(mx, M);
    const float ref = (mx == -INFINITY) ? 0.0f : mx;
    const float corr = exp2f(M - ref), wgt = exp2f(ml.x - ref);
    float l = wgt * ml.y;                   // 0 * NaN where a piece is NaN: as it should be
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, k);
    L = fmaf(L, corr, l);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= corr;
    for (int j = 0; j < n; j += BATCH) {
      if (j > 0) load(i0 + j);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float wi = __shfl_sync(0xFFFFFFFFu, wgt, j + i);
        if (j + i < n) {
#pragma unroll
          for (int c = 0; c < C; ++c) o[c] = fmaf(wi, v[i][c], o[c]);
        }
      }
    }
    M = mx;
  }
  const float inv = (L == 0.0f) ? 0.0f : 1.0f / L;
  uint16_t* op = a.out + kv.row(cut.b) * a.out_stride + (int64_t)(cut.hq + head) * D;
  if (Cache::kLse && a.lse && lane == 0)
    a.lse[kv.row(cut.b) * (kv.H * a.G) + cut.hq + head] = log_sum(M, L);
#pragma unroll
  for (int c = 0; c < C; ++c) op[c * 32 + lane] = f2h(in_range(o[c] * inv));
}

// The most tiles that `sets` row sets can have: every sequence full, or its window and first positions.
inline int64_t most_tiles(int64_t sets, int cap, int window, int sinks) {
  const SeqTiles s = seq_tiles(cap, window, sinks);
  return sets * (s.nt + 2);
}
inline int grid_ctas(int64_t most, int nsm) {
  return (int)std::min<int64_t>(most / kMinTiles + 1, std::max(nsm, 1));
}
inline size_t cut_bytes(int64_t ncuts) { return ((size_t)ncuts * sizeof(Cut) + 255) / 256 * 256; }

// Shared memory and carveout of the kernel on the current device, set once per device.
template <int D, int HEADS, typename Cache>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 0 || dev >= 64 || done[dev]) return cudaSuccess;
  auto* kernel = decode_window_kernel<D, HEADS, Cache>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Ring<D, Cache::kRestored>::CTA_BYTES)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) !=
          cudaSuccess)
    return e;
  done[dev] = true;
  return cudaSuccess;
}

template <int D, int HEADS, typename Cache>
cudaError_t launch_d(const Args& a, const Cache& kv, int ctas, cudaStream_t st) {
  cudaError_t e = prepare<D, HEADS, Cache>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_window_kernel<D, HEADS, Cache>, dim3(ctas),
                 dim3(Ring<D, Cache::kRestored>::WARPS * 32), Ring<D, Cache::kRestored>::CTA_BYTES,
                 st, a, kv);
  if (e != cudaSuccess) return e;
  return launch_pdl(merge_kernel<D, HEADS, Cache>, dim3(a.ncuts), dim3(HEADS * 32), 0, st, a, kv);
}

template <bool RESTORED>
int warps_of(int d) { return d == 128 ? Ring<128, RESTORED>::WARPS : Ring<64, RESTORED>::WARPS; }
// Shares that a call of at most `most` tiles can have.
template <bool RESTORED>
int64_t most_cuts(int64_t most, int nsm, int d) {
  return std::min<int64_t>(most / kMinTiles + 1,
                           (int64_t)grid_ctas(most, nsm) * warps_of<RESTORED>(d));
}
// Query heads of a row set: 1, 2 or 4, of restored values also 8.
inline int set_heads(int G, bool restored) { return G < 3 ? G : (G < 5 || !restored ? 4 : 8); }

// Scratch for calls of at most `sets` row sets of up to cap positions, on up to nsm SMs.
template <bool RESTORED>
size_t workspace_bytes(int64_t sets, int cap, int heads, int d, int nsm) {
  const int64_t n = most_cuts<RESTORED>(most_tiles(sets, cap, 0, 0), nsm, d);
  return cut_bytes(n) + (size_t)n * 2 * heads * (d + 2) * sizeof(float);
}
// Fills in the work's extent and its scratch, and launches; `sets` row sets.
template <typename Cache>
cudaError_t launch_sets(Args& a, const Cache& kv, int64_t sets, int cap, int d, void* ws, int nsm,
                        cudaStream_t st) {
  const int64_t most =
      std::min(most_tiles(sets, cap, a.window, a.sinks), most_tiles(sets, cap, 0, 0));
  const int ctas = grid_ctas(most, nsm);
  a.ncuts = (int)most_cuts<Cache::kRestored>(most, nsm, d);
  a.cuts = static_cast<Cut*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + cut_bytes(a.ncuts));
  const int heads = set_heads(a.G, Cache::kRestored);
  auto* launch = heads == 1   ? (d == 128 ? launch_d<128, 1, Cache> : launch_d<64, 1, Cache>)
                 : heads == 2 ? (d == 128 ? launch_d<128, 2, Cache> : launch_d<64, 2, Cache>)
                              : (d == 128 ? launch_d<128, 4, Cache> : launch_d<64, 4, Cache>);
  if constexpr (Cache::kRestored)
    if (heads == 8) launch = d == 128 ? launch_d<128, 8, Cache> : launch_d<64, 8, Cache>;
  return launch(a, kv, ctas, st);
}

}  // namespace decode_window
}  // namespace fg
