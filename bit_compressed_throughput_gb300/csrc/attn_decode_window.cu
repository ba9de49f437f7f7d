// Decode attention over the 4-bit cache for sequences of different lengths, with a sliding
// window, first positions that stay visible, and query heads that share K/V heads (sm_103a).
//
// The query of sequence b is its newest position i = lens[b] - 1:
//   out_hq = sum_t softmax_t(scale * q_hq . k^_t) v^_t   over the t that i sees,
// K/V head hq / G of G = Hq / H query heads each; a sequence of length 0 sees nothing and gets
// zeros.  Per group g of 64 channels (a = min, s = (b - a)/15, c = code)
//   q . k^ = sum_g (s_g sum_j c_j q_j + a_g sum_j q_j),   sum_t p_t v^_tj = sum_t (p_t s_t) c_tj +
//   sum_t p_t a_t,
// so the products run on mma.sync m16n8k16 over the codes (exact fp16 subnormals, attn_q4.cuh) with
// fp32 sums.  The work is bound by reading the visible part of the cache once.
//
// Heads: the 8 columns of a product are (query head, group) pairs -- 4 heads of one K/V head (for
// d = 64 the second column of a pair repeats the first) -- so lane (gid, tig) ends up with the
// scores, weights and outputs of head tig for the rows and channels of gid: up to 4 heads cost
// what one does.  More than 4 heads per K/V head are further row sets over the same positions,
// adjacent in the work order, which find them in L2.
//
// Work split: the visible 16-position tiles of all row sets (sequence, K/V head, 4 query heads) stand
// in one order, cut evenly among the warps of the grid, whatever the lengths.  A warp's range crosses
// row sets; a row set that lies within one range is finished there, one that is cut leaves softmax
// partials (m, l, unnormalised o), merged by a second kernel in a fixed order.  So the scratch is
// two partials per warp, whatever the call.
//
// Memory pipeline, as in the dense decode attention: per warp a ring of slots (3 tiles of K and V
// codes and statistics), filled by bulk async copies that run ahead across row sets.  Every wait is
// bounded; on timeout the warp sets the device error word, drains its copies and stops.
#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attn_q4.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_decode_window_error = 0;

namespace {

using q4attn::mma16816;
using q4attn::movtrans;

constexpr int kWarps = 4;                 // per CTA
constexpr int kCtasPerSm = 4;
constexpr int kHeads = 4;                 // query heads of a row set
constexpr int kSub = 3;                   // tiles per ring slot
constexpr int kSlotPos = kSub * kTilePos;
constexpr int kRing = 2;                  // slots per warp
constexpr int kMinTiles = 3;              // per warp of a small call: one slot
constexpr long long kWaitCycles = 1ll << 32;
constexpr unsigned int kErrWait = 1u, kErrDrain = 2u;

template <int D>
struct Ring {
  static constexpr int NG = D / 64;
  static constexpr int ROW_CODE = D / 2;                // code bytes of one position
  static constexpr int ROW_AB = NG * 4;                 // statistics bytes of one position
  static constexpr int V_OFF = kSlotPos * ROW_CODE;     // V codes in a slot
  static constexpr int KAB_OFF = 2 * V_OFF;
  static constexpr int VAB_OFF = KAB_OFF + kSlotPos * ROW_AB;
  static constexpr int SLOT = VAB_OFF + kSlotPos * ROW_AB;
  static constexpr int CTA_BYTES = kWarps * kRing * (SLOT + 8);
};

// What a warp leaves of its first row set when an earlier warp began it: the warp before the first
// such cut merges `pieces` partials, from its own on.
struct Cut {
  int pieces;          // 0: nothing to merge here
  int b, hq, heads;
  int prev_slot;       // partial slot of the first piece
};

struct Args {
  const uint16_t* q;
  const int32_t* lens;
  uint16_t* out;
  int64_t q_stride, out_stride;
  int G, nhb;          // query heads per K/V head; row sets per K/V head
  int window, sinks;
  float scale_log2;
  Cut* cuts;           // [warps]
  float* partial;      // [2 * warps][kHeads][D + 2]
};

// 2^x on the special-function unit (x <= 2 here; results below 2^-126 flush to zero)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, unsigned int err) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (clock64() - t0 > kWaitCycles) {
      atomicOr(&g_decode_window_error, err);
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

// A sequence's length, 0 when it does not fit the cache.
__device__ __forceinline__ int length_of(const Args& a, const fg_kvcache& kv, int b) {
  const int len = a.lens[b];
  return (len < 0 || len > kv.cap) ? 0 : len;
}

// A place in the work order: tile u of row set rs of sequence b.
struct Cursor {
  int b, rs, u;
  SeqTiles s;
};
__device__ __forceinline__ void next_row_set(Cursor& c, const Args& a, const fg_kvcache& kv) {
  c.u = 0;
  if (++c.rs < kv.H * a.nhb) return;
  c.rs = 0;
  do {
    if (++c.b >= kv.B) {                   // the end of the order: never asked for
      c.b = kv.B - 1;
      return;
    }
    c.s = seq_tiles(length_of(a, kv, c.b), a.window, a.sinks);
  } while (c.s.nt == 0);
}

// The query heads of a row set as B fragments (column n = gid: head gid / 2, group gid & 1; indexes
// permuted as the lanes hold the codes), the group sums of head tig and the code-scale factor, in
// the base-2 score scale.
template <int D>
struct QFrag {
  uint32_t bq[2 * (D / 32)][2];
  float Q[D / 64];
};
template <int D>
__device__ __forceinline__ void load_q(const uint16_t* q_heads, int heads, int lane,
                                       float scale_log2, QFrag<D>& f) {
  constexpr int NW = D / 32, NG = D / 64;
  const int gid = lane >> 2, tig = lane & 3;
  uint32_t qw[NW * 4];
#pragma unroll
  for (int c = 0; c < NW; ++c) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if ((gid >> 1) < heads) u = ldg_nc_v4(q_heads + (gid >> 1) * D + tig * 8 * NW + 8 * c);
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
  for (int g = 0; g < NG; ++g)              // head tig: lanes gid = 2 tig, tig = 2 g
    f.Q[g] = __shfl_sync(0xFFFFFFFFu, qsum, 8 * tig + 2 * g) * scale_log2;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
decode_window_kernel(const Args a, const fg_kvcache kv) {
  using R = Ring<D>;
  constexpr int NW = D / 32, NG = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * kRing * R::SLOT;
  const uint32_t bar0 = smem_u32(smem + kWarps * kRing * R::SLOT) + warp * kRing * 8;
  if (lane == 0) {
    for (int i = 0; i < kRing; ++i) mbar_init(bar0 + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  pdl_launch_dependents();
  pdl_wait();

  // ---- the order of the work: tiles of all sequences, and this warp's share.  Neighbouring
  // warps of the order sit on different SMs, so a small call spreads over the GPU.
  const int nwarps = gridDim.x * kWarps, w = warp * gridDim.x + blockIdx.x;
  const int rsets = kv.H * a.nhb;          // row sets of one sequence
  int64_t tiles = 0;
  for (int b0 = 0; b0 < kv.B; b0 += 32) {
    const int b = b0 + lane;
    const unsigned nt = b < kv.B ? seq_tiles(length_of(a, kv, b), a.window, a.sinks).nt : 0;
    tiles += __reduce_add_sync(0xFFFFFFFFu, nt);
  }
  for (int b = w; b < kv.B; b += nwarps) {  // sequences that see nothing
    const int len = a.lens[b];
    if (lane == 0 && (len < 0 || len > kv.cap)) atomicOr(&g_decode_window_error, kErrExtent);
    if (length_of(a, kv, b) == 0)
      for (int i = lane; i < rsets / a.nhb * a.G * (D / 8); i += 32)
        reinterpret_cast<uint4*>(a.out + b * a.out_stride)[i] = make_uint4(0, 0, 0, 0);
  }
  const int64_t total = tiles * rsets;
  const int nw = (int)max((int64_t)1, min((int64_t)nwarps, total / kMinTiles));
  Cut cut{};
  if (w >= nw || total == 0) {
    if (lane == 0) a.cuts[w] = cut;
    return;
  }
  const int64_t x0 = first_tile(total, nw, w), x1 = first_tile(total, nw, w + 1);
  Cursor cc{};                              // compute cursor
  {
    int64_t before = 0;                     // tiles of earlier sequences, once per row set
    for (int b0 = 0;; b0 += 32) {
      const int b = b0 + lane;
      const unsigned nt = b < kv.B ? seq_tiles(length_of(a, kv, b), a.window, a.sinks).nt : 0;
      unsigned incl = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      const unsigned past = __ballot_sync(0xFFFFFFFFu, (before + incl) * rsets > x0);
      if (past) {
        const int l = __ffs(past) - 1;
        cc.b = b0 + l;
        before += __shfl_sync(0xFFFFFFFFu, incl - nt, l);
        break;
      }
      before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (b0 + 32 >= kv.B) return;          // not reached: x0 < total
    }
    cc.s = seq_tiles(length_of(a, kv, cc.b), a.window, a.sinks);
    const int64_t rel = x0 - before * rsets;
    cc.rs = (int)(rel / cc.s.nt);
    cc.u = (int)(rel - (int64_t)cc.rs * cc.s.nt);
    // what has to be merged: this warp speaks for the row set it begins inside of, when the warp
    // before holds that row set's first tile
    const int64_t r0 = x0 - cc.u;
    if (cc.u > 0) {
      const int64_t xp = first_tile(total, nw, w - 1);
      if (xp <= r0) {
        const int hk = cc.rs / a.nhb, hb = cc.rs - hk * a.nhb;
        cut.pieces = worker_of_tile(total, nw, r0 + cc.s.nt - 1) - (w - 1) + 1;
        cut.b = cc.b;
        cut.hq = hk * a.G + hb * kHeads;
        cut.heads = min(kHeads, a.G - hb * kHeads);
        cut.prev_slot = 2 * (w - 1) + (xp == r0 ? 0 : 1);
      }
    }
    if (lane == 0) a.cuts[w] = cut;
  }

  // ---- the issue cursor, kRing slots ahead of the compute cursor
  Cursor ic = cc;
  int ileft = (int)(x1 - x0);              // the scratch and the cache bound it far below 2^31
  int is = 0, issued = 0;
  auto issue = [&]() {
    if (ileft <= 0) return;
    const int u1 = min(ic.s.nt, ic.u + ileft);
    const int cnt = slot_tiles(ic.s, ic.u, u1, kSub);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * is;
      uint8_t* slot = ring + is * R::SLOT;
      const uint32_t rows = cnt * kTilePos;          // whole tiles: never past cap
      const int64_t row0 =
          ((int64_t)ic.b * kv.H + ic.rs / a.nhb) * kv.cap + tile_pos(ic.s, ic.u);
      // the slot was last read through the generic proxy; order that before the copy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_expect_tx(bar, rows * 2 * (R::ROW_CODE + R::ROW_AB));
      bulk_copy(smem_u32(slot), kv.k_codes + row0 * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(smem_u32(slot + R::KAB_OFF), kv.k_ab + row0 * NG, rows * R::ROW_AB, bar);
      bulk_copy(smem_u32(slot + R::V_OFF), kv.v_codes + row0 * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(smem_u32(slot + R::VAB_OFF), kv.v_ab + row0 * NG, rows * R::ROW_AB, bar);
    }
    ++issued;
    if (++is == kRing) is = 0;
    ileft -= cnt;
    ic.u += cnt;
    if (ic.u == ic.s.nt && ileft > 0) next_row_set(ic, a, kv);
  };
  for (int i = 0; i < kRing; ++i) issue();

  const float ck = (16777216.0f / 15.0f) * a.scale_log2;
  int cs = 0, consumed = 0;
  uint32_t cph = 0;
  int left = (int)(x1 - x0);
  bool ok = true;
  for (int seg_no = 0; left > 0 && ok; ++seg_no) {
    const int u1 = min(cc.s.nt, cc.u + left);
    const bool whole = cc.u == 0 && u1 == cc.s.nt;
    const int seg = u1 - cc.u;
    const int hk = cc.rs / a.nhb, hb = cc.rs - hk * a.nhb;
    const int hq = hk * a.G + hb * kHeads, heads = min(kHeads, a.G - hb * kHeads);
    QFrag<D> qf;
    load_q<D>(a.q + cc.b * a.q_stride + (int64_t)hq * D, heads, lane, a.scale_log2, qf);

    // head tig, the lane's rows (l, asum) and channels (acc)
    float m_run = -INFINITY, l_run = 0.0f;
    float acc[2 * NW][4], asum[NG];
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[u][c] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) asum[g] = 0.0f;

    // One slot: scores of every tile, one softmax step, the values of every tile.  MASK: positions
    // that are not visible, and tiles the copy left out (whose stale bytes are still codes), get
    // weight 0 by selects on the score and on the statistics.
    auto process = [&](const uint8_t* slot, int ts, int cnt, auto mask_tag) {
      constexpr bool MASK = decltype(mask_tag)::value;
      auto valid = [&](int sub, int r) {
        const int t = ts + sub * kTilePos + gid + 8 * r;
        return !MASK || (sub < cnt && t < cc.s.len && (t >= cc.s.wstart || t < a.sinks));
      };
      float sc[kSub][2];
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        uint32_t kw[2][NW], ka[2][NG];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = sub * kTilePos + gid + 8 * r;
          load_words<NW>(slot + row * R::ROW_CODE + tig * 4 * NW, kw[r]);
          load_words<NG>(slot + R::KAB_OFF + row * R::ROW_AB, ka[r]);
        }
        float dk[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int wd = 0; wd < NW; ++wd) {
          uint32_t c0[4], c1[4];
          q4attn::code_pairs(kw[0][wd], c0);
          q4attn::code_pairs(kw[1][wd], c1);
          mma16816(dk, c0[0], c1[0], c0[1], c1[1], qf.bq[2 * wd][0], qf.bq[2 * wd][1]);
          mma16816(dk, c0[2], c1[2], c0[3], c1[3], qf.bq[2 * wd + 1][0], qf.bq[2 * wd + 1][1]);
        }
        // dk[2r], dk[2r + 1]: row gid + 8r, head tig, groups 0 and 1
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float dot = 0.0f, off = 0.0f;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float2 ab = unpack_h2(ka[r][g]);
            dot = fmaf(ab.y - ab.x, dk[2 * r + g], dot);
            off = fmaf(ab.x, qf.Q[g], off);
          }
          const float s = fmaf(dot, ck, off);
          sc[sub][r] = valid(sub, r) ? s : -INFINITY;
        }
      }
      // The reference maximum moves only when a score exceeds it by more than 2^2, so that p <= 4
      // and the fp16 weight p (b - a) / 15 cannot overflow (131008 / 15 * 4 < 65504).
      float mloc = fmaxf(sc[0][0], sc[0][1]);
#pragma unroll
      for (int sub = 1; sub < kSub; ++sub) mloc = fmaxf(mloc, fmaxf(sc[sub][0], sc[sub][1]));
      if (__any_sync(0xFFFFFFFFu, mloc > m_run + 2.0f)) {
        float mx = fmaxf(mloc, m_run);
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        const float corr = (m_run == -INFINITY) ? 0.0f : ex2(m_run - mx);
        l_run *= corr;
#pragma unroll
        for (int g = 0; g < NG; ++g) asum[g] *= corr;
        // acc column 2 tig + g belongs to head tig as well
#pragma unroll
        for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[u][c] *= corr;
        m_run = mx;
      }
      const float m_ref = (m_run == -INFINITY) ? 0.0f : m_run;
      float p[kSub][2];
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        p[sub][0] = ex2(sc[sub][0] - m_ref);
        p[sub][1] = ex2(sc[sub][1] - m_ref);
        l_run += p[sub][0] + p[sub][1];
      }
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        uint32_t vw[2][NW], wrow[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = sub * kTilePos + gid + 8 * r;
          uint32_t va[NG];
          load_words<NW>(slot + R::V_OFF + row * R::ROW_CODE + tig * 4 * NW, vw[r]);
          load_words<NG>(slot + R::VAB_OFF + row * R::ROW_AB, va);
          const float p15 = p[sub][r] * (1.0f / 15.0f);
          float wt[2];
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float2 ab = unpack_h2(valid(sub, r) ? va[g] : 0u);
            wt[g] = p15 * (ab.y - ab.x);
            asum[g] = fmaf(p[sub][r], ab.x, asum[g]);
          }
          wrow[r] = pack_h2(wt[0], NG == 2 ? wt[NG - 1] : wt[0]);
        }
        // rows x (head, group) -> the B operand: (head, group) x rows
        const uint32_t bv0 = movtrans(wrow[0]), bv1 = movtrans(wrow[1]);
#pragma unroll
        for (int wd = 0; wd < NW; ++wd) {
          uint32_t c0[4], c1[4];
          q4attn::code_pairs(movtrans(vw[0][wd]), c0);
          q4attn::code_pairs(movtrans(vw[1][wd]), c1);
          mma16816(acc[2 * wd], c0[0], c0[1], c1[0], c1[1], bv0, bv1);
          mma16816(acc[2 * wd + 1], c0[2], c0[3], c1[2], c1[3], bv0, bv1);
        }
      }
    };

    while (cc.u < u1) {
      const int cnt = slot_tiles(cc.s, cc.u, u1, kSub), ts = tile_pos(cc.s, cc.u);
      ok = __all_sync(0xFFFFFFFFu, bounded_wait(bar0 + 8 * cs, cph, kErrWait));
      if (!ok) break;
      const uint8_t* slot = ring + cs * R::SLOT;
      const int te = ts + kSlotPos;
      if (cnt == kSub && te <= cc.s.len && (ts >= cc.s.wstart || te <= a.sinks))
        process(slot, ts, cnt, std::false_type{});
      else
        process(slot, ts, cnt, std::true_type{});
      __syncwarp();                         // every lane has read the slot: refill it
      issue();
      ++consumed;
      if (++cs == kRing) {
        cs = 0;
        cph ^= 1u;
      }
      cc.u += cnt;
    }
    if (!ok) break;

    // ---- end of the segment
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, o);
#pragma unroll
      for (int g = 0; g < NG; ++g) asum[g] += __shfl_xor_sync(0xFFFFFFFFu, asum[g], o);
    }
    if (tig < heads) {
      const int g = (NG == 2) ? (gid >> 2) : 0;        // group of the lane's channels
      const float A = (NG == 2 && g) ? asum[NG - 1] : asum[0];
      const int cbase = 8 * NW * (gid >> 1) + 4 * (gid & 1);
      const float inv = (l_run == 0.0f) ? 0.0f : 1.0f / l_run;
      uint16_t* o = a.out + cc.b * a.out_stride + (int64_t)(hq + tig) * D;
      float* pp = a.partial + ((int64_t)(2 * w + (seg_no > 0)) * kHeads + tig) * (D + 2);
#pragma unroll
      for (int u = 0; u < 2 * NW; ++u) {
        const int ch = cbase + 8 * (u >> 1) + 2 * (u & 1);
        const float y0 = fmaf(g ? acc[u][1] : acc[u][0], 16777216.0f, A);
        const float y1 = fmaf(g ? acc[u][3] : acc[u][2], 1048576.0f, A);
        if (whole)
          *reinterpret_cast<uint32_t*>(o + ch) = pack_h2(in_range(y0 * inv), in_range(y1 * inv));
        else
          *reinterpret_cast<float2*>(pp + ch) = make_float2(y0, y1);
      }
      if (!whole && gid == 0) *reinterpret_cast<float2*>(pp + D) = make_float2(m_run, l_run);
    }
    __syncwarp();
    left -= seg;
    if (left > 0) next_row_set(cc, a, kv);
  }

  // ---- every issued copy lands before the warp's shared memory is released
  for (int i = consumed; i < issued; ++i)
    bounded_wait(bar0 + 8 * (uint32_t)(i % kRing), (uint32_t)((i / kRing) & 1), kErrDrain);
}

// One warp per (cut, head of its row set): merges the pieces (m, l, unnormalised o) in order.
template <int D>
__global__ void __launch_bounds__(kHeads * 32)
merge_kernel(const Args a) {
  pdl_launch_dependents();
  pdl_wait();
  const Cut cut = a.cuts[blockIdx.x];
  const int head = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (cut.pieces == 0 || head >= cut.heads) return;
  auto piece = [&](int i) {
    const int slot = i == 0 ? cut.prev_slot : 2 * ((int)blockIdx.x + i - 1);
    return a.partial + ((int64_t)slot * kHeads + head) * (D + 2);
  };
  float M = -INFINITY;
  for (int i = lane; i < cut.pieces; i += 32) M = fmaxf(M, piece(i)[D]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  if (M == -INFINITY) M = 0.0f;
  constexpr int C = D / 32;
  float L = 0.0f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < cut.pieces; ++i) {
    const float* pp = piece(i);
    const float wgt = exp2f(pp[D] - M);
    L = fmaf(wgt, pp[D + 1], L);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(wgt, pp[c * 32 + lane], o[c]);
  }
  const float inv = (L == 0.0f) ? 0.0f : 1.0f / L;
  uint16_t* op = a.out + cut.b * a.out_stride + (int64_t)(cut.hq + head) * D;
#pragma unroll
  for (int c = 0; c < C; ++c) op[c * 32 + lane] = f2h(in_range(o[c] * inv));
}

// The most tiles a call can have: every sequence full, or its window and first positions.
int64_t most_tiles(const fg_kvcache& kv, int nhb, int window, int sinks) {
  const SeqTiles s = seq_tiles(kv.cap, window, sinks);
  return (int64_t)kv.B * kv.H * nhb * (s.nt + 2);
}
int grid_ctas(const fg_kvcache& kv, int nhb, int window, int sinks, int nsm) {
  const int64_t want = most_tiles(kv, nhb, window, sinks) / (kMinTiles * kWarps) + 1;
  return (int)std::min<int64_t>(want, (int64_t)nsm * kCtasPerSm);
}
size_t cut_bytes(int ctas) { return ((size_t)ctas * kWarps * sizeof(Cut) + 255) / 256 * 256; }

// Shared memory and carveout of the kernel on the current device, set once per device.
template <int D>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 0 || dev >= 64 || done[dev]) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(decode_window_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Ring<D>::CTA_BYTES)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(decode_window_kernel<D>,
                                cudaFuncAttributePreferredSharedMemoryCarveout, 100)) != cudaSuccess)
    return e;
  done[dev] = true;
  return cudaSuccess;
}

template <int D>
cudaError_t launch_d(const Args& a, const fg_kvcache& kv, int ctas, cudaStream_t st) {
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_window_kernel<D>, dim3(ctas), dim3(kWarps * 32), Ring<D>::CTA_BYTES, st, a,
                 kv);
  if (e != cudaSuccess) return e;
  return launch_pdl(merge_kernel<D>, dim3(ctas * kWarps), dim3(kHeads * 32), 0, st, a);
}

int head_blocks(int G) { return (G + kHeads - 1) / kHeads; }

}  // namespace

size_t decode_attn_window_ws_bytes(const fg_kvcache& kv, int32_t Hq) {
  const int ctas = grid_ctas(kv, head_blocks(Hq / kv.H), 0, 0, kMaxSms);
  return cut_bytes(ctas) + (size_t)ctas * kWarps * 2 * kHeads * (kv.h / kv.H + 2) * sizeof(float);
}

cudaError_t launch_decode_attn_window(const uint16_t* q, int64_t q_stride, int32_t Hq,
                                      const fg_kvcache& kv, const int32_t* lens, int32_t window,
                                      int32_t sinks, float scale, uint16_t* out,
                                      int64_t out_stride, void* ws, int nsm, cudaStream_t st) {
  Args a;
  a.q = q;
  a.lens = lens;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.G = Hq / kv.H;
  a.nhb = head_blocks(a.G);
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int ctas = std::min(grid_ctas(kv, a.nhb, window, sinks, nsm),
                            grid_ctas(kv, a.nhb, 0, 0, kMaxSms));
  a.cuts = static_cast<Cut*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + cut_bytes(ctas));
  return kv.h / kv.H == 128 ? launch_d<128>(a, kv, ctas, st) : launch_d<64>(a, kv, ctas, st);
}

cudaError_t decode_window_read_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_decode_window_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_decode_window_error, &zero, sizeof(unsigned int));
}

}  // namespace fg
