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
// Columns: the 8 columns of a product are (part, query head, group) with NP parts of HEADS = 4 / NP
// query heads of one K/V head (for d = 64 the second column of a group pair repeats the first), so
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
// codes and statistics), filled by bulk async copies that run ahead across row sets.  Every wait is
// bounded; on timeout the warp sets the device error word, drains its copies and stops.
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

constexpr int kSub = 2;                   // tiles per ring slot
constexpr int kSlotPos = kSub * kTilePos;
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
// 2).
template <int D>
struct Ring {
  static constexpr int WARPS = (D == 128) ? 12 : 16, DEPTH = (D == 128) ? 2 : 3;
  static constexpr int NG = D / 64;
  static constexpr int ROW_CODE = D / 2;                // code bytes of one position
  static constexpr int ROW_AB = NG * 4;                 // statistics bytes of one position
  static constexpr int V_OFF = kSlotPos * ROW_CODE;     // V codes in a slot
  static constexpr int KAB_OFF = 2 * V_OFF;
  static constexpr int VAB_OFF = KAB_OFF + kSlotPos * ROW_AB;
  static constexpr int SLOT = VAB_OFF + kSlotPos * ROW_AB;
  static constexpr int CTA_BYTES = WARPS * DEPTH * (SLOT + 8);
};
static_assert(Ring<128>::CTA_BYTES + 1024 <= 227 * 1024, "shared memory per CTA");

// What is to be merged at the cut before a warp's share: the pieces of the row set that it begins
// inside of, when the share before holds that row set's first tile.
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
  int ncuts;           // the grid's warps
  Cut* cuts;           // [ncuts]
  float* partial;      // [2 * ncuts][HEADS][D + 2]
};

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
// The K/V head of a row set (most calls have one row set each: no division for them).
__device__ __forceinline__ int kv_head(int rs, const Args& a) {
  return a.nhb == 1 ? rs : rs / a.nhb;
}
// Moves to the next sequence that sees something, found by the whole warp 32 at a time (a batch
// may have many empty places).
__device__ __forceinline__ bool next_sequence(Cursor& c, const Args& a, const fg_kvcache& kv) {
  const int lane = threadIdx.x & 31;
  for (int b = c.b + 1; b < kv.B; b += 32) {
    const int len = b + lane < kv.B ? length_of(a, kv, b + lane) : 0;
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
__device__ __forceinline__ void next_row_set(Cursor& c, const Args& a, const fg_kvcache& kv) {
  c.u = 0;
  if (++c.rs < kv.H * a.nhb) return;
  c.rs = 0;
  next_sequence(c, a, kv);
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

// Moves a place dx tiles on in the order.
__device__ __forceinline__ void skip_tiles(Cursor& c, int64_t dx, const Args& a,
                                           const fg_kvcache& kv) {
  const int rsets = kv.H * a.nhb;
  int64_t at = (int64_t)c.rs * c.s.nt + c.u + dx;        // within sequence b
  while (at >= (int64_t)rsets * c.s.nt) {
    at -= (int64_t)rsets * c.s.nt;
    if (!next_sequence(c, a, kv)) return;
  }
  c.rs = at < 0x7FFFFFFF ? (int)((unsigned)at / (unsigned)c.s.nt) : (int)(at / c.s.nt);
  c.u = (int)(at - (int64_t)c.rs * c.s.nt);
}

template <int D, int NP>
__global__ void __launch_bounds__(Ring<D>::WARPS * 32, 1)
decode_window_kernel(const Args a, const fg_kvcache kv) {
  using R = Ring<D>;
  constexpr int kWarps = R::WARPS, kRing = R::DEPTH;
  constexpr int NW = D / 32, NG = D / 64;
  constexpr int HEADS = 4 / NP, RPL = 4 / NP;   // heads of a row set; rows of a slot per lane
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned warp_nt[kWarps];
  __shared__ int first_b;                  // the sequence of the CTA's first tile,
  __shared__ int64_t first_before;         // and the tiles of the sequences before it
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3, part = tig / HEADS;
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
    mine = b < kv.B ? seq_tiles(length_of(a, kv, b), a.window, a.sinks).nt : 0;
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
  int64_t irow = 0;                        // the run's next position, as a row of the cache
  Cursor ic{};
  const bool has_share = busy && warp < per_cta && w < n;
  if (has_share) {
    const int64_t x0 = shares.first(w);
    ileft = (int)(shares.first(w + 1) - x0);           // the host bounds the call's tiles by 2^40
    ic.b = first_b;
    ic.s = seq_tiles(length_of(a, kv, ic.b), a.window, a.sinks);
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
        const int hq = hk * a.G + (ic.rs - hk * a.nhb) * HEADS + (lane >> 3);
        if ((lane >> 3) < HEADS && hq < hk * a.G + a.G && (lane & 7) * 16 < D)
          prefetch_l2(a.q + ic.b * a.q_stride + (int64_t)hq * D + (lane & 7) * 16);
      }
      irun = run_tiles(ic.s, ic.u, min(ic.s.nt, ic.u + ileft));
      irow = ((int64_t)ic.b * kv.H + kv_head(ic.rs, a)) * kv.cap + tile_pos(ic.s, ic.u);
      ic.u += irun;
      ileft -= irun;
    }
    const int cnt = min(kSub, irun);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * is, rows = cnt * kTilePos;   // whole tiles: never past cap
      const uint32_t slot = ring0 + is * R::SLOT;
      // the slot was last read through the generic proxy; order that before the copy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_expect_tx(bar, rows * 2 * (R::ROW_CODE + R::ROW_AB));
      bulk_copy(slot, kv.k_codes + irow * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(slot + R::KAB_OFF, kv.k_ab + irow * NG, rows * R::ROW_AB, bar);
      bulk_copy(slot + R::V_OFF, kv.v_codes + irow * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(slot + R::VAB_OFF, kv.v_ab + irow * NG, rows * R::ROW_AB, bar);
    }
    irow += cnt * kTilePos;
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
    const int len = a.lens[b];
    if (lane == 0 && (len < 0 || len > kv.cap)) atomicOr(&g_decode_window_error, kErrExtent);
    if (length_of(a, kv, (int)b) == 0)
      for (int i = lane; i < kv.H * a.G * (D / 8); i += 32)
        reinterpret_cast<uint4*>(a.out + b * a.out_stride)[i] = make_uint4(0, 0, 0, 0);
  }
  for (int c = (total > 0 ? n : 0) + blockIdx.x * kWarps * 32 + threadIdx.x; c < a.ncuts;
       c += gridDim.x * kWarps * 32)
    a.cuts[c].pieces = 0;

  const float ck = (16777216.0f / 15.0f) * a.scale_log2;
  int cs = 0, consumed = 0;
  uint32_t cph = 0;
  bool ok = true;
  for (int seg_no = 0; left > 0 && ok; ++seg_no) {
    const int u1 = min(cc.s.nt, cc.u + left);
    const bool whole = cc.u == 0 && u1 == cc.s.nt;
    const int seg = u1 - cc.u;
    const int hk = kv_head(cc.rs, a), hb = cc.rs - hk * a.nhb;
    const int hq = hk * a.G + hb * HEADS, heads = min(HEADS, a.G - hb * HEADS);
    QFrag<D> qf;
    load_q<D, HEADS>(a.q + cc.b * a.q_stride + (int64_t)hq * D, heads, lane, a.scale_log2, qf);

    // head tig % HEADS: the part's rows (l, asum) and columns (acc)
    float m_run = -INFINITY, l_run = 0.0f;
    float acc[2 * NW][4], asum[NG], wsum[NG], f[NG];   // acc and wsum: times f
#pragma unroll
    for (int u = 0; u < 2 * NW; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[u][c] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      asum[g] = wsum[g] = 0.0f;
      f[g] = kFirstF;
    }
    int slots = 0;

    // One slot: scores of every tile, one softmax step, the values of every tile.  MASK: positions
    // that are not visible, and tiles the copy left out (whose stale bytes are still codes), get
    // weight 0 by selects on the score and on the statistics.
    auto process = [&](const uint8_t* slot, int ts, int cnt, auto mask_tag) {
      constexpr bool MASK = decltype(mask_tag)::value;
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
        valid[j] = !MASK || (row < cnt * kTilePos && t < cc.s.len &&
                             (t >= cc.s.wstart || t < a.sinks));
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
    };

    // Codes are not negative: sums of them grow with the positions, while the output, a mean of
    // values of both signs, gets smaller, and the products' additions truncate.  So every kRecentre
    // slots the codes' middle times the weights since then moves from these sums to those of the
    // minima, binary32 additions of a lane's own.  Relative error of outputs over 65536 positions a
    // warp: 3.5e-4 (without it 6e-2); 1% of the time.
    auto recentre = [&]() {
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
    };

    while (cc.u < u1 && ok) {
      int run = run_tiles(cc.s, cc.u, u1), ts = tile_pos(cc.s, cc.u);
      cc.u += run;
      for (; run > 0; run -= kSub, ts += kSlotPos) {
        ok = __all_sync(0xFFFFFFFFu, bounded_wait(bar0 + 8 * cs, cph, kErrWait));
        if (!ok) break;
        const uint8_t* slot = ring + cs * R::SLOT;
        const int te = ts + kSlotPos;
        if (run >= kSub && te <= cc.s.len && (ts >= cc.s.wstart || te <= a.sinks))
          process(slot, ts, kSub, std::false_type{});
        else
          process(slot, ts, min(run, kSub), std::true_type{});
        __syncwarp();                       // every lane has read the slot: refill it
        issue();
        if ((++slots & (kRecentre - 1)) == 0) recentre();
        ++consumed;
        if (++cs == kRing) {
          cs = 0;
          cph ^= 1u;
        }
      }
    }
    if (!ok) break;

    // ---- end of the segment: sums over the rows' lanes and the parts
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
    if (head < heads) {
      const float inv = (l_run == 0.0f) ? 0.0f : 1.0f / l_run;
      uint16_t* o = a.out + cc.b * a.out_stride + (int64_t)(hq + head) * D;
      float* pp = a.partial + ((int64_t)(2 * w + (seg_no > 0)) * HEADS + head) * (D + 2);
#pragma unroll
      for (int i = 0; i < NY; ++i) {
        const int ch = cbase + 8 * ((u0 + i) >> 1) + 2 * ((u0 + i) & 1);
        const float y0 = y[i].x + A, y1 = y[i].y + A;
        if (whole)
          *reinterpret_cast<uint32_t*>(o + ch) =
              pack_h2(in_range(y0 * inv), in_range(y1 * inv));
        else
          *reinterpret_cast<float2*>(pp + ch) = make_float2(y0, y1);
      }
      if (!whole && gid == 0 && part == 0)
        *reinterpret_cast<float2*>(pp + D) = make_float2(m_run, l_run);
    }
    __syncwarp();
    left -= seg;
    if (left > 0) next_row_set(cc, a, kv);
  }

  // ---- every issued copy lands before the warp's shared memory is released
  for (int i = consumed; i < issued; ++i)
    bounded_wait(bar0 + 8 * (uint32_t)(i % kRing), (uint32_t)((i / kRing) & 1), kErrDrain);
}

// One warp per (cut, head of its row set): merges the pieces (m, l, unnormalised o) in order,
// 32 at a time: a lane takes one piece's m and l, then all lanes that piece's channels.
template <int D, int HEADS>
__global__ void __launch_bounds__(HEADS * 32)
merge_kernel(const Args a) {
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
  uint16_t* op = a.out + cut.b * a.out_stride + (int64_t)(cut.hq + head) * D;
#pragma unroll
  for (int c = 0; c < C; ++c) op[c * 32 + lane] = f2h(in_range(o[c] * inv));
}

// The most tiles a call can have: every sequence full, or its window and first positions.
int64_t most_tiles(const fg_kvcache& kv, int nhb, int window, int sinks) {
  const SeqTiles s = seq_tiles(kv.cap, window, sinks);
  return (int64_t)kv.B * kv.H * nhb * (s.nt + 2);
}
int grid_ctas(int64_t most, int nsm) {
  return (int)std::min<int64_t>(most / kMinTiles + 1, std::max(nsm, 1));
}
size_t cut_bytes(int64_t ncuts) { return ((size_t)ncuts * sizeof(Cut) + 255) / 256 * 256; }

// Shared memory and carveout of the kernel on the current device, set once per device.
template <int D, int NP>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 0 || dev >= 64 || done[dev]) return cudaSuccess;
  auto* kernel = decode_window_kernel<D, NP>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Ring<D>::CTA_BYTES)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100)) !=
          cudaSuccess)
    return e;
  done[dev] = true;
  return cudaSuccess;
}

template <int D, int NP>
cudaError_t launch_d(const Args& a, const fg_kvcache& kv, int ctas, cudaStream_t st) {
  cudaError_t e = prepare<D, NP>();
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_window_kernel<D, NP>, dim3(ctas), dim3(Ring<D>::WARPS * 32),
                 Ring<D>::CTA_BYTES, st, a, kv);
  if (e != cudaSuccess) return e;
  return launch_pdl(merge_kernel<D, 4 / NP>, dim3(a.ncuts), dim3(4 / NP * 32), 0, st, a);
}

int warps_of(int d) { return d == 128 ? Ring<128>::WARPS : Ring<64>::WARPS; }
// Shares that a call of at most `most` tiles can have.
int64_t most_cuts(int64_t most, int nsm, int d) {
  return std::min<int64_t>(most / kMinTiles + 1, (int64_t)grid_ctas(most, nsm) * warps_of(d));
}
// Query heads of a row set: 1, 2 or 4.
int set_heads(int G) { return G < 3 ? G : 4; }

}  // namespace

size_t decode_attn_window_ws_bytes(const fg_kvcache& kv, int32_t Hq) {
  const int G = Hq / kv.H, heads = set_heads(G);
  const int64_t n = most_cuts(most_tiles(kv, (G + heads - 1) / heads, 0, 0), kMaxSms, kv.h / kv.H);
  return cut_bytes(n) + (size_t)n * 2 * heads * (kv.h / kv.H + 2) * sizeof(float);
}

cudaError_t launch_decode_attn_window(const uint16_t* q, int64_t q_stride, int32_t Hq,
                                      const fg_kvcache& kv, const int32_t* lens, int32_t window,
                                      int32_t sinks, float scale, uint16_t* out,
                                      int64_t out_stride, void* ws, int nsm, cudaStream_t st) {
  const int G = Hq / kv.H, heads = set_heads(G);
  Args a;
  a.q = q;
  a.lens = lens;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.G = G;
  a.nhb = (G + heads - 1) / heads;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int64_t most = std::min(most_tiles(kv, a.nhb, window, sinks), most_tiles(kv, a.nhb, 0, 0));
  const int ctas = grid_ctas(most, nsm);
  a.ncuts = (int)most_cuts(most, nsm, kv.h / kv.H);
  a.cuts = static_cast<Cut*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + cut_bytes(a.ncuts));
  const bool wide = kv.h / kv.H == 128;
  auto* launch = heads == 1   ? (wide ? launch_d<128, 4> : launch_d<64, 4>)
                 : heads == 2 ? (wide ? launch_d<128, 2> : launch_d<64, 2>)
                              : (wide ? launch_d<128, 1> : launch_d<64, 1>);
  return launch(a, kv, ctas, st);
}

cudaError_t decode_window_read_error(unsigned int* out) {
  return read_and_clear(g_decode_window_error, out);
}

}  // namespace fg
