// Prefill attention over fp16 K/V rows of sequences of different lengths, with a sliding window,
// first positions that stay visible, and query heads that share K/V heads, on the 5th-generation
// tensor cores (sm_103a).
//
// Sequence b has nq = q_off[b+1] - q_off[b] query rows and nk = kv_off[b+1] - kv_off[b] K/V rows;
// query row r is position i = nk - nq + r (the newest positions), and
//   out_r,hq = sum_t softmax_t(scale * q_r,hq . k_t) v_t   over the t that i sees,
// K/V head hq / G of G = Hq / Hkv query heads each; a row that sees nothing gets zeros.
//
// A CTA owns a block of 256 query rows of one (sequence, query head): two Q tiles (A, B) of 128
// rows that share the K/V tiles of 128 keys.  The key tiles of a block are those that one of its
// rows sees (first positions, then the window; key_tiles in ragged.cuh): a window costs what it
// shows, not the sequence.  Q, K and V are read in place by TMA (boxes of 64 columns x 128 rows,
// 128B swizzle) at the sequence's own rows, so a box may end in another sequence's rows or past the
// buffer (zeros); such rows are masked or not stored.
//   S = Q K^T     tcgen05.mma kind::f16, S (fp32) in TMEM
//   softmax       one thread per query row, two passes over its 128 key columns in TMEM (the
//                 maximum, then P): base-2 online softmax with a lazily moved reference maximum
//                 (by more than 2^8), P = 2^(s - m + 7) rounded to fp16 over S's columns (at most
//                 2^15: what is 14 nats below the maximum is still a normal number).  Tiles that
//                 every row of the Q tile sees in full are not masked; the others take a bit mask
//                 per row.
//   O += P V      tcgen05.mma with P from TMEM
// TMEM: S of A and B (128 columns each), O of A and B (d columns each).  A Q tile takes part only
// in the key tiles that it sees, and in the 16-key steps of them that it sees.
//   warp 0       TMA producer: K tiles, V tiles and Q, rings of two each
//   warps 1, 2   MMA issuers of Q tiles A and B: S_t(0); then per key tile P_t(j) V_j, S_t(j + 1)
//   warps 3-10   softmax of A and B (TMEM lanes 32 (w % 4) ..)
//   warps 11-14  output: O_t / l of a finished block, 32 rows a warp, staged in shared memory and
//                stored by TMA
//   warp 15      the work items
//
// A sequence of up to 128 query rows has no second Q tile.  Both tiles then hold its rows, take
// every other of its key tiles, and are joined at the output (a piece of 100 rows behind 4000 x 32
// heads 50 -> 38 us, 64 of them behind 300 with 64 channels 92 -> 84 us, behind 30 59 -> 58 us).
// The last block of a longer sequence is left to one tile: the other one works on the next item
// meanwhile (ragged prompts 61 us; 63 us with such blocks split).
//
// Masked keys.  A masked key has P = 0, but 0 times an infinity or a NaN in its V row is NaN: it
// would reach the rows of the Q tile that do not see it.  The output warps therefore test their
// rows: a row with an infinity or a NaN is computed again on its own, over its visible keys alone
// (attend_rows), so that only what it sees can reach it.  A row whose sum of weights is NaN has its
// answer: masked scores take no part in that sum, so one that it sees is NaN or infinite.  Finite
// inputs take the path only where rounding carries an output past fp16's range.  The rows behind a
// sequence in its last 16-key step, which may hold anything, are zeroed in shared memory first.
//
// The work order: blocks by descending index, for each the sequences that have one (longest first),
// for each the query heads (which share K/V in L2).  One persistent CTA per SM; offsets are read
// and checked on the device, kMaxSeqs sequences per launch.  A warp of its own works the items out
// and hands them to the others through a ring in shared memory (by the producer, between its loads:
// the 8k window 249 us instead of 246).
//
// What bounds it: the turn that a Q tile takes -- P V and S (16 MMAs, 1024 cycles of tensor work),
// the softmax (about 400 cycles for the maximum, 900 for P: 128 exponentials a thread, 512 cycles
// of the special-function unit), and the barriers between -- with two Q tiles taking turns: 3200
// cycles for a pair of key tiles of both, of which the tensor core works 2050.  Calls one after
// another: two sequences of 8192, 32 heads, no window: 815 us, 1350 TFLOP/s (0.71 of the measured
// burst rate); a window of 1024 with 4 first positions over two documents of 8k, grouped heads: 254
// us, 939 TFLOP/s of visible pairs (captured in a graph 247 us, 966); ragged prompts of 300 .. 512:
// 62 us, where the first loads (10000 cycles to the first S), the masked tiles and the turns of
// short blocks count.  A masked tile's softmax takes 2700 cycles instead of 1250.  Steps that
// brought it there, on the 8k window: one thread per row instead of two that exchange maxima
// 345 -> 318 us, an issuer warp per Q tile and key steps from the producer 318 -> 307, MMAs issued
// under one lane's predicate on warp-uniform values 307 -> 254.  Not kept: one pass instead of two (a chunk's maximum checked before its
// exponentials: 254 -> 277 us, the exponentials stand still meanwhile); the next load in flight in
// masked tiles too (249 -> 259 us: registers), or masks in the code of the unmasked ones
// (249 -> 276 us); more registers for the softmax warps (setmaxnreg, 16 warps: 252 -> 262 us);
// prefetching the next Q and K/V tiles into L2 (prompts 62 -> 66 us).
//
// Every mbarrier wait is bounded; on timeout the CTA sets the device error word (read by
// fg_check_device_error), drains its copies and MMAs and frees TMEM.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "attn_tc.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_prefill_window_error = 0;

namespace {

constexpr int QB = 2 * QT;                  // query rows per block
constexpr int STAGES = 2;                   // K/V ring
constexpr int THREADS = 16 * 32;
constexpr int W_MMA = 1;                    // MMA issuers: warps 1 and 2, one per Q tile
constexpr int W_SM = 3;                     // softmax warps 3..10: Q tile (w - 3) / 4, TMEM lane
                                            // quarter w % 4
constexpr int W_OUT = 11;                   // first output warp (11..14)
constexpr int W_ITEM = 15;                  // work items
constexpr uint32_t TMEM_COLS = 512;
constexpr long long kWaitCycles = 1ll << 36;   // attend_rows may keep the other warps waiting (64
                                               // rows of 10^6 keys: 3 s)
constexpr long long kDrainCycles = 1ll << 32;  // for copies and products in flight
constexpr unsigned int kErrWait = 1u, kErrDrain = 2u;
constexpr int BOX = QT * 128;               // bytes of one 64-column x 128-row box
constexpr int kMaxSeqs = 384;               // sequences per launch
static_assert(kMaxSeqs <= THREADS, "one thread per sequence reads its offsets");

constexpr float kLag = 8.0f;                // base-2 score by which a row may pass its reference
constexpr float kPExp = 7.0f;               // P is scaled by 2^7, as its row sum is: with that lag
                                            // P <= 2^15, and down to 2^-21 of the reference's P a
                                            // weight is a normal fp16 number, to 2^-31 not zero
constexpr int ITEMS = 4;                    // ring of work items
constexpr unsigned kAllSteps = (KT / 16) << 4;   // every 16-key step of a tile (s0 | s1 << 4)
constexpr unsigned kLastTile = 8u;               // the Q tile's last key tile (s0 < 8)

struct Seq {
  int q0, nq, k0, nk;                       // first query row, rows, first K/V row, rows
};

template <int D>
struct PSmem {
  static constexpr int TILE = (D / 64) * BOX;          // one Q, K or V tile
  static constexpr int Q_OFF = 0;                      // Q_A, Q_B
  static constexpr int K_OFF = 2 * TILE;               // K stages
  static constexpr int V_OFF = K_OFF + STAGES * TILE;  // V stages
  static constexpr int O_OFF = V_OFF + STAGES * TILE;  // one output box
  static constexpr int L_OFF = O_OFF + BOX;            // row sums l [tile][row], maxima the same
  static constexpr int NQ_OFF = L_OFF + 4 * QT * 4;    // the sequences' query rows (start only)
  static constexpr int BAR_OFF = NQ_OFF + kMaxSeqs * 4;
  static constexpr int ITEM_OFF = BAR_OFF + 512;
  static constexpr int SEQ_OFF = ITEM_OFF + ITEMS * 64;  // sequences, longest first
  static constexpr int BYTES = SEQ_OFF + kMaxSeqs * (int)sizeof(Seq) + 1024;   // 1024: alignment
};
static_assert(PSmem<128>::BYTES <= 227 * 1024, "shared memory per CTA");

// barriers: q_full[2], q_free[2], k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2],
// o_done[2], o_free[2], l_full[2], drain[2], item_full[4], item_free[4]
constexpr int B_QFULL = 0, B_QFREE = 2, B_KFULL = 4, B_KFREE = 6, B_VFULL = 8, B_VFREE = 10,
              B_SFULL = 12, B_PFULL = 14, B_ODONE = 16, B_OFREE = 18, B_LFULL = 20, B_DRAIN = 22,
              B_IFULL = 24, B_IFREE = B_IFULL + ITEMS, NBARS = B_IFREE + ITEMS;
static_assert(NBARS * 8 + 12 + STAGES * 8 <= 512, "barrier space");

__device__ __forceinline__ bool bwait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      atomicOr(&g_prefill_window_error, kErrWait);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (clock64() - t0 > kDrainCycles) {
      atomicOr(&g_prefill_window_error, kErrDrain);
      return;
    }
  }
}

// An output is a mean of values within fp16's range: what rounding carries past its end is put
// back; infinities stay.
__device__ __forceinline__ float in_range(float y) {
  return fabsf(y) < 66000.0f ? fminf(fmaxf(y, -65504.0f), 65504.0f) : y;
}

// Rows on their own, by a whole warp: up to kRowsAtOnce of its 32 (the bits of `rows`), the first
// of which is row qrow at position pos of a sequence whose K/V rows start at k0; lane l returns
// channels 64 box + 2l and the next.  Scores are computed a key per lane, values a channel pair per
// lane; what a row does not see takes no part in it, and once all of the rows' channels are NaN
// nothing changes them.  (4 rows of 16384 keys: 3 ms.)
constexpr int kRowsAtOnce = 4;
template <int D>
__device__ __noinline__ void attend_rows(const PrefillWindow& a, int qrow, int hq, int k0, int pos,
                                         unsigned rows, int box, float2 (&out)[kRowsAtOnce]) {
  constexpr int R = kRowsAtOnce;
  const int lane = threadIdx.x & 31;
  const int64_t kcol = (int64_t)(hq / (a.Hq / a.Hkv)) * D;
  const float sl2 = a.scale * 1.4426950408889634f;
  const uint16_t* q[R];
  int i[R];                                 // the rows' positions, ascending (the last repeats)
  float m[R], l[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = __ffs(rows) - 1;
    if (rows & (rows - 1)) rows &= rows - 1;
    q[r] = a.q + (int64_t)(qrow + row) * a.q_stride + (int64_t)hq * D;
    i[r] = pos + row;
    m[r] = -INFINITY;
    l[r] = 0.0f;
    out[r] = make_float2(0.0f, 0.0f);
  }
  const int w0 = (a.window == 0 || i[0] < a.window) ? 0 : i[0] - a.window + 1;
  const int first = min(a.sinks, w0), n = first + (i[R - 1] + 1 - w0);   // keys that a row sees
  auto key = [&](int u) { return u < first ? u : u - first + w0; };
#pragma unroll 1
  for (int u0 = 0; u0 < n; u0 += 32) {
    const int cnt = min(32, n - u0), t = key(u0 + min(lane, cnt - 1));
    const uint16_t* k = a.k + (int64_t)(k0 + t) * a.kv_stride + kcol;
    float s[R] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 8) {
      const uint4 y = ldg_nc_v4(k + c);
      const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint4 x = ldg_nc_v4(q[r] + c);
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 xf = unpack_h2(xw[e]), yf = unpack_h2(yw[e]);
          s[r] = fmaf(xf.x, yf.x, fmaf(xf.y, yf.y, s[r]));
        }
      }
    }
    unsigned sees[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool vis = lane < cnt && visible(t, i[r], a.window, a.sinks);
      sees[r] = __ballot_sync(0xFFFFFFFFu, vis);
      const float x = vis ? s[r] * sl2 : -INFINITY;
      float mx = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
      mx = fmaxf(mx, m[r]);
      const float ref = (mx == -INFINITY) ? 0.0f : mx, corr = exp2f(m[r] - ref);
      s[r] = vis ? exp2f(x - ref) : 0.0f;
      l[r] = l[r] * corr + s[r];
      out[r].x *= corr;
      out[r].y *= corr;
      m[r] = mx;
    }
    constexpr int BATCH = 8;                // values in flight
#pragma unroll 1
    for (int j0 = 0; j0 < cnt; j0 += BATCH) {
      uint32_t v[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        v[j] = *reinterpret_cast<const uint32_t*>(
            a.v + (int64_t)(k0 + key(u0 + min(j0 + j, cnt - 1))) * a.kv_stride + kcol + 64 * box +
            2 * lane);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const float2 x = unpack_h2(v[j]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool vis = sees[r] >> (j0 + j) & 1u;
          const float pj = __shfl_sync(0xFFFFFFFFu, s[r], j0 + j);
          out[r].x = fmaf(pj, vis ? x.x : 0.0f, out[r].x);
          out[r].y = fmaf(pj, vis ? x.y : 0.0f, out[r].y);
        }
      }
    }
    bool settled = true;
#pragma unroll
    for (int r = 0; r < R; ++r)
      settled = settled && (i[r] < 0 || (isnan(out[r].x) && isnan(out[r].y)));
    if (__all_sync(0xFFFFFFFFu, settled)) break;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], d);
    out[r].x = i[r] < 0 ? 0.0f : in_range(out[r].x / l[r]);
    out[r].y = i[r] < 0 ? 0.0f : in_range(out[r].y / l[r]);
  }
}

// The rows of an item whose key tiles both Q tiles worked on, 32 by a warp: `rows` of them are the
// sequence's, lane r has row qrow + r in O of A and B (D columns each from o_addr on) and their
// sums and maxima in l.  (O_A 2^(m_A - m) + O_B 2^(m_B - m)) / l, l joined alike.  A called
// function: the output of unsplit items keeps its registers.
template <int D>
__device__ __noinline__ void store_split(const PrefillWindow& w, int qrow, int rows, int hq, int k0,
                                         int pos, uint32_t o_addr, const float* l,
                                         uint32_t o_free) {
  const int lane = threadIdx.x & 31;
  const float ma = l[2 * QT + lane], mb = l[3 * QT + lane], mx = fmaxf(ma, mb);
  const float wa = ex2(ma - mx), wb = ex2(mb - mx);
  const float sum = l[lane] * wa + l[QT + lane] * wb;
  const bool sees = pos + lane >= 0;
  const float fa = sees ? wa / sum : 0.0f, fb = sees ? wb / sum : 0.0f;
  uint16_t* out = w.out + (int64_t)(qrow + lane) * w.out_stride + (int64_t)hq * D;
  unsigned redo[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float a[32], b[32];
    tmem_ld32(o_addr + 32 * c, a);
    tmem_ld32(o_addr + D + 32 * c, b);
    tmem_wait_ld_dep(a);
    tmem_wait_ld_dep(b);
    __half2 zero = __float2half2_rn(0.0f);  // x * 0: NaN for an infinity or a NaN
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 8 * k + 2 * e;
        p[e] = pack_h2(fmaf(b[i], fb, a[i] * fa), fmaf(b[i + 1], fb, a[i + 1] * fa));
        zero = __hfma2(*reinterpret_cast<const __half2*>(&p[e]), __float2half2_rn(0.0f), zero);
      }
      if (lane < rows)
        reinterpret_cast<uint4*>(out + 32 * c)[k] = make_uint4(p[0], p[1], p[2], p[3]);
    }
    redo[c >> 1] |= __ballot_sync(0xFFFFFFFFu, lane < rows && !(sees && isnan(sum)) &&
                                                   (__hisnan(__low2half(zero)) ||
                                                    __hisnan(__high2half(zero))));
  }
  tc_fence_before();
  __syncwarp();
  if (lane < 2) mbar_arrive(o_free + 8 * lane);        // of A and of B
#pragma unroll 1
  for (int box = 0; box < D / 64; ++box) {
    for (unsigned left = box ? redo[1] : redo[0]; left;) {
      float2 x[kRowsAtOnce];
      attend_rows<D>(w, qrow, hq, k0, pos, left, box, x);
#pragma unroll
      for (int r = 0; r < kRowsAtOnce; ++r) {
        if (!left) break;
        *reinterpret_cast<uint32_t*>(w.out + (int64_t)(qrow + __ffs(left) - 1) * w.out_stride +
                                     (int64_t)hq * D + 64 * box + 2 * lane) =
            pack_h2(x[r].x, x[r].y);
        left &= left - 1;
      }
    }
  }
  __syncwarp();
}

struct PArgs {
  PrefillWindow w;
  int s0, ns;                               // sequences s0 .. s0 + ns - 1 of the call
  float scale_log2;
};

// Rows `tail` .. of a V tile in their 16-key step become 0, written by a whole warp (a called
// function: in line it takes registers that the other warps' loops need, 1.5% of an 8k window's
// time).  Both MMA issuers may write (the same zeros); each does before its own products read them
// and before its part of V's release.
__device__ __noinline__ void clear_rows(uint8_t* v, int tail, int boxes) {
  const int chunks = 8 * (((tail + 15) & ~15) - tail);
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < boxes * chunks; i += 32)
    *reinterpret_cast<uint4*>(v + 128 * tail + (i < chunks ? 16 * i : BOX + 16 * (i - chunks))) =
        make_uint4(0, 0, 0, 0);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// A work item: a block of 256 query rows of one (sequence, query head).
struct Item {
  int hq;                                   // query head; -1: no more items
  int qrow, rows;                           // the block's first row in q and out; how many
  int krow;                                 // the sequence's first K/V row
  int pos;                                  // position of the block's first row (may be negative)
  KeyTiles t[2], u;                         // the Q tiles' key tiles, and their union
  int split;                                // the Q tiles hold the same rows, and tile t works on
                                            // the key tiles number t, t + 2, .. of them
};
static_assert(sizeof(Item) <= 64, "item ring");
// The place of an item in the work order.
struct Cursor {
  int level, cnt, i;                        // block index; sequences that have it; item within it
};
__device__ __forceinline__ int blocks_of(int nq) { return (nq + QB - 1) / QB; }
// How many of the sequences (longest first) have a block `level`.
__device__ __forceinline__ int level_count(const Seq* seqs, int n, int level) {
  int lo = 0, hi = n;                       // seqs[lo - 1] has it, seqs[hi] does not
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (blocks_of(seqs[mid].nq) > level) lo = mid + 1; else hi = mid;
  }
  return lo;
}
// Moves n items on; false past the last.
__device__ __forceinline__ bool advance(Cursor& c, int n, const Seq* seqs, int nseq, int Hq) {
  int64_t i = (int64_t)c.i + n;
  while (c.level >= 0 && i >= (int64_t)c.cnt * Hq) {
    i -= (int64_t)c.cnt * Hq;
    if (--c.level >= 0) c.cnt = level_count(seqs, nseq, c.level);
  }
  c.i = (int)i;
  return c.level >= 0;
}
__device__ __forceinline__ Cursor first_item(const Seq* seqs, int nseq) {
  Cursor c;
  c.level = nseq > 0 ? blocks_of(seqs[0].nq) - 1 : -1;
  c.cnt = c.level >= 0 ? level_count(seqs, nseq, c.level) : 0;
  c.i = 0;
  return c;
}
__device__ __forceinline__ Item item_at(const Cursor& c, const Seq* seqs, const PrefillWindow& w) {
  Item it;
  const int b = c.i / w.Hq, q0 = c.level * QB;
  const Seq s = seqs[b];
  it.hq = c.i - b * w.Hq;
  it.qrow = s.q0 + q0;
  it.rows = s.nq - q0;
  it.krow = s.k0;
  it.pos = s.nk - s.nq + q0;
  it.t[0] = key_tiles(q0, s.nq, s.nk, w.window, w.sinks);
  it.t[1] = key_tiles(q0 + QT, s.nq, s.nk, w.window, w.sinks);
  it.u = either(it.t[0], it.t[1]);
  it.split = s.nq <= QT && it.u.count() >= 2;   // (what it gains: at the top)
  if (it.split) it.t[1] = it.t[0];
  return it;
}

// Persistent: CTA c takes items c, c + gridDim, ...  The producer loads the next item's Q as
// soon as the current item's last S product is done and streams K/V through the rings across
// items; each Q tile's MMA issuer starts the next item's S products while the current item's last
// P V products run, and the output warps store an item's O while the softmax warps work on the
// next.
template <int D>
__global__ void __launch_bounds__(THREADS, 1)
prefill_window_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmO, const __grid_constant__ PArgs pa) {
  using L = PSmem<D>;
  constexpr int NB = D / 64;                           // 64-column boxes per tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* live = reinterpret_cast<int*>(tmem_slot + 2);   // sequences with rows
  unsigned* steps_of = tmem_slot + 3;                  // [STAGES]: key steps of the K tile
  unsigned* tail_of = steps_of + STAGES;               // [STAGES]: where rows of a V tile that are
                                                       // not the sequence's begin in a step, or 0
  Seq* seqs = reinterpret_cast<Seq*>(smem + L::SEQ_OFF);
  auto item_slot = [&](int n) {
    return reinterpret_cast<Item*>(smem + L::ITEM_OFF + 64 * (n % ITEMS));
  };
  float* l_buf = reinterpret_cast<float*>(smem + L::L_OFF);
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8u * i; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PrefillWindow& w = pa.w;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(bar(B_KFULL + i), 1);
      mbar_init(bar(B_VFULL + i), 1);
      mbar_init(bar(B_KFREE + i), 2);                  // one arrival per MMA issuer
      mbar_init(bar(B_VFREE + i), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(B_QFULL + t), 1);
      mbar_init(bar(B_QFREE + t), 1);
      mbar_init(bar(B_SFULL + t), 1);
      mbar_init(bar(B_PFULL + t), 4);                  // one arrival per softmax warp
      mbar_init(bar(B_ODONE + t), 1);
      mbar_init(bar(B_OFREE + t), 4);                  // one arrival per output warp
      mbar_init(bar(B_LFULL + t), 4);                  // one arrival per softmax warp
    }
    mbar_init(bar(B_DRAIN), 1);
    mbar_init(bar(B_DRAIN + 1), 1);
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(bar(B_IFULL + i), 1);
      mbar_init(bar(B_IFREE + i), 1 + 2 + 8 + 4);     // every other warp
    }
    *abort_flag = 0;
    *live = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---- the sequences, longest first (by query rows, then by index).  The ones whose offsets do
  // not fit their buffers count as empty.
  Seq me{0, 0, 0, 0};
  int* nq_all = reinterpret_cast<int*>(smem + L::NQ_OFF);
  if (threadIdx.x < kMaxSeqs) {
    if ((int)threadIdx.x < pa.ns) {
      const int b = pa.s0 + threadIdx.x;
      const int q0 = w.q_off[b], q1 = w.q_off[b + 1], k0 = w.kv_off[b], k1 = w.kv_off[b + 1];
      if (q0 >= 0 && q0 <= q1 && q1 <= w.q_rows && k0 >= 0 && k0 <= k1 && k1 <= w.kv_rows)
        me = Seq{q0, q1 - q0, k0, k1 - k0};
      else if (blockIdx.x == 0)
        atomicOr(&g_prefill_window_error, kErrExtent);
    }
    nq_all[threadIdx.x] = me.nq;
  }
  __syncthreads();
  if (me.nq > 0) {
    int rank = 0;
    for (int b = 0; b < pa.ns; ++b)
      rank += nq_all[b] > me.nq || (nq_all[b] == me.nq && b < (int)threadIdx.x);
    seqs[rank] = me;
    atomicAdd(live, 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nseq = *live;
  // TMEM columns: S_A 0..127, S_B 128..255, O_A 256.., O_B 256 + D..
  auto s_col = [&](int t) { return (uint32_t)(t * KT); };
  auto o_col = [&](int t) { return (uint32_t)(2 * KT + t * D); };
  // Item n of this CTA for a consuming thread (null: a wait ran out), and the end of its use.
  auto item_wait = [&](int n) -> const Item* {
    return bwait(bar(B_IFULL + n % ITEMS), (uint32_t)((n / ITEMS) & 1), abort_flag) ? item_slot(n)
                                                                                    : nullptr;
  };
  auto item_done = [&](int n) { mbar_arrive(bar(B_IFREE + n % ITEMS)); };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int kvg = 0, qn = 0, kn = 0, vn = 0;             // key tiles, Q pairs, K and V tiles issued
      int qt[2] = {0, 0};                              // Q tiles A and B issued
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item* slot = item_wait(n);
        if (slot == nullptr || slot->hq < 0) break;
        const Item it = *slot;
        item_done(n);
        const int nkv = it.u.count();
        if (nkv == 0) continue;
        const int hk = it.hq / (w.Hq / w.Hkv);
        for (int j = 0; j < nkv; ++j, ++kvg) {
          // K and V have rings of their own: a K stage is free once both Q tiles' S products
          // have read it, a whole softmax before the V stage of the same tile
          const int st = kvg % STAGES, row = it.krow + it.u.tile(j) * KT;
          auto load = [&](const CUtensorMap* tm, int off, int full, int free, unsigned note) {
            if (kvg >= STAGES &&
                !bwait(bar(free + st), (uint32_t)(((kvg / STAGES) & 1) ^ 1), abort_flag))
              return false;
            (full == B_KFULL ? steps_of : tail_of)[st] = note;   // handed on by the barrier
            mbar_expect_tx(bar(full + st), (uint32_t)L::TILE);
            for (int c = 0; c < NB; ++c)
              tma_load_2d(smem_u32(smem + off + st * L::TILE + c * BOX), tm, hk * D + 64 * c, row,
                          bar(full + st));
            return true;
          };
          // the 16-key steps that the Q tiles take of the tile, a byte each: s0 | s1 << 4 (s1 0:
          // none), and kLastTile when they take none of a later one
          auto steps = [&](int t) -> unsigned {
            if (it.split) {
              const bool now = (j & 1) == t;
              const unsigned last = j + 1 + now < nkv ? 0u : kLastTile;
              if (!now) return last;
              const KeySteps k = key_steps(it.u.tile(j), it.pos, it.pos + it.rows - 1, w.window,
                                           w.sinks);
              return (unsigned)(k.s0 | k.s1 << 4) | last;
            }
            const int tile = it.u.tile(j), lo = it.pos + t * QT;
            const unsigned last = (it.t[t].count() == 0 || tile >= it.t[t].te - 1) ? kLastTile : 0u;
            if (!it.t[t].has(tile)) return last;
            const KeySteps k = key_steps(tile, lo, it.pos + min(t * QT + QT, it.rows) - 1, w.window,
                                         w.sinks);
            return (unsigned)(k.s0 | k.s1 << 4) | last;
          };
          if (!load(&tmK, L::K_OFF, B_KFULL, B_KFREE, steps(0) | steps(1) << 8)) {
            ok = false;
            break;
          }
          kn = kvg + 1;
          if (j == 0) {
            // each Q tile, when its last S product of the previous item is done with it
            for (int t = 0; t < 2 && ok; ++t) {
              if (qn > 0 && !bwait(bar(B_QFREE + t), (uint32_t)((qn - 1) & 1), abort_flag)) {
                ok = false;
                break;
              }
              mbar_expect_tx(bar(B_QFULL + t), (uint32_t)L::TILE);
              for (int c = 0; c < NB; ++c)
                tma_load_2d(smem_u32(smem + L::Q_OFF + t * L::TILE + c * BOX), &tmQ,
                            it.hq * D + 64 * c, it.qrow + (it.split ? 0 : t * QT),
                            bar(B_QFULL + t));
              qt[t] = qn + 1;
            }
            if (!ok) break;
            ++qn;
          }
          // the sequence may end inside a 16-key step
          const int valid = min(KT, it.pos + it.rows - it.u.tile(j) * KT);
          if (!load(&tmV, L::V_OFF, B_VFULL, B_VFREE, valid % 16 ? valid : 0)) {
            ok = false;
            break;
          }
          vn = kvg + 1;
        }
      }
      // every issued copy has landed before the CTA exits
      for (int t = 0; t < 2; ++t)
        if (qt[t] > 0) drain_wait(bar(B_QFULL + t), (uint32_t)((qt[t] - 1) & 1));
      for (int i = max(0, kn - STAGES); i < kn; ++i)
        drain_wait(bar(B_KFULL + i % STAGES), (uint32_t)((i / STAGES) & 1));
      for (int i = max(0, vn - STAGES); i < vn; ++i)
        drain_wait(bar(B_VFULL + i % STAGES), (uint32_t)((i / STAGES) & 1));
    }
  } else if (warp < W_SM) {
    // ------------------------------------------------------------ MMA issuer of Q tile t.  Each
    // Q tile has a warp of its own: the order that matters is within a Q tile (S_t(j + 1)
    // overwrites the columns of P_t(j) only after P_t(j) V_j has read them), and the rings count an
    // arrival of each.  What is between a P and the next S is on the critical path (softmax and
    // products of one Q tile take turns), so everything else is done before P is waited for or
    // after S is issued, and which key steps the Q tiles take of a key tile comes from the producer
    // with the tile.  The whole warp runs the loop on values that are the same in every lane, and
    // one lane's predicate issues: descriptors stay in uniform registers.
    const int t = __shfl_sync(0xFFFFFFFFu, warp - W_MMA, 0);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), sbase = smem_u32(smem);
    const uint32_t one = elect_one();
    const uint32_t od = tm + o_col(t), scol = tm + s_col(t);
    const uint64_t qd = smem_desc(sbase + L::Q_OFF + t * L::TILE, 16, 1024);
    const uint32_t idesc_o = idesc_pv(D);
    int kvg = 0, qn = 0;                               // K/V tiles, items consumed
    int pc = 0, uses = 0;                              // P V products; items of this Q tile
    bool ok = true;
    auto wait = [&](int b, int parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, bwait(bar(b), (uint32_t)parity, abort_flag));
    };
    auto commit = [&](int b) { umma_commit_if(bar(b), one); };
    // S_t = Q_t K^T of the key steps `ks` of K/V tile g over K = D: k-step i reads 16 columns,
    // 32 bytes into box i / 4; 16 keys are 2048 bytes of each box
    auto issue_s = [&](int g, unsigned ks) {
      const int s0 = ks & 7, s1 = ks >> 4;
      const uint64_t kd = smem_desc(sbase + L::K_OFF + (g % STAGES) * L::TILE, 16, 1024) +
                          (uint64_t)(s0 * 128);
      const uint32_t idesc = idesc_qk(16 * (s1 - s0)), col = scol + 16 * s0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint64_t off = (uint64_t)(((i >> 2) * BOX + (i & 3) * 32) >> 4);
        umma_f16_if(col, qd + off, kd + off, idesc, i > 0, one);
      }
      commit(B_SFULL + t);
    };
    // O_t (+)= P_t V of the same key steps: step i reads the 8 TMEM columns of P of keys 16i..
    // (32 keys keep their P in the first 16 of their S columns) and rows 16i.. of V (2048 bytes
    // per step in its MN-major 128B-swizzled layout)
    auto issue_pv = [&](int g, unsigned ks, uint32_t add) {
      const uint64_t vd = smem_desc(sbase + L::V_OFF + (g % STAGES) * L::TILE, BOX, 1024);
      if ((ks & ~kLastTile) == kAllSteps) {
        umma_ts_if(od, scol, vd, idesc_o, add, one);
#pragma unroll
        for (int i = 1; i < KT / 16; ++i)
          umma_ts_if(od, scol + 32 * (i >> 1) + 8 * (i & 1), vd + (uint64_t)(i * 128), idesc_o, 1u,
                     one);
      } else {
        for (int i = ks & 7; i < (int)(ks >> 4); ++i, add = 1u)
          umma_ts_if(od, scol + 32 * (i >> 1) + 8 * (i & 1), vd + (uint64_t)(i * 128), idesc_o, add,
                     one);
      }
    };
    // waits for K of tile g; the steps of it that this Q tile takes
    auto wait_k = [&](int g) -> unsigned {
      wait(B_KFULL + g % STAGES, (g / STAGES) & 1);
      const unsigned all = __shfl_sync(0xFFFFFFFFu, steps_of[g % STAGES], 0);
      return all >> (8 * t) & 0xFFu;
    };
    for (int n = 0; ok; ++n) {
      const Item* slot = item_wait(n);
      if (!__all_sync(0xFFFFFFFFu, slot != nullptr)) break;
      const int hq = __shfl_sync(0xFFFFFFFFu, slot->hq, 0);
      if (hq < 0) break;
      const int nkv = __shfl_sync(0xFFFFFFFFu, slot->u.count(), 0);
      if (lane == 0) item_done(n);
      if (nkv == 0) continue;
      wait(B_QFULL + t, qn & 1);
      unsigned cur = wait_k(kvg);
      if (!ok) break;
      tc_fence_after();
      ++qn;
      uint32_t add = 0;                                // there is a P V product of this item
      bool q_free = false;                             // every S product of the item issued
      auto after_s = [&](int g, unsigned ks) {
        commit(B_KFREE + g % STAGES);                  // K of the tile read by the product before
        if ((ks & kLastTile) && !q_free) {
          commit(B_QFREE + t);
          q_free = true;
        }
      };
      if (cur & ~kLastTile) issue_s(kvg, cur);
      after_s(kvg, cur);
      for (int j = 0; j < nkv; ++j) {
        const int g = kvg + j;
        const bool more = j + 1 < nkv;
        // both tiles first: P is the last to come.  (V is waited for in any case: an issuer
        // that ran ahead of the other would arrive twice in one phase of its free barrier.)
        wait(B_VFULL + g % STAGES, (g / STAGES) & 1);
        const unsigned next = more ? wait_k(g + 1) : 0u;
        const bool pv = cur & ~kLastTile;
        if (pv) {
          const unsigned tail = __shfl_sync(0xFFFFFFFFu, tail_of[g % STAGES], 0);
          if (tail && ok) clear_rows(smem + L::V_OFF + (g % STAGES) * L::TILE, tail, NB);
          // the first product of an item overwrites O_t: the output warps have read it
          if (!add && uses > 0) wait(B_OFREE + t, (uses - 1) & 1);
          wait(B_PFULL + t, pc & 1);
        }
        if (!ok) break;
        tc_fence_after();
        if (pv) {
          issue_pv(g, cur, add);
          if (!add) ++uses;
          add = 1;
          ++pc;
        }
        // S_t of the next key tile: its columns hold no P that is still to be read (this Q
        // tile's earlier products were issued before)
        if (next & ~kLastTile) issue_s(g + 1, next);
        commit(B_VFREE + g % STAGES);                  // V of tile g read by the product above
        if (more) after_s(g + 1, next);
        cur = next;
      }
      if (!ok) break;
      if (add) commit(B_ODONE + t);                    // the item's P V products
      kvg += nkv;
    }
    // the CTA frees TMEM only after every MMA issued here has completed
    commit(B_DRAIN + t);
    if (one) drain_wait(bar(B_DRAIN + t), 0u);
    __syncwarp();
  } else if (warp >= W_SM && warp < W_OUT) {
    // ------------------------------------------------------------ softmax of one Q tile's rows
    const int t = (warp - W_SM) >> 2;
    const int quarter = warp & 3;                      // TMEM lanes 32 quarter ..
    const int m = 32 * quarter + lane;                 // row within the Q tile
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t srow = lane_addr + s_col(t);
    const float sl2 = pa.scale_log2;
    int sc = 0, uses = 0;                              // S products consumed, items finished
    bool ok = true;
    // tcgen05.ld / st are warp-collective (.sync.aligned): every branch around them is
    // decided for the whole warp, waits included (a lane that gave up takes its warp along)
    for (int n = 0; ok; ++n) {
      const volatile Item* it = item_wait(n);          // read where needed: no registers for it
      if (!__all_sync(0xFFFFFFFFu, it != nullptr) || it->hq < 0) break;
      const int nt = it->t[t].ns + it->t[t].te - it->t[t].tw;
      const int step = 1 + it->split, row0 = step == 1 ? t * QT : 0;
      if (nt == 0) {
        if (lane == 0) item_done(n);
        continue;
      }
      // (rows behind the sequence: no score of theirs moves the reference of the warp's rows)
      float m_ref = row0 + m < it->rows ? -INFINITY : INFINITY, l_sum = 0.0f;
      for (int j = step == 1 ? 0 : t; j < nt; j += step, ++sc) {
        // masked: some row of the Q tile does not see every key of the tile (warp-uniform); ahead:
        // the position of the Q tile's first row less the key tile's first position
        const int ns = it->t[t].ns;
        const int k0 = (j < ns ? j : j - ns + it->t[t].tw) * KT, ahead = it->pos + row0 - k0;
        const bool masked = ahead < KT - 1 ||
                            (w.window != 0 && k0 + KT > w.sinks &&
                             ahead + min(QT, it->rows - row0) > w.window);
        const bool got = bwait(bar(B_SFULL + t), (uint32_t)(sc & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // pass 1: the row's maximum, 32 columns at a time (the next load in flight)
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto max_chunk = [&](const float (&v)[32]) {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], v[e], v[e + 1]);
        };
        float va[32], vb[32];
        unsigned none = 0;                             // chunks that no row of the warp sees
        if (masked) {
          // keys that a row does not see are set to -inf, in TMEM too: pass 2 reads them there
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint32_t vis = visible_bits(k0 + 32 * c, k0 + ahead + m, w.window, w.sinks);
            if (!__any_sync(0xFFFFFFFFu, vis != 0u)) {
              none |= 1u << c;
              continue;
            }
            tmem_ld32(srow + 32 * c, va);
            tmem_wait_ld_dep(va);
            if (!__all_sync(0xFFFFFFFFu, vis == ~0u)) {
#pragma unroll
              for (int e = 0; e < 32; ++e) va[e] = (vis >> e & 1u) ? va[e] : -INFINITY;
              tmem_st16(srow + 32 * c, reinterpret_cast<const uint32_t*>(va));
              tmem_st16(srow + 32 * c + 16, reinterpret_cast<const uint32_t*>(va) + 16);
            }
            max_chunk(va);
          }
          tmem_wait_st();
        } else {
          tmem_ld32(srow, va);
          tmem_wait_ld_dep(va);
          tmem_ld32(srow + 32, vb);
          max_chunk(va);
          tmem_wait_ld_dep(vb);
          tmem_ld32(srow + 64, va);
          max_chunk(vb);
          tmem_wait_ld_dep(va);
          tmem_ld32(srow + 96, vb);
          max_chunk(va);
          tmem_wait_ld_dep(vb);
          max_chunk(vb);
        }
        // in base 2 (scale > 0, so scaling after the maximum is the same); -inf for a row that
        // has seen no key yet
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
        if (__any_sync(0xFFFFFFFFu, mx > m_ref + kLag)) {
          // move the reference maximum of every row of the warp to max(m_ref, mx): O and l
          // scale by 2^(m_ref - m_new) (1 for rows whose maximum did not grow).  O holds P V of the
          // item's earlier tiles: those MMAs were issued, and so are done, before this S
          const float m_new = fmaxf(m_ref, mx);
          const float alpha = (m_ref == -INFINITY) ? 0.0f : ex2(m_ref - m_new);
          if (j >= step) {
#pragma unroll 1
            for (int c16 = 0; c16 < D / 16; ++c16) {
              uint32_t wv[16];
              const uint32_t oa = lane_addr + o_col(t) + (uint32_t)(16 * c16);
              tmem_ld16(oa, wv);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                wv[e] = __float_as_uint(__uint_as_float(wv[e]) * alpha);
              tmem_st16(oa, wv);
            }
            tmem_wait_st();
          }
          l_sum *= alpha;
          m_ref = m_new;
        }
        // pass 2: p = 2^(s * scale - m_ref + 7), 32 columns at a time (the scaling and the row sums
        // two elements per instruction), packed to fp16 over the first 16 of the 32 S columns
        const float ref = (m_ref == -INFINITY) ? 0.0f : m_ref;
        const uint64_t sl2x2 = f2pack(sl2, sl2), negm2 = f2pack(kPExp - ref, kPExp - ref);
        uint64_t ls2[2] = {f2pack(0.0f, 0.0f), f2pack(0.0f, 0.0f)};
        auto p_chunk = [&](const float (&v)[32], int c) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = f2unpack(ffma2(f2pack(v[e], v[e + 1]), sl2x2, negm2));
            const float p0 = ex2(x.x), p1 = ex2(x.y);
            ls2[(e >> 1) & 1] = fadd2(ls2[(e >> 1) & 1], f2pack(p0, p1));
            pw[e / 2] = pack_h2(p0, p1);
          }
          tmem_st16(srow + 32 * c, pw);
        };
        if (!masked) {
          // the last chunk is still in registers
          tmem_ld32(srow, va);
          p_chunk(vb, 3);
          tmem_wait_ld_dep(va);
          tmem_ld32(srow + 32, vb);
          p_chunk(va, 0);
          tmem_wait_ld_dep(vb);
          tmem_ld32(srow + 64, va);
          p_chunk(vb, 1);
          tmem_wait_ld_dep(va);
          p_chunk(va, 2);
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (none >> c & 1u) {
              const uint32_t zeros[16] = {};
              tmem_st16(srow + 32 * c, zeros);
            } else {
              tmem_ld32(srow + 32 * c, va);
              tmem_wait_ld_dep(va);
              p_chunk(va, c);
            }
          }
        }
        tmem_wait_st();
        const float2 la = f2unpack(fadd2(ls2[0], ls2[1]));
        l_sum += la.x + la.y;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + t));
      }
      if (!ok) break;
      // the row sums for the output warps, once they have taken the previous item's
      if (uses > 0) {
        const bool fr = bwait(bar(B_OFREE + t), (uint32_t)((uses - 1) & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, fr)) {
          ok = false;
          break;
        }
      }
      l_buf[t * QT + m] = l_sum;
      if (it->split) l_buf[(2 + t) * QT + m] = m_ref;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(B_LFULL + t));
        item_done(n);
      }
      ++uses;
    }
  } else if (warp == W_ITEM) {
    // ------------------------------------------------------------ work items
    if (lane == 0) {
      Cursor cur = first_item(seqs, nseq);
      bool have = advance(cur, blockIdx.x, seqs, nseq, w.Hq);
      for (int n = 0;; ++n) {
        if (n >= ITEMS &&
            !bwait(bar(B_IFREE + n % ITEMS), (uint32_t)((n / ITEMS - 1) & 1), abort_flag))
          break;
        Item it;
        it.hq = -1;
        if (have) it = item_at(cur, seqs, w);
        *item_slot(n) = it;
        mbar_arrive(bar(B_IFULL + n % ITEMS));
        if (!have) break;
        have = advance(cur, gridDim.x, seqs, nseq, w.Hq);
      }
    }
  } else if (warp >= W_OUT) {
    // ------------------------------------------------------------ output of both Q tiles
    const int quarter = warp & 3;
    const int m = 32 * quarter + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16);
    int uses[2] = {0, 0};                              // items per Q tile
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const Item* it = item_wait(n);
      if (!__all_sync(0xFFFFFFFFu, it != nullptr) || it->hq < 0) break;
      for (int t = 0; t < 2 && ok; ++t) {
        const int rows = min(QT, it->rows - t * QT);   // valid rows
        if (rows <= 0) continue;
        const int nt = it->t[t].count(), qrow = it->qrow + t * QT, pos = it->pos + t * QT;
        uint16_t* out = w.out + (int64_t)(qrow + m) * w.out_stride + (int64_t)it->hq * D;
        if (nt == 0) {                                 // no row of the tile sees a key
          if (m < rows)
            for (int c = 0; c < D / 8; ++c)
              reinterpret_cast<uint4*>(out)[c] = make_uint4(0, 0, 0, 0);
          continue;
        }
        // the row sums, then the item's P V products into O_t
        bool got = bwait(bar(B_LFULL + t), (uint32_t)(uses[t] & 1), abort_flag);
        got = got && bwait(bar(B_ODONE + t), (uint32_t)(uses[t] & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        if (it->split) {
          got = bwait(bar(B_LFULL + 1), (uint32_t)(uses[1] & 1), abort_flag);
          got = got && bwait(bar(B_ODONE + 1), (uint32_t)(uses[1] & 1), abort_flag);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          ++uses[0];
          ++uses[1];
          store_split<D>(w, qrow + 32 * quarter, rows - 32 * quarter, it->hq, it->krow,
                         pos + 32 * quarter, lane_addr + o_col(0), l_buf + 32 * quarter,
                         bar(B_OFREE));
          break;
        }
        tc_fence_after();
        ++uses[t];
        // (a row that sees nothing: O 0, or NaN, which is mended below)
        const float inv = pos + m >= 0
                              ? 1.0f / l_buf[t * QT + m]
                              : 0.0f;
        // O / l in boxes of 64 columns x the warp's 32 rows, staged in shared memory (the
        // 128B-swizzled layout of the output map: 16-byte chunk k of row m at chunk k ^ (m % 8))
        // and stored by TMA, each warp by itself (one box of the tile's 128 rows, with the four
        // warps waiting for one another: ragged prompts 62 -> 65 us).  Where a sequence ends, each
        // thread stores its own row.
        const bool full = rows >= 32 * quarter + 32;   // the warp's rows
#pragma unroll 1
        for (int hb = 0; hb < NB; ++hb) {
          const uint32_t stage = smem_u32(smem + L::O_OFF);
          if (lane == 0) bulk_wait_read();              // the previous store has read the box
          __syncwarp();
          __half2 zero = __float2half2_rn(0.0f);       // x * 0: NaN for an infinity or a NaN
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float o[32];
            tmem_ld32(lane_addr + o_col(t) + 64 * hb + 32 * c, o);
            tmem_wait_ld_dep(o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 4 * c + i;
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                p[e] = pack_h2(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv);
                zero = __hfma2(*reinterpret_cast<const __half2*>(&p[e]), __float2half2_rn(0.0f),
                               zero);
              }
              if (full)
                st_shared_v4(stage + 128 * m + ((k ^ (m & 7)) << 4), p[0], p[1], p[2], p[3]);
              else if (m < rows)
                reinterpret_cast<uint4*>(out + 64 * hb)[k] = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
          const unsigned redo =
              __ballot_sync(0xFFFFFFFFu, m < rows && !isnan(inv) && (__hisnan(__low2half(zero)) ||
                                                                     __hisnan(__high2half(zero))));
          if (hb == NB - 1) {
            // O_t has been read: the next item's first P V product may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_OFREE + t));
          }
          if (redo) {
            __syncwarp();                              // over what the row's own thread stored
            for (unsigned left = redo; left;) {
              float2 x[kRowsAtOnce];
              attend_rows<D>(w, qrow + 32 * quarter, it->hq, it->krow, pos + 32 * quarter, left, hb,
                             x);
#pragma unroll
              for (int r = 0; r < kRowsAtOnce; ++r) {
                if (!left) break;
                const int rr = 32 * quarter + __ffs(left) - 1, ch = 2 * lane;
                left &= left - 1;
                uint8_t* dst =
                    full ? smem + L::O_OFF + 128 * rr + (((ch >> 3) ^ (rr & 7)) << 4) + (ch & 7) * 2
                         : reinterpret_cast<uint8_t*>(w.out + (int64_t)(qrow + rr) * w.out_stride +
                                                      (int64_t)it->hq * D + 64 * hb + ch);
                *reinterpret_cast<uint32_t*>(dst) = pack_h2(x[r].x, x[r].y);
              }
            }
          }
          if (full) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmO, stage + 4096 * quarter, it->hq * D + 64 * hb, qrow + 32 * quarter);
              bulk_commit();
            }
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (lane == 0) item_done(n);
    }
    // the CTA's shared memory stays valid until its stores have completed
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
}

// Shared memory of the kernel on the current device, set once per device.
template <int D>
cudaError_t prepare() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (dev < 0 || dev >= 64 || done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(prefill_window_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           PSmem<D>::BYTES);
  done[dev] = e == cudaSuccess;
  return e;
}

template <int D>
cudaError_t launch_d(const PrefillWindow& a, int nsm, cudaStream_t st) {
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess || (e = get_encode()) != cudaSuccess) return e;
  CUtensorMap tq, tk, tv, to;
  auto map = [](CUtensorMap* m, const uint16_t* p, int64_t cols, int64_t rows, int64_t stride,
                int box = QT) {
    return make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, (uint64_t)cols, (uint64_t)rows,
                       (uint64_t)stride * 2, 64, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const int64_t wq = (int64_t)a.Hq * D, wk = (int64_t)a.Hkv * D;
  if ((e = map(&tq, a.q, wq, a.q_rows, a.q_stride)) != cudaSuccess ||
      (e = map(&to, a.out, wq, a.q_rows, a.out_stride, 32)) != cudaSuccess)
    return e;
  tk = tv = tq;                             // without K/V rows no key tile is loaded
  if (a.kv_rows > 0 && ((e = map(&tk, a.k, wk, a.kv_rows, a.kv_stride)) != cudaSuccess ||
                        (e = map(&tv, a.v, wk, a.kv_rows, a.kv_stride)) != cudaSuccess))
    return e;
  for (int s0 = 0; s0 < a.nseq; s0 += kMaxSeqs) {
    const int ns = std::min(kMaxSeqs, a.nseq - s0);
    const PArgs pa{a, s0, ns, a.scale * 1.4426950408889634f};
    // the blocks of ns sequences of q_rows rows in all are at most this many
    const int64_t items = ((int64_t)a.q_rows / QB + ns) * a.Hq;
    const int64_t grid = std::min<int64_t>(items, std::max(1, nsm));   // one CTA per SM
    e = launch_pdl(prefill_window_kernel<D>, dim3((unsigned)grid), dim3(THREADS), PSmem<D>::BYTES,
                   st, tq, tk, tv, to, pa);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_prefill_attn_window(const PrefillWindow& a, int d, int nsm, cudaStream_t st) {
  return d == 128 ? launch_d<128>(a, nsm, st) : launch_d<64>(a, nsm, st);
}

cudaError_t prefill_window_read_error(unsigned int* out) {
  return read_and_clear(g_prefill_window_error, out);
}

}  // namespace fg
