// Attention of the newest tokens of every sequence over the paged 4-bit cache, on the
// 5th-generation tensor cores (sm_103a).
//
// Query row r of sequence b (nq rows, n cached positions) is position i = n - nq + r, and
//   out_r,hq = sum_t softmax_t(scale * q_r,hq . k^_t) v^_t   over the t that i sees,
// K/V head hq / G of G = Hq / H query heads each.  The rows of a product are a K/V head's tokens' G
// heads, so that a key tile is restored once for all of them (paged_work.cuh: row tiles, blocks,
// the order of the work, its even split into shares and the pieces of a block that a share cuts).
//
// A CTA owns a share.  For a block of two row tiles, chain A and chain B take one each and share
// the key tiles; for a block of one, they hold the same rows and take the key tiles in turn, joined
// at the end.  Per key tile of 128 positions:
//   codes         one bulk copy per page and half (K or V: codes and statistics lie side by side)
//                 into a ring of parts
//   restore       eight warps write the part as fp16 into the tensor core's 128B-swizzled tiles,
//                 fp16(a + q (b - a) / 15) exactly as defined.  Rows behind the sequence become 0.
//   S = Q K^T     tcgen05.mma kind::f16, fp32 in TMEM
//   softmax       one thread per row, two passes over its 128 columns (the maximum, then P): base-2
//                 online softmax with a lazily moved reference maximum (by more than 2^8), P =
//                 2^(s - m + 7) rounded to fp16 over S's columns
//   O += P V      tcgen05.mma with P from TMEM
//   warp 0        page table lookups and bulk copies
//   warps 1, 2    MMA issuers of chains A and B
//   warp 3        the share's segments, handed to the others through a ring; Q by TMA
//   warps 4-11    softmax of A and B (TMEM lanes 32 (w % 4) ..), and their output
//   warps 12-19   restore
// A second kernel puts cut blocks together, piece after piece in order.
//
// What bounds it: per key tile of a block of two row tiles, a chain's turn of softmax (3430 cycles) and
// the wait for its next S (1930: the two products, one behind the other, as P stands where S stood);
// for a block of one, restoring (2 x 1370 cycles a key tile).  Two documents' pieces of 1501 .. 2048
// tokens behind 12,001 .. 16,384 positions, 32 heads over 8, window 8192: 647 us, 0.74 PFLOP/s.
// (S in two halves of 64 keys, so that one is computed while the other is read, costs more turns
// than it hides: 795 us, and 382 us instead of 259 us where blocks have one row tile.  Restoring in
// code unrolled for K, V and tails: 755 us.  Moving registers between the warps' roles: no gain.)
//
// The products' additions truncate: 65,536 positions in one share, of values of one sign, lose 2e-4.
// Masked positions have P = 0, but 0 times an infinity or NaN in V is NaN: rows that end with one
// are computed again over what they see alone (attend_row).  Rows whose sum of weights is NaN have
// their answer.
//
// Every wait is bounded; on timeout the CTA sets the device error word, drains its copies and MMAs
// and frees TMEM.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "attn_tc.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "paged.cuh"
#include "paged_tc.cuh"
#include "paged_work.cuh"
#include "q4_restore.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_paged_attn_error = 0;

namespace {

using namespace paged;

__device__ __forceinline__ bool bwait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return bounded_wait(bar, parity, abort_flag, &g_paged_attn_error);
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  bounded_drain(bar, parity, &g_paged_attn_error);
}

constexpr int THREADS = 20 * 32;
constexpr int W_MMA = 1, W_SEG = 3, W_SM = 4, W_RST = 12;
constexpr int RST_WARPS = 8;
// A block's start and output take as long as this many units: 8 pieces of 100 .. 256 tokens behind
// 400 .. 2000 positions, 32 heads, 119 us with 0, 95 us with 4, 94 us with 7 when a CTA took 206,000
// cycles at most, 123,000 on average; now 99 us with 4.  Not in calls of few units per CTA, whose
// shares would become fewer.
constexpr int kLead = 4, kLeadFrom = 16;
constexpr int SEGS = 4;                    // ring of segments
constexpr int MAX_PARTS = 12;              // ring of parts (K or V codes of a key tile)
constexpr float kLag = 8.0f;               // base-2 score by which a row may pass its reference
constexpr float kPExp = 7.0f;              // P is scaled by 2^7, as its row sum is: P <= 2^15, and
                                           // down to 2^-21 of the reference's P normal in fp16

// ---------------------------------------------------------------- rows on their own

__device__ __forceinline__ float restored(uint32_t code, uint32_t abw) {
  const float2 ab = unpack_h2(abw);
  const float s = __fdiv_rn(__fsub_rn(ab.y, ab.x), 15.0f);
  return h2f(f2h(__fadd_rn(ab.x, __fmul_rn((float)code, s))));
}
// The K (which 0) or V (1) row of one position and head; null for a bad page.
template <int D>
__device__ __forceinline__ const uint8_t* row_of(const PagedCache& c, int b, int head, int64_t t,
                                                 int which, const uint32_t** ab) {
  const int64_t s = c.slot(b, t);
  if (s < 0) {
    atomicOr(&g_paged_attn_error, kErrExtent);
    return nullptr;
  }
  const uint8_t* k = c.block(s, head, D) + which * c.half_bytes(D);
  const int64_t at = s & ((1 << c.lg) - 1);
  *ab = reinterpret_cast<const uint32_t*>(k + ((int64_t)(D / 2) << c.lg)) + at * (D / 64);
  return k + at * (D / 2);
}
__device__ __forceinline__ float in_range(float y) {
  return fabsf(y) < 66000.0f ? fminf(fmaxf(y, -65504.0f), 65504.0f) : y;
}

// One row on its own, by a whole warp, over the positions that it sees of key tiles j0 .. j1 - 1:
// a position per lane for the scores, channels lane * D/32 .. for the values.  o: unnormalised; m,
// l in the base-2 scale of the kernel.
template <int D>
__device__ __noinline__ void attend_row(const PagedAttn& a, const PagedSeg& g, const uint16_t* q,
                                        int i, float (&o)[D / 32], float& m, float& l) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const float sl2 = a.scale * 1.4426950408889634f;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.0f;
#pragma unroll 1
  for (int j = g.j0; j < g.j1; ++j) {
#pragma unroll 1
    for (int t0 = g.kt.tile(j) * kKeyTile, e = t0 + kKeyTile; t0 < e; t0 += 32) {
      const int t = t0 + lane;
      const bool vis = i >= 0 && visible(t, i, a.window, a.sinks);
      if (!__any_sync(0xFFFFFFFFu, vis)) continue;
      float s = -INFINITY;
      const uint32_t* ab;
      if (vis) {
        const uint8_t* k = row_of<D>(a.cache, g.b, g.hk, t, 0, &ab);
        s = 0.0f;
#pragma unroll 1
        for (int c = 0; k && c < D / 2; ++c)
          s += h2f(q[2 * c]) * restored(k[c] & 15u, ab[c / 32]) +
               h2f(q[2 * c + 1]) * restored(k[c] >> 4, ab[c / 32]);
        s *= sl2;
      }
      float mx = s;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
      mx = fmaxf(mx, m);
      const float ref = mx == -INFINITY ? 0.0f : mx, corr = ex2(m - ref);
      const float p = vis ? ex2(s - ref + kPExp) : 0.0f;
      l = l * corr + p;
      m = mx;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= corr;
#pragma unroll 1
      for (int u = 0; u < 32; ++u) {
        if (!__shfl_sync(0xFFFFFFFFu, vis, u)) continue;
        const float pu = __shfl_sync(0xFFFFFFFFu, p, u);
        const uint8_t* v = row_of<D>(a.cache, g.b, g.hk, t0 + u, 1, &ab);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int ch = lane * C + c;
          if (v) o[c] += pu * restored(v[ch / 2] >> (4 * (ch & 1)) & 15u, ab[ch / 64]);
        }
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
}

// ---------------------------------------------------------------- the kernel

struct PArgs {
  PagedAttn a;
  float scale_log2;
  int G, tpt;
  int parts;           // depth of the ring of parts
  int two;             // blocks of two row tiles occur: Q_B has a buffer
  int min_units;       // of a share
  int slot_rows;       // rows of a partial slot
  PagedCut* cuts;      // [grid]
  float* partial;      // [2 * grid][D/4][slot_rows][4], then maxima and sums [2 * grid][slot_rows][2]
};

// K stages, V stages, Q_A, (Q_B,) parts; barriers and rings behind them.
template <int D>
struct Smem {
  static constexpr int TILE = (D / 64) * BOX;
  static constexpr int PART = 128 * (9 * D / 16);
  static constexpr int K_OFF = 0, V_OFF = 2 * TILE, Q_OFF = 4 * TILE;
  static constexpr int CTRL = 512 + SEGS * 64 + 2 * 128 * 4;      // barriers, segments, B's m and l
  __host__ __device__ static constexpr int part_off(int two) { return Q_OFF + (1 + two) * TILE; }
  __host__ __device__ static constexpr int ctrl_off(int two, int parts) {
    return part_off(two) + parts * PART;
  }
  static constexpr int bytes(int two, int parts) { return ctrl_off(two, parts) + CTRL + 1024; }
  static constexpr int depth(int two) {
    int n = MAX_PARTS;
    while (bytes(two, n) > 227 * 1024) --n;
    return n;
  }
};
static_assert(Smem<128>::depth(1) >= 3 && Smem<128>::depth(0) >= 6, "room for codes in flight");

constexpr int B_CFULL = 0, B_CFREE = MAX_PARTS, B_QFULL = 2 * MAX_PARTS, B_QFREE = B_QFULL + 2,
              B_KFULL = B_QFREE + 2, B_KFREE = B_KFULL + 2, B_VFULL = B_KFREE + 2,
              B_VFREE = B_VFULL + 2, B_SFULL = B_VFREE + 2, B_PFULL = B_SFULL + 2,
              B_ODONE = B_PFULL + 2, B_OFREE = B_ODONE + 2, B_LFULL = B_OFREE + 2,
              B_GFULL = B_LFULL + 1, B_GFREE = B_GFULL + SEGS, B_DRAIN = B_GFREE + SEGS,
              NBARS = B_DRAIN + 2;
static_assert(NBARS * 8 + 16 <= 512 && sizeof(PagedSeg) <= 64, "control space");

// Tokens of row tile t of a block, and whether it takes part in key tile number j.
__device__ __forceinline__ int tile_tokens(const PagedSeg& g, int t, int tpt) {
  return g.single ? g.ntok : (t ? g.ntok - tpt : tpt);
}
__device__ __forceinline__ bool takes_part(const PagedSeg& g, int t, int j, int tpt, int window,
                                           int sinks) {
  if (g.single) return ((j - g.j0) & 1) == t;
  const int lo = g.pos + t * tpt;
  return span_sees(g.kt.tile(j), lo, lo + tile_tokens(g, t, tpt) - 1, window, sinks);
}

// (a called function: groups with infinities or NaN are rare)
__device__ __noinline__ uint4 restore8_any(uint32_t codes, uint32_t abw) {
  return restore8_fp16(codes, abw);
}

// A part from a ring stage into an fp16 tile: two threads per position, 64 channels each (d = 64:
// 32), in binary32, two values per instruction.  (In fp16 arithmetic, with s = (b - a) / 15 as a sum of
// two fp16 numbers, 614 us instead of 647 for the long pieces above, but neighbours of the defined
// values, and up to 5 steps off where s is near fp16's smallest numbers.)
// The upper 64 channels' threads take their words in another order, so that the 16-byte stores of 8
// threads meet all banks.  Positions `valid` .. are not the sequence's: 0.  (The loop stays a loop, for
// K, V and tails alike, so that its instructions stay near.)
template <int D>
__device__ __forceinline__ void restore_part(uint32_t part, uint32_t tile, int lgb, int valid,
                                             int tid) {
  const int row = tid >> 1, h = tid & 1, r = row & ((1 << lgb) - 1);
  const uint32_t sub = part + (((row >> lgb) * (9 * D / 16)) << lgb);
  const uint32_t codes = sub + r * (D / 2) + h * (D / 4);
  const uint32_t abw = ld_shared(sub + ((D / 2) << lgb) + r * (D / 16) + (D == 128 ? 4 * h : 0));
  const uint32_t stats = row < valid ? abw : 0u;       // (0, 0): every code is 0
  const GroupFp16 g(stats);
  const bool plain = __all_sync(0xFFFFFFFFu, g.plain);
  const uint32_t dst = tile + (D == 128 ? h * BOX : 0) + row * 128;
#pragma unroll 1
  for (int it = 0; it < D / 64; ++it) {
    const int half = D == 128 ? it ^ h : h;
    const uint4 w = ld_shared_v4(codes + (D == 128 ? 16 * half : 0));
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const uint32_t to = dst + (((4 * half) ^ (row & 4)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 o = plain ? g.restore(ww[i]) : restore8_any(ww[i], stats);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((i ^ (row & 3)) << 4)),
                   "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w));
    }
  }
}

// 8 output channels as fp16.
__device__ __forceinline__ uint4 pack_channels(const float* o) {
  return make_uint4(pack_h2(in_range(o[0]), in_range(o[1])), pack_h2(in_range(o[2]), in_range(o[3])),
                    pack_h2(in_range(o[4]), in_range(o[5])), pack_h2(in_range(o[6]), in_range(o[7])));
}
template <int D>
__global__ void __launch_bounds__(THREADS, 1)
attend_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ PArgs pa) {
  using L = Smem<D>;
  constexpr int NB = D / 64;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* ctrl = smem + L::ctrl_off(pa.two, pa.parts);
  const uint32_t bar0 = smem_u32(ctrl);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto seg_slot = [&](int n) { return reinterpret_cast<PagedSeg*>(ctrl + 512 + 64 * (n % SEGS)); };
  float* ml_b = reinterpret_cast<float*>(ctrl + 512 + SEGS * 64);   // chain B's maxima and sums
  __shared__ int64_t warp_units[THREADS / 32];
  __shared__ int first_b;                  // the sequence of the share's first unit, and
  __shared__ int64_t first_before;         // the units before it

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedAttn& a = pa.a;
  PagedShape shape{pa.tpt, a.window, a.sinks, 0};
  const int nseq = a.cache.B, H = a.cache.H;

  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_PARTS; ++i) {
      mbar_init(bar(B_CFULL + i), 1);
      mbar_init(bar(B_CFREE + i), RST_WARPS);   // one arrival per restore warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_QFREE + i), 2);      // two arrivals of the issuers' (q_given_*)
      mbar_init(bar(B_KFULL + i), RST_WARPS);
      mbar_init(bar(B_KFREE + i), 2);
      mbar_init(bar(B_VFULL + i), RST_WARPS);
      mbar_init(bar(B_VFREE + i), 2);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), 4);      // one arrival per softmax warp
      mbar_init(bar(B_ODONE + i), 1);
      mbar_init(bar(B_OFREE + i), 4);
      mbar_init(bar(B_DRAIN + i), 1);
    }
    mbar_init(bar(B_LFULL), 4);
    for (int i = 0; i < SEGS; ++i) {
      mbar_init(bar(B_GFULL + i), 1);
      mbar_init(bar(B_GFREE + i), 1 + 2 + 8 + RST_WARPS);      // every other warp
    }
    *abort_flag = 0;
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

  // ---- the order of the work: its units, and where this share's begin
  auto ours = [&](const PagedSeq& s) { return !(a.steps && s.nq == 1); };
  int64_t total = 0, before = 0, incl = 0, mine = 0;
  auto scan_round = [&](int b0) {          // a sequence per thread: its units, those up to it
    const int b = b0 + threadIdx.x;
    mine = 0;
    if (b < nseq) {
      PagedSeq s;
      if (extent_of(a, b, s))
        mine = ours(s) ? H * head_units(s, shape) : 0;
      else if (blockIdx.x == 0)
        atomicOr(&g_paged_attn_error, kErrExtent);
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_units[warp] = incl;
    __syncthreads();
    int64_t round = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
      const int64_t n = warp_units[i];
      if (i < warp) incl += n;
      round += n;
    }
    __syncthreads();
    return round;
  };
  auto scan = [&]() {
    total = 0;
    for (int b0 = 0; b0 < nseq; b0 += THREADS) total += scan_round(b0);
  };
  scan();
  if (total >= (int64_t)kLeadFrom * gridDim.x) {
    shape.lead = kLead;
    scan();
  }
  const int64_t most = total / (pa.min_units + shape.lead);      // so that each begins a key tile
  const int n_shares = (int)min((int64_t)gridDim.x, max((int64_t)1, most));
  const Shares shares(total, n_shares);
  const int share = blockIdx.x;
  const bool busy = total > 0 && share < n_shares;
  const int64_t x0 = busy ? shares.first(share) : 0, x1 = busy ? shares.first(share + 1) : 0;
  if (busy) {
    for (int b0 = 0; b0 < nseq; b0 += THREADS) {
      const int64_t round = nseq > THREADS ? scan_round(b0) : total;
      if (before + round > x0) {
        if (before + incl > x0 && before + incl - mine <= x0) {
          first_b = b0 + threadIdx.x;
          first_before = before + incl - mine;
        }
        break;
      }
      before += round;
    }
  }
  if (!busy && threadIdx.x == 0) pa.cuts[share].pieces = 0;
  // rows before the first position see nothing
  for (int b = blockIdx.x; b < nseq; b += gridDim.x) {
    PagedSeq s;
    if (!extent_of(a, b, s) || s.nq <= s.n) continue;
    const int64_t words = (int64_t)a.Hq * D / 8;
    for (int64_t i = threadIdx.x; i < (s.nq - s.n) * words; i += THREADS) {
      const int64_t row = s.q0 + i / words;
      reinterpret_cast<uint4*>(a.out + row * a.out_stride)[i % words] = make_uint4(0, 0, 0, 0);
    }
    if (a.lse)
      for (int64_t i = threadIdx.x; i < (int64_t)(s.nq - s.n) * a.Hq; i += THREADS)
        a.lse[(int64_t)s.q0 * a.Hq + i] = -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S_A 0..127, S_B 128..255, O_A 256.., O_B 256 + D..
  auto s_col = [&](int t) { return (uint32_t)(t * KT); };
  auto o_col = [&](int t) { return (uint32_t)(2 * KT + t * D); };
  const int lgb = min(a.cache.lg, 7);      // positions of a page within one key tile: 2^lgb
  auto seg_wait = [&](int n) -> bool {
    const bool got = bwait(bar(B_GFULL + n % SEGS), (uint32_t)((n / SEGS) & 1), abort_flag);
    return __all_sync(0xFFFFFFFFu, got);
  };
  auto seg_done = [&](int n) { mbar_arrive(bar(B_GFREE + n % SEGS)); };

  if (warp == 0) {
    // ------------------------------------------------------------ codes
    int np = 0, st = 0, turn = 0;                      // parts issued; ring stage, its turn
    bool ok = true;
    const int subs = 128 >> lgb;
    for (int n = 0; ok; ++n) {
      if (!seg_wait(n)) break;
      const PagedSeg g = *seg_slot(n);
      __syncwarp();
      if (lane == 0) seg_done(n);
      if (g.b < 0) break;
      // lane l holds the block of the page of positions l * 2^lgb .. of a key tile
      auto lookup = [&](int j) -> int64_t {
        const int64_t t = (int64_t)g.kt.tile(j) * kKeyTile + ((int64_t)lane << lgb);
        return lane < subs && t < g.n ? a.cache.slot(g.b, t) : -2;
      };
      int64_t slot = lookup(g.j0);
      for (int j = g.j0; j < g.j1 && ok; ++j) {
        const int64_t at = slot;
        if (j + 1 < g.j1) slot = lookup(j + 1);        // in flight meanwhile
        if (at == -1) atomicOr(&g_paged_attn_error, kErrExtent);
        const unsigned live = __ballot_sync(0xFFFFFFFFu, at >= 0);
        for (int which = 0; which < 2; ++which, ++np) {
          if (turn > 0) {
            const bool fr = bwait(bar(B_CFREE + st), (uint32_t)((turn - 1) & 1), abort_flag);
            if (!__all_sync(0xFFFFFFFFu, fr)) {
              ok = false;
              break;
            }
          }
          const uint32_t bytes = (uint32_t)(9 * D / 16) << lgb;
          if (lane == 0) {
            // the stage was last read through the generic proxy; order that before the copies
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_expect_tx(bar(B_CFULL + st), bytes * __popc(live));
          }
          __syncwarp();
          if (at >= 0) {
            const uint32_t dst = smem_u32(smem + L::part_off(pa.two) + st * L::PART) + lane * bytes;
            const uint8_t* src = a.cache.block(at, g.hk, D) + which * a.cache.half_bytes(D);
            if (a.cache.lg <= 7) {
              bulk_copy(dst, src, bytes, bar(B_CFULL + st));
            } else {                                   // a key tile's piece of a longer page
              const int64_t r = at & ((1 << a.cache.lg) - 1);
              bulk_copy(dst, src + r * (D / 2), 128 * (D / 2), bar(B_CFULL + st));
              bulk_copy(dst + 128 * (D / 2), src + ((int64_t)(D / 2) << a.cache.lg) + r * (D / 16),
                        128 * (D / 16), bar(B_CFULL + st));
            }
          }
          if (++st == pa.parts) {
            st = 0;
            ++turn;
          }
        }
      }
    }
    // every issued copy has landed before the CTA exits
    if (lane == 0)
      for (int i = max(0, np - pa.parts); i < np; ++i)
        drain_wait(bar(B_CFULL + i % pa.parts), (uint32_t)((i / pa.parts) & 1));
    __syncwarp();
  } else if (warp < W_SEG) {
    // ------------------------------------------------------------ MMA issuer of chain t
    // Both chains go through the K and V stages of every key tile in order, and release each: a
    // parity wait cannot tell a use of a stage from the next but one, so neither may fall two behind.
    const int t = __shfl_sync(0xFFFFFFFFu, warp - W_MMA, 0);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), sbase = smem_u32(smem);
    const uint32_t one = elect_one();
    const uint32_t od = tm + o_col(t), scol = tm + s_col(t);
    const uint32_t idesc_o = idesc_pv(D);
    int g0 = 0;                                        // key tiles before the segment
    int q_uses[2] = {0, 0}, pc = 0, uses = 0;          // Q loads; P products; segments with tiles
    bool ok = true;
    auto wait = [&](int b, int parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, bwait(bar(b), (uint32_t)parity, abort_flag));
    };
    auto commit = [&](int b) { umma_commit_if(bar(b), one); };
    auto arrive = [&](int b) {
      if (lane == 0) mbar_arrive(bar(b));
    };
    for (int n = 0; ok; ++n) {
      if (!seg_wait(n)) break;
      const PagedSeg g = *seg_slot(n);
      __syncwarp();
      if (lane == 0) seg_done(n);
      if (g.b < 0) break;
      const int qb = g.single ? 0 : t;                 // the chain's Q buffer
      const uint64_t qd =
          smem_desc(__shfl_sync(0xFFFFFFFFu, sbase + L::Q_OFF + qb * L::TILE, 0), 16, 1024);
      wait(B_QFULL, q_uses[0]++ & 1);
      if (!g.single) {
        if (t == 1) wait(B_QFULL + 1, q_uses[1] & 1);
        ++q_uses[1];
      }
      if (!ok) break;
      if (q_given_at_once(t, g.single)) arrive(B_QFREE);
      const int q_given = q_given_after_use(t, g.single);
      auto own = [&](int j) { return takes_part(g, t, j, pa.tpt, a.window, a.sinks); };
      auto next_own = [&](int j) {
        while (j < g.j1 && !own(j)) ++j;
        return __shfl_sync(0xFFFFFFFFu, j, 0);
      };
      // waits for the stages of key tiles seen .. j, of which all but j are the other chain's
      int k_seen = g.j0, v_seen = g.j0;
      auto wait_to = [&](int& seen, int j, int full, int free) {
        for (; seen < j; ++seen) {
          const int x = g0 + seen - g.j0;
          wait(full + (x & 1), (x >> 1) & 1);
          if (ok) arrive(free + (x & 1));
        }
        if (j < g.j1) {
          const int x = g0 + j - g.j0;
          wait(full + (x & 1), (x >> 1) & 1);
          ++seen;
        }
      };
      auto issue_s = [&](int j) {
        const int st = __shfl_sync(0xFFFFFFFFu, (g0 + j - g.j0) & 1, 0);
        const uint64_t kd =
            smem_desc(__shfl_sync(0xFFFFFFFFu, sbase + L::K_OFF + st * L::TILE, 0), 16, 1024);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint64_t off = (uint64_t)(((i >> 2) * BOX + (i & 3) * 32) >> 4);
          umma_f16_if(scol, qd + off, kd + off, kIdescS, i > 0, one);
        }
        commit(B_SFULL + t);
        commit(B_KFREE + st);
      };
      auto issue_pv = [&](int j, uint32_t add) {
        const int st = __shfl_sync(0xFFFFFFFFu, (g0 + j - g.j0) & 1, 0);
        const uint64_t vd =
            smem_desc(__shfl_sync(0xFFFFFFFFu, sbase + L::V_OFF + st * L::TILE, 0), BOX, 1024);
        umma_ts_if(od, scol, vd, idesc_o, add, one);
#pragma unroll
        for (int i = 1; i < KT / 16; ++i)
          umma_ts_if(od, scol + 32 * (i >> 1) + 8 * (i & 1), vd + (uint64_t)(i * 128), idesc_o, 1u,
                     one);
        commit(B_VFREE + st);
      };
      int j = next_own(g.j0);
      uint32_t add = 0;
      wait_to(k_seen, j, B_KFULL, B_KFREE);
      if (!ok) break;
      if (j < g.j1) {
        tc_fence_after();
        issue_s(j);
      }
      while (j < g.j1) {
        const int jn = next_own(j + 1);
        if (jn >= g.j1) {                              // the chain's last S product of the segment
          commit(B_QFREE + qb);
          if (q_given == 2) commit(B_QFREE + qb);
        }
        wait_to(v_seen, j, B_VFULL, B_VFREE);
        // the first product of a segment overwrites O_t: its last values have been read
        if (!add && uses > 0) wait(B_OFREE + t, (uses - 1) & 1);
        wait(B_PFULL + t, pc++ & 1);
        if (!ok) break;
        tc_fence_after();
        issue_pv(j, add);
        add = 1;
        wait_to(k_seen, jn, B_KFULL, B_KFREE);
        if (!ok) break;
        if (jn < g.j1) {
          // S's columns hold no P that is still to be read (the product above was issued before)
          tc_fence_after();
          issue_s(jn);
        }
        j = jn;
      }
      if (!ok) break;
      if (add) {
        commit(B_ODONE + t);
        ++uses;
      } else {                                         // no part in any key tile
        arrive(B_QFREE + qb);
        if (q_given == 2) arrive(B_QFREE + qb);
      }
      wait_to(v_seen, g.j1, B_VFULL, B_VFREE);
      g0 += g.j1 - g.j0;
    }
    // the CTA frees TMEM only after every MMA issued here has completed
    commit(B_DRAIN + t);
    if (one) drain_wait(bar(B_DRAIN + t), 0u);
    __syncwarp();
  } else if (warp == W_SEG) {
    // ------------------------------------------------------------ segments, and their Q
    if (lane == 0) {
      PagedWalk k;
      k.sh = shape;
      k.share = share;
      k.H = H;
      k.x0 = x0;
      k.x1 = x1;
      bool more = busy;
      if (busy) {
        PagedSeq s;
        extent_of(a, first_b, s);
        k.start(s, first_b, first_before);
      }
      PagedCut cut{};
      // the next segment of the share (b < 0: none)
      auto next = [&](bool first) {
        PagedSeg g;
        g.b = -1;
        while (more) {
          bool got = false;
          if (k.at >= k.x1) {
            more = false;
            break;
          }
          const PagedBlock blk = paged_block(k.s, k.blk, shape);
          got = k.segment(g, blk);
          if (got && first && g.j0 > 0 && shares.share_of(k.at) == share - 1) {
            const int64_t last = k.at + blk.begin(blk.kt.count() - 1);
            cut = PagedCut{shares.share_of(last) - share + 2, g.q0, g.ntok, g.hk};
          }
          k.at += blk.units();
          if (++k.blk >= paged_blocks(k.s, shape.tpt)) {
            k.blk = 0;
            if (++k.hk == H) {
              k.hk = 0;
              do {
                if (++k.b >= nseq) {
                  more = false;
                  break;
                }
                k.per_head = extent_of(a, k.b, k.s) && ours(k.s) ? head_units(k.s, shape) : 0;
              } while (k.per_head == 0);
            }
          }
          if (got) break;
          g.b = -1;
        }
        return g;
      };
      int made = 0, loaded = 0, q_b = 0;               // segments; of them with Q issued; Q_B loads
      bool ended = false;
      long long t0 = clock64();
      while (!ended || loaded < made) {
        bool moved = false;
        if (!ended && (made < SEGS || mbar_test(bar(B_GFREE + made % SEGS),
                                                (uint32_t)((made / SEGS - 1) & 1)))) {
          const PagedSeg g = next(made == 0);
          *seg_slot(made) = g;
          mbar_arrive(bar(B_GFULL + made % SEGS));
          ended = g.b < 0;
          if (!ended) ++made;
          moved = true;
        }
        if (loaded < made) {
          const PagedSeg* g = seg_slot(loaded);
          const int two = !g->single;
          if ((loaded == 0 || mbar_test(bar(B_QFREE), (uint32_t)((loaded - 1) & 1))) &&
              (!two || q_b == 0 || mbar_test(bar(B_QFREE + 1), (uint32_t)((q_b - 1) & 1)))) {
            for (int t = 0; t <= two; ++t) {
              mbar_expect_tx(bar(B_QFULL + t), (uint32_t)(NB * pa.G * pa.tpt * 128));
              for (int c = 0; c < NB; ++c)
                tma_load_3d(smem_u32(smem + L::Q_OFF + t * L::TILE + c * BOX), &tmQ, 64 * c,
                            g->hk * pa.G, g->q0 + t * pa.tpt, bar(B_QFULL + t));
            }
            ++loaded;
            q_b += two;
            moved = true;
          }
        }
        if (moved) {
          t0 = clock64();
          continue;
        }
        __nanosleep(400);                              // leaves the issue slots to the others
        if (*abort_flag || clock64() - t0 > kWaitCycles) {
          if (!*abort_flag) atomicOr(&g_paged_attn_error, kErrWait);
          *abort_flag = 1;
          break;
        }
      }
      if (busy) pa.cuts[share] = cut;
      if (loaded > 0) drain_wait(bar(B_QFULL), (uint32_t)((loaded - 1) & 1));
      if (q_b > 0) drain_wait(bar(B_QFULL + 1), (uint32_t)((q_b - 1) & 1));
    }
    __syncwarp();
  } else if (warp >= W_RST) {
    // ------------------------------------------------------------ restore
    const int tid = threadIdx.x - W_RST * 32;
    int st = 0, turn = 0, g2 = 0;                      // ring stage, its turn; key tiles restored
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!seg_wait(n)) break;
      const PagedSeg* slot = seg_slot(n);
      const int b = slot->b, j1 = slot->j1, len = slot->n;
      const KeyTiles kt = slot->kt;
      int j = slot->j0;
      __syncwarp();
      if (lane == 0) seg_done(n);
      if (b < 0) break;
      for (; j < j1 && ok; ++j) {
        const int valid = min(128, len - kt.tile(j) * kKeyTile);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
          bool got = bwait(bar(B_CFULL + st), (uint32_t)(turn & 1), abort_flag);
          if (g2 >= 2)
            got = got && bwait(bar((which ? B_VFREE : B_KFREE) + (g2 & 1)),
                               (uint32_t)(((g2 >> 1) - 1) & 1), abort_flag);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          const uint32_t part = smem_u32(smem + L::part_off(pa.two) + st * L::PART);
          const uint32_t tile = smem_u32(smem + (which ? L::V_OFF : L::K_OFF) + (g2 & 1) * L::TILE);
          restore_part<D>(part, tile, lgb, valid, tid);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(B_CFREE + st));
            mbar_arrive(bar((which ? B_VFULL : B_KFULL) + (g2 & 1)));
          }
          g2 += which;
          if (++st == pa.parts) {
            st = 0;
            ++turn;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and output of chain t
    const int t = (warp - W_SM) >> 2;
    const int quarter = warp & 3;                      // TMEM lanes 32 quarter ..
    const int m = 32 * quarter + lane;                 // row within the row tile
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t srow = lane_addr + s_col(t);
    const float sl2 = pa.scale_log2;
    const int tok = m / pa.G, gh = m - tok * pa.G;     // the row's token in the tile, its head
    const float* mb = ml_b;
    const float* lb = ml_b + 128;
    int sc = 0, uses = 0, uses_b = 0, joins = 0;       // S products, own segments, B's, joined ones
    bool ok = true;
    // tcgen05.ld / st are warp-collective: every branch around them is decided for the whole warp
    for (int n = 0; ok; ++n) {
      if (!seg_wait(n)) break;
      const PagedSeg& g = *seg_slot(n);                // read where needed: no registers for it
      if (g.b < 0) break;
      const int ntok = tile_tokens(g, t, pa.tpt), pos0 = g.pos + (g.single ? 0 : t * pa.tpt);
      const bool mine = tok < ntok && m < pa.G * pa.tpt;
      const bool any_row = __any_sync(0xFFFFFFFFu, mine);
      const int i = pos0 + tok;                        // the row's position
      // (rows of no token: no score of theirs moves the reference of the warp's rows)
      float m_ref = mine ? -INFINITY : INFINITY, l_sum = 0.0f;
      bool some = false;                               // a key tile of the segment is the chain's
      for (int j = g.j0; j < g.j1; ++j) {
        if (!takes_part(g, t, j, pa.tpt, a.window, a.sinks)) continue;
        const bool got = bwait(bar(B_SFULL + t), (uint32_t)(sc++ & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (any_row) {
          // masked: some row does not see every key of the tile; ahead: the first row's position
          // less the key tile's first
          const int k0 = g.kt.tile(j) * kKeyTile, ahead = pos0 - k0;
          const bool masked = ahead < KT - 1 || (a.window != 0 && k0 + KT > a.sinks &&
                                                 ahead + ntok > a.window);
          // (16 columns at a time in loops: 32 at a time and unrolled took twice the instructions,
          // for want of registers, and the warps waited for them)
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto max_chunk = [&](const float (&v)[16]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], v[e], v[e + 1]);
          };
          float va[16], vb[16];
          unsigned none = 0;                           // chunks that no row of the warp sees
          if (masked) {
            // keys that a row does not see are set to -inf, in TMEM too: pass 2 reads them there
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              const uint32_t vis =
                  mine && i >= 0 ? visible_bits(k0 + 16 * c, i, a.window, a.sinks) & 0xFFFFu : 0u;
              if (!__any_sync(0xFFFFFFFFu, vis != 0u)) {
                none |= 1u << c;
                continue;
              }
              tmem_ld16f(srow + 16 * c, va);
              tmem_wait_ld_dep(va);
              if (!__all_sync(0xFFFFFFFFu, vis == 0xFFFFu)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) va[e] = (vis >> e & 1u) ? va[e] : -INFINITY;
                tmem_st16(srow + 16 * c, reinterpret_cast<const uint32_t*>(va));
              }
              max_chunk(va);
            }
            tmem_wait_st();
          } else {
            tmem_ld16f(srow, va);
            tmem_wait_ld_dep(va);
#pragma unroll 1
            for (int c = 0; c < 8; c += 2) {           // the next load in flight
              tmem_ld16f(srow + 16 * c + 16, vb);
              max_chunk(va);
              tmem_wait_ld_dep(vb);
              if (c < 6) tmem_ld16f(srow + 16 * c + 32, va);
              max_chunk(vb);
              tmem_wait_ld_dep(va);
            }
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
          if (__any_sync(0xFFFFFFFFu, mx > m_ref + kLag)) {
            // move the reference of every row of the warp to max(m_ref, mx): O and l scale by
            // 2^(m_ref - m_new).  O holds P V of the segment's earlier tiles: done before this S
            const float m_new = fmaxf(m_ref, mx);
            const float alpha = (m_ref == -INFINITY) ? 0.0f : ex2(m_ref - m_new);
            if (some) {
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
          const float ref = (m_ref == -INFINITY) ? 0.0f : m_ref;
          const uint64_t sl2x2 = f2pack(sl2, sl2), negm2 = f2pack(kPExp - ref, kPExp - ref);
          uint64_t ls2[2] = {f2pack(0.0f, 0.0f), f2pack(0.0f, 0.0f)};
          // P of keys 32 c .. lies in the first 16 of their S columns
          auto p_chunk = [&](const float (&v)[16], int c) {
            uint32_t pw[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 x = f2unpack(ffma2(f2pack(v[e], v[e + 1]), sl2x2, negm2));
              const float p0 = ex2(x.x), p1 = ex2(x.y);
              ls2[(e >> 1) & 1] = fadd2(ls2[(e >> 1) & 1], f2pack(p0, p1));
              pw[e / 2] = pack_h2(p0, p1);
            }
            tmem_st8(srow + 32 * (c >> 1) + 8 * (c & 1), pw);
          };
          if (!masked) {
            tmem_ld16f(srow, va);
            tmem_wait_ld_dep(va);
#pragma unroll 1
            for (int c = 0; c < 8; c += 2) {
              tmem_ld16f(srow + 16 * c + 16, vb);
              p_chunk(va, c);
              tmem_wait_ld_dep(vb);
              if (c < 6) tmem_ld16f(srow + 16 * c + 32, va);
              p_chunk(vb, c + 1);
              tmem_wait_ld_dep(va);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              if (none >> c & 1u) {
                const uint32_t zeros[8] = {};
                tmem_st8(srow + 32 * (c >> 1) + 8 * (c & 1), zeros);
              } else {
                tmem_ld16f(srow + 16 * c, va);
                tmem_wait_ld_dep(va);
                p_chunk(va, c);
              }
            }
          }
          tmem_wait_st();
          const float2 la = f2unpack(fadd2(ls2[0], ls2[1]));
          l_sum += la.x + la.y;
        }
        some = true;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + t));
      }
      if (!ok) break;

      // ---- the segment's rows
      const bool b_has = g.single && g.j1 - g.j0 >= 2;  // a single block's key tiles are both's
      if (g.single && t == 1) {
        if (b_has) {
          // A joins: hand it the maxima and sums, once it has taken those of the join before
          if (uses > 0) {
            const bool fr = bwait(bar(B_OFREE + 1), (uint32_t)((uses - 1) & 1), abort_flag);
            if (!__all_sync(0xFFFFFFFFu, fr)) break;
          }
          ml_b[m] = m_ref;
          ml_b[128 + m] = l_sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_LFULL));
          ++uses;
        }
        __syncwarp();
        if (lane == 0) seg_done(n);
        continue;
      }
      bool got = true;
      if (some) got = bwait(bar(B_ODONE + t), (uint32_t)(uses & 1), abort_flag);
      if (b_has) {
        got = got && bwait(bar(B_LFULL), (uint32_t)(joins & 1), abort_flag);
        got = got && bwait(bar(B_ODONE + 1), (uint32_t)(uses_b & 1), abort_flag);
      }
      if (!__all_sync(0xFFFFFFFFu, got)) break;
      tc_fence_after();
      // O = O_A fa + O_B fb over the common maximum
      float fa = 1.0f, fb = 0.0f, l = l_sum, mm = m_ref;
      if (b_has) {
        const float m2 = mb[m], l2 = lb[m];
        mm = fmaxf(m_ref, m2);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        fa = ex2(m_ref - ref);
        fb = ex2(m2 - ref);
        l = l_sum * fa + l2 * fb;
      }
      if (l == 0.0f) mm = -INFINITY;
      if (any_row) {
        const int row = g.q0 + (g.single ? 0 : t * pa.tpt) + tok, hq = g.hk * pa.G + gh;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = a.out + (int64_t)row * a.out_stride + (int64_t)hq * D;
        // (4 channels of all rows side by side, so that a warp's store is one run of 512 bytes, and the
        // merge's loads are: 169 us for a mixed batch, 172 us with a row's channels together)
        const int in_slot = (g.single ? 0 : t * pa.tpt * pa.G) + m;
        const int64_t pr = (int64_t)g.slot * pa.slot_rows + in_slot;
        float* part = pa.partial + (int64_t)g.slot * pa.slot_rows * D + 4 * in_slot;
        if (g.slot < 0) {
          fa *= inv;
          fb *= inv;
        }
        // x * 0 summed: NaN for an infinity or a NaN.  Those rows are computed again; where out is q
        // they are found before anything is stored over their queries.
        __half2 zero = __float2half2_rn(0.0f);
        bool stores = mine;
        const int first = g.slot < 0 && a.out == a.q ? -D / 16 : 0;
#pragma unroll 1
        for (int cc = first; cc < D / 16; ++cc) {
          const int c = cc < 0 ? cc + D / 16 : cc;
          if (first < 0 && cc == 0)
            stores = mine && !__hisnan(__low2half(zero)) && !__hisnan(__high2half(zero));
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.0f;
          if (some) {
            tmem_ld16f(lane_addr + o_col(t) + 16 * c, o);
            tmem_wait_ld_dep(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= fa;
          }
          if (b_has) {
            float o2[16];
            tmem_ld16f(lane_addr + o_col(1) + 16 * c, o2);
            tmem_wait_ld_dep(o2);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(o2[e], fb, o[e]);
          }
          if (g.slot < 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4 p = pack_channels(o + 8 * k);
              const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
              if (stores && cc >= 0) *reinterpret_cast<uint4*>(out + 16 * c + 8 * k) = p;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                zero = __hfma2(*reinterpret_cast<const __half2*>(&pw[e]), __float2half2_rn(0.0f),
                               zero);
            }
          } else {
            float z = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              if (mine)
                *reinterpret_cast<float4*>(part + (int64_t)(16 * c + e) * pa.slot_rows) =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
#pragma unroll
              for (int x = 0; x < 4; ++x) z = fmaf(o[e + x], 0.0f, z);
            }
            zero = __hadd2(zero, __float2half2_rn(z));
          }
        }
        if (mine) {
          if (g.slot < 0) {
            if (a.lse)
              a.lse[(int64_t)row * a.Hq + hq] =
                  l == 0.0f ? -INFINITY : (mm + log2f(l) - kPExp) * 0.6931471805599453f;
          } else {
            float* ml = pa.partial + (int64_t)2 * gridDim.x * pa.slot_rows * D + pr * 2;
            ml[0] = mm;
            ml[1] = l;
          }
        }
        // rows with an infinity or NaN, over what they see alone
        unsigned redo = __ballot_sync(0xFFFFFFFFu, mine && !isnan(l) &&
                                                       (__hisnan(__low2half(zero)) ||
                                                        __hisnan(__high2half(zero))));
        for (; redo; redo &= redo - 1) {
          const int src = __ffs(redo) - 1;
          const int rrow = __shfl_sync(0xFFFFFFFFu, row, src), rhq = __shfl_sync(0xFFFFFFFFu, hq, src);
          const int ri = __shfl_sync(0xFFFFFFFFu, i, src);
          const int64_t rpr = pr - lane + src;
          float o[D / 32], rm, rl;
          attend_row<D>(a, g, a.q + (int64_t)rrow * a.q_stride + (int64_t)rhq * D, ri, o, rm, rl);
          const float f = rl == 0.0f ? 0.0f : 1.0f / rl;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const int ch = lane * (D / 32) + c;
            if (g.slot < 0)
              a.out[(int64_t)rrow * a.out_stride + (int64_t)rhq * D + ch] = f2h(in_range(o[c] * f));
            else
              pa.partial[(int64_t)g.slot * pa.slot_rows * D + (int64_t)(ch & ~3) * pa.slot_rows +
                         4 * (in_slot - lane + src) + (ch & 3)] = o[c];
          }
          if (g.slot >= 0 && lane == 0) {
            float* ml = pa.partial + (int64_t)2 * gridDim.x * pa.slot_rows * D + rpr * 2;
            ml[0] = rl == 0.0f ? -INFINITY : rm;
            ml[1] = rl;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (some) mbar_arrive(bar(B_OFREE + t));
        if (b_has) mbar_arrive(bar(B_OFREE + 1));
      }
      if (some) ++uses;
      if (b_has) {
        ++uses_b;
        ++joins;
      }
      if (t == 0 && !g.single)                         // B's segments with key tiles
        for (int j = g.j1 - 1; j >= g.j0; --j)
          if (takes_part(g, 1, j, pa.tpt, a.window, a.sinks)) {
            ++uses_b;
            break;
          }
      __syncwarp();
      if (lane == 0) seg_done(n);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS)
                 : "memory");
  }
}

// Puts cut blocks together: a thread per row and 16 channels, its pieces (m, l, unnormalised O) in
// order.
constexpr int kMergeWarps = 8, kMergeSplit = 16;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(const PArgs pa, int ncta) {
  pdl_launch_dependents();
  pdl_wait();
  const PagedCut cut = pa.cuts[blockIdx.x];
  if (cut.pieces == 0) return;
  const int lane = threadIdx.x & 31, rows = cut.ntok * pa.G;
  const int64_t slot_floats = (int64_t)pa.slot_rows * D;
  const float* ml = pa.partial + 2 * ncta * slot_floats;
  for (int u = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); u < (rows + 31) / 32 * (D / 16);
       u += gridDim.y * kMergeWarps) {
    const int r = u / (D / 16) * 32 + lane, ch = u % (D / 16) * 16;
    if (r >= rows) continue;
    auto slot = [&](int i) { return (int64_t)cut_slot(blockIdx.x, cut.pieces, i); };
    auto max_sum = [&](int i) {
      return *reinterpret_cast<const float2*>(ml + 2 * (slot(i) * pa.slot_rows + r));
    };
    float M = -INFINITY, L = 0.0f, o[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] = 0.0f;
#pragma unroll 8
    for (int i = 0; i < cut.pieces; ++i) M = fmaxf(M, max_sum(i).x);
    const float ref = (M == -INFINITY) ? 0.0f : M;
#pragma unroll 4
    for (int i = 0; i < cut.pieces; ++i) {
      const float2 x = max_sum(i);
      const float* p = pa.partial + slot(i) * slot_floats + (int64_t)ch * pa.slot_rows + 4 * r;
      float4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = *reinterpret_cast<const float4*>(p + (int64_t)(4 * c) * pa.slot_rows);
      const float w = exp2f(x.x - ref);    // 0 * NaN where a piece is NaN: as without a cut
      L = fmaf(w, x.y, L);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[4 * c] = fmaf(w, v[c].x, o[4 * c]);
        o[4 * c + 1] = fmaf(w, v[c].y, o[4 * c + 1]);
        o[4 * c + 2] = fmaf(w, v[c].z, o[4 * c + 2]);
        o[4 * c + 3] = fmaf(w, v[c].w, o[4 * c + 3]);
      }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t row = cut.q0 + r / pa.G;
    const int hq = cut.hk * pa.G + r % pa.G;
#pragma unroll
    for (int c = 0; c < 16; ++c) o[c] *= inv;
    uint4* op = reinterpret_cast<uint4*>(pa.a.out + row * pa.a.out_stride + (int64_t)hq * D + ch);
    op[0] = pack_channels(o);
    op[1] = pack_channels(o + 8);
    if (pa.a.lse && ch == 0)
      pa.a.lse[row * pa.a.Hq + hq] =
          L == 0.0f ? -INFINITY : (M + log2f(L) - kPExp) * 0.6931471805599453f;
  }
}

// ---------------------------------------------------------------- host

int tokens_per_tile(int G) { return 128 / G; }
int slot_rows_of(int G, int max_q) {
  const int tpt = tokens_per_tile(G);
  return G * std::min(max_q, 2 * tpt);
}
size_t cut_bytes(int grid) { return (grid * sizeof(PagedCut) + 255) / 256 * 256; }

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
  using L = Smem<D>;
  e = cudaFuncSetAttribute(attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           std::max(L::bytes(0, L::depth(0)), L::bytes(1, L::depth(1))));
  done[dev] = e == cudaSuccess;
  return e;
}

template <int D>
cudaError_t launch_d(const PagedAttn& a, void* ws, int nsm, cudaStream_t st) {
  using L = Smem<D>;
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess || (e = get_encode()) != cudaSuccess) return e;
  PArgs pa;
  pa.a = a;
  pa.scale_log2 = a.scale * 1.4426950408889634f;
  pa.G = a.Hq / a.cache.H;
  pa.tpt = tokens_per_tile(pa.G);
  pa.two = std::min(a.max_q, a.q_rows) > pa.tpt;
  pa.parts = L::depth(pa.two);
  pa.min_units = 1 + pa.two;
  pa.slot_rows = slot_rows_of(pa.G, a.max_q);
  const int grid = std::max(nsm, 1);       // one CTA per SM
  pa.cuts = static_cast<PagedCut*>(ws);
  pa.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + cut_bytes(grid));
  CUtensorMap tq;
  e = make_map_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q, D, (uint64_t)a.Hq, (uint64_t)a.q_rows,
                  2 * D, (uint64_t)a.q_stride * 2, 64, pa.G, CU_TENSOR_MAP_SWIZZLE_128B, pa.tpt);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attend_kernel<D>, dim3(grid), dim3(THREADS), L::bytes(pa.two, pa.parts), st, tq,
                 pa);
  if (e != cudaSuccess) return e;
  const int units = (pa.slot_rows + 31) / 32 * (D / 16);
  const int split = std::min((units + kMergeWarps - 1) / kMergeWarps, kMergeSplit);
  return launch_pdl(merge_kernel<D>, dim3(grid, split), dim3(kMergeWarps * 32), 0, st, pa, grid);
}

}  // namespace

// Scratch of this file's kernels; that of the single tokens' follows.
static size_t tiles_ws_bytes(int G, int d, int max_q) {
  return (cut_bytes(kMaxSms) +
          (size_t)2 * kMaxSms * slot_rows_of(G, max_q) * (d + 2) * sizeof(float) + 255) /
         256 * 256;
}
size_t attn_paged_ws_bytes(const fg_kvpages& kv, int32_t Hq, int32_t max_q) {
  const int G = Hq / kv.H;
  return tiles_ws_bytes(G, kv.h / kv.H, max_q) +
         (G <= kStepHeads ? attn_paged_step_ws_bytes(kv, Hq) : 0);
}

// Single query rows with few heads go to the streaming kernels: alone where no sequence has more, and
// ahead of the others where several sequences may be mixed.  (16 contexts of 9000 .. 32760, 8 K/V
// heads: 178 to 182 us there with 1 to 8 query heads each, 290 us here with any.)
cudaError_t launch_attn_paged(const PagedAttn& call, int d, void* ws, int nsm, cudaStream_t st) {
  PagedAttn a = call;
  const int G = a.Hq / a.cache.H;
  a.steps = G <= kStepHeads && (a.max_q == 1 || a.cache.B > 1);
  if (a.steps) {
    void* sws = static_cast<uint8_t*>(ws) + tiles_ws_bytes(G, d, a.max_q);
    cudaError_t e = launch_attn_paged_step(a, d, sws, nsm, st);
    if (e != cudaSuccess || a.max_q == 1) return e;
  }
  return d == 128 ? launch_d<128>(a, ws, nsm, st) : launch_d<64>(a, ws, nsm, st);
}

cudaError_t paged_attn_read_error(unsigned int* out) {
  return read_and_clear(g_paged_attn_error, out);
}

}  // namespace fg
