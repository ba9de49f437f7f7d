// The softmax weights that positions of the paged 4-bit cache receive from given queries, on the
// 5th-generation tensor cores (sm_103a):
//   acc_out[b][hk][t] = acc[b][hk][t] + sum exp(scale q_row,hq . k^_t - lse[row][hq])
// over sequence b's query rows that see position t and the query heads of K/V head hk.
//
// The log-sum-exp of a row is given, so no softmax runs: a position's sum needs nothing of the
// others, and with positions in the rows of the product (S^T = K Q^T: tensor memory lanes) and query
// rows in its columns, a thread owns a position and adds up its columns.  No partial sums, no
// atomics, one order of additions.
//
// An item is 256 positions of one K/V head (two key tiles of 128), against every row tile (128 / G
// tokens of G heads) that sees one; items stand in one order, cut evenly by cost (paged_work.cuh).
//   warp 0        page table lookups and bulk copies of the K codes and statistics, one per page
//   warp 1        MMA issuer: per row tile S^T of both key tiles, two S buffers each
//   warp 2        Q row tiles by TMA, a ring of two (two or fewer stay while the K/V head does)
//   warp 3        items
//   warps 4-11    a key tile each four: exponentials and sums
//   warps 12-15   K^ = fp16(a + q (b - a) / 15) exactly as defined (the sums are binary32, and
//                 errors of K^ would show in them), once per item
// What bounds it: with few rows, restoring K (25 instructions for every 8 codes) and its bytes (0.5625
// d per position); with many, the exponentials beside it, one per pair.  The last 64 tokens of 8 prompts
// of 8001 .. 16,001 positions, 32 query heads over 8, 196 million pairs: 95 us (126 us with 20 warps of
// 96 registers, whose exponentials took three times the instructions; 3 us are the test for rows of
// log-sum-exp -inf with infinities or NaN in their scores); the restoring warps work 98,000 cycles of a
// CTA's time.
#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "paged_tc.cuh"
#include "q4_restore.cuh"

namespace fg {

__device__ unsigned int g_weights_error = 0;

namespace {

using namespace paged;

__device__ __forceinline__ bool bwait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return bounded_wait(bar, parity, abort_flag, &g_weights_error);
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  bounded_drain(bar, parity, &g_weights_error);
}

constexpr int THREADS = 16 * 32;
constexpr int W_MMA = 1, W_Q = 2, W_ITEM = 3, W_EXP = 4, W_RST = 12, RST_WARPS = 4;
constexpr int ITEMS = 4, KRING = 4, MAX_PARTS = 8;

struct Item {
  int b, hk;           // sequence (-1: no more items), K/V head
  int q0, nq, n, k0, r0, r1;
  int tiles;           // row tiles of the sequence
  int keep, keep_next; // its Q tiles are those of the item before; stay for the next
};
static_assert(sizeof(Item) <= 64, "item ring");

struct WArgs {
  PagedAttn a;
  float scale_log2;
  int G, tpt, parts;
};

template <int D>
struct Smem {
  static constexpr int TILE = (D / 64) * BOX;
  static constexpr int PART = 128 * (9 * D / 16);
  static constexpr int K_OFF = 0, Q_OFF = KRING * TILE, PART_OFF = Q_OFF + 2 * TILE;
  static constexpr int LSE = 2 * 2 * 128 * 4;
  static constexpr int CTRL = 512 + ITEMS * 64 + LSE;
  __host__ __device__ static constexpr int ctrl_off(int parts) { return PART_OFF + parts * PART; }
  static constexpr int bytes(int parts) { return ctrl_off(parts) + CTRL + 1024; }
  static constexpr int depth() {
    int n = MAX_PARTS;
    while (bytes(n) > 226 * 1024) --n;
    return n;
  }
};
static_assert(Smem<128>::depth() >= 2, "room for codes in flight");

constexpr int B_CFULL = 0, B_CFREE = MAX_PARTS, B_KFULL = 2 * MAX_PARTS, B_KFREE = B_KFULL + KRING,
              B_QFULL = B_KFREE + KRING, B_QFREE = B_QFULL + 2, B_SFULL = B_QFREE + 2,
              B_SFREE = B_SFULL + 4, B_ZFULL = B_SFREE + 4, B_IFULL = B_ZFULL + 4,
              B_IFREE = B_IFULL + ITEMS, B_DRAIN = B_IFREE + ITEMS, NBARS = B_DRAIN + 1;
static_assert(NBARS * 8 + 16 <= 512, "control space");

// Columns of a row tile that a position adds up: all; those that see it; of those, the ones whose row
// has a log-sum-exp.
enum { kAll, kSome, kHeard };
template <int N>
using Columns = std::integral_constant<int, N>;
constexpr float kSilent = -0x1.fffffep127f;

// (a called function: groups with infinities or NaN are rare)
__device__ __noinline__ uint4 restore8_any(uint32_t codes, uint32_t abw) {
  return restore8_fp16(codes, abw);
}

// A K part into an fp16 tile, a thread per position.  Positions take their 16-byte pieces of codes in
// different orders, so that 8 threads' loads, and their stores, meet all banks (the loops stay loops,
// so that their instructions stay near).
template <int D>
__device__ __forceinline__ void restore_k(uint32_t part, uint32_t tile, int lgb, int valid,
                                          int row) {
  const int r = row & ((1 << lgb) - 1);
  const uint32_t sub = part + (((row >> lgb) * (9 * D / 16)) << lgb);
  const uint32_t codes = sub + r * (D / 2), ab = sub + ((D / 2) << lgb) + r * (D / 16);
#pragma unroll 1
  for (int it = 0; it < D / 64; ++it) {
    const int gr = D == 128 ? it ^ (row >> 2 & 1) : 0;
    const uint32_t word = ld_shared(ab + 4 * gr);
    const uint32_t abw = row < valid ? word : 0u;      // (0, 0): every code is 0
    const GroupFp16 g(abw);
    const bool plain = __all_sync(0xFFFFFFFFu, g.plain);
    const uint32_t dst = tile + gr * BOX + row * 128;
#pragma unroll 1
    for (int jt = 0; jt < 2; ++jt) {
      const int half = jt ^ (row >> (D == 128 ? 1 : 2) & 1);
      const uint4 w = ld_shared_v4(codes + gr * 32 + half * 16);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      const uint32_t to = dst + (((4 * half) ^ (row & 4)) << 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 o = plain ? g.restore(ww[i]) : restore8_any(ww[i], abw);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((i ^ (row & 3)) << 4)),
                     "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w));
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ WArgs wa) {
  using L = Smem<D>;
  constexpr int NB = D / 64;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* ctrl = smem + L::ctrl_off(wa.parts);
  const uint32_t bar0 = smem_u32(ctrl);
  auto bar = [&](int i) { return bar0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + NBARS * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto item_slot = [&](int n) { return reinterpret_cast<Item*>(ctrl + 512 + 64 * (n % ITEMS)); };
  float* lse_buf = reinterpret_cast<float*>(ctrl + 512 + ITEMS * 64);    // [key tile][buffer][row]
  __shared__ int64_t warp_units[THREADS / 32];
  __shared__ int first_b;                  // the sequence of the share's first unit, and
  __shared__ int64_t first_before;         // the units before it

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedAttn& a = wa.a;
  const PagedShape shape{wa.tpt, a.window, a.sinks, 0};
  const int nseq = a.cache.B, H = a.cache.H;

  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_PARTS; ++i) {
      mbar_init(bar(B_CFULL + i), 1);
      mbar_init(bar(B_CFREE + i), RST_WARPS);
    }
    for (int i = 0; i < KRING; ++i) {
      mbar_init(bar(B_KFULL + i), RST_WARPS);
      mbar_init(bar(B_KFREE + i), 1);
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_SFREE + i), 4);
      mbar_init(bar(B_ZFULL + i), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      mbar_init(bar(B_QFREE + i), 1);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(bar(B_IFULL + i), 1);
      mbar_init(bar(B_IFREE + i), 3 + 8 + RST_WARPS);   // every other warp
    }
    mbar_init(bar(B_DRAIN), 1);
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
  auto extent = [&](int b, PagedSeq& s) { return extent_of(a, b, s) && s.n <= a.acc_stride; };
  auto ours = [&](const PagedSeq& s) { return (int64_t)s.nq * wa.G > kStepRows; };
  int64_t total = 0, before = 0, incl = 0, mine = 0;
  auto scan_round = [&](int b0) {
    const int b = b0 + threadIdx.x;
    mine = 0;
    if (b < nseq) {
      PagedSeq s;
      if (extent(b, s))
        mine = ours(s) ? H * weight_units(s, shape) : 0;
      else if (blockIdx.x == 0)
        atomicOr(&g_weights_error, kErrExtent);
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
#pragma unroll 1
  for (int b0 = 0; b0 < nseq; b0 += THREADS) total += scan_round(b0);
  // (a share without an item's beginning has nothing to do)
  const int n_shares = (int)min((int64_t)gridDim.x, max((int64_t)1, total));
  const Shares shares(total, n_shares);
  const bool busy = total > 0 && (int)blockIdx.x < n_shares;
  const int64_t x0 = busy ? shares.first(blockIdx.x) : 0;
  const int64_t x1 = busy ? shares.first(blockIdx.x + 1) : 0;
  if (busy) {
#pragma unroll 1
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int lgb = min(a.cache.lg, 7);      // positions of a page within one key tile: 2^lgb
  auto item_wait = [&](int n) -> bool {
    const bool got = bwait(bar(B_IFULL + n % ITEMS), (uint32_t)((n / ITEMS) & 1), abort_flag);
    return __all_sync(0xFFFFFFFFu, got);
  };
  auto item_done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_IFREE + n % ITEMS));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ codes
    int np = 0, st = 0, turn = 0;                      // parts issued; ring stage, its turn
    bool ok = true;
    const int subs = 128 >> lgb;
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const Item* it = item_slot(n);
      const int b = it->b, hk = it->hk, k0 = it->k0, len = it->n;
      item_done(n);
      if (b < 0) break;
      auto lookup = [&](int e) -> int64_t {
        const int64_t t = (int64_t)k0 + e * kKeyTile + ((int64_t)lane << lgb);
        return lane < subs && t < len ? a.cache.slot(b, t) : -2;
      };
      const int64_t slots[2] = {lookup(0), lookup(1)};
#pragma unroll 1
      for (int e = 0; e < 2; ++e, ++np) {
        const int64_t at = e ? slots[1] : slots[0];
        if (at == -1) atomicOr(&g_weights_error, kErrExtent);
        const unsigned live = __ballot_sync(0xFFFFFFFFu, at >= 0);
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
          const uint32_t dst = smem_u32(smem + L::PART_OFF + st * L::PART) + lane * bytes;
          const uint8_t* src = a.cache.block(at, hk, D);
          if (a.cache.lg <= 7) {
            bulk_copy(dst, src, bytes, bar(B_CFULL + st));
          } else {                                     // a key tile's piece of a longer page
            const int64_t r = at & ((1 << a.cache.lg) - 1);
            bulk_copy(dst, src + r * (D / 2), 128 * (D / 2), bar(B_CFULL + st));
            bulk_copy(dst + 128 * (D / 2), src + ((int64_t)(D / 2) << a.cache.lg) + r * (D / 16),
                      128 * (D / 16), bar(B_CFULL + st));
          }
        }
        if (++st == wa.parts) {
          st = 0;
          ++turn;
        }
      }
    }
    if (lane == 0)
      for (int i = max(0, np - wa.parts); i < np; ++i)
        drain_wait(bar(B_CFULL + i % wa.parts), (uint32_t)((i / wa.parts) & 1));
    __syncwarp();
  } else if (warp == W_MMA) {
    // ------------------------------------------------------------ MMA issuer.  What the products take
    // is the same in every lane, and comes from a shuffle so that it stays in uniform registers.
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0), sbase = smem_u32(smem);
    const uint32_t one = elect_one();
    int q_made = 0, q_base = 0, cnt = 0;               // Q tiles so far; the K/V head's first; S pairs
    bool ok = true;
    auto wait = [&](int b, int parity) {
      ok = ok && __all_sync(0xFFFFFFFFu, bwait(bar(b), (uint32_t)parity, abort_flag));
    };
    auto commit = [&](int b) { umma_commit_if(bar(b), one); };
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const Item it = *item_slot(n);
      item_done(n);
      if (it.b < 0) break;
      const bool resident = it.tiles <= 2;
      if (!it.keep) {
        q_base = q_made;
        if (resident) q_made += it.tiles;
      }
      const int ks[2] = {(2 * n) % KRING, (2 * n + 1) % KRING};
      wait(B_KFULL + ks[0], (2 * n / KRING) & 1);
      wait(B_KFULL + ks[1], (2 * n / KRING) & 1);
#pragma unroll 1
      for (int r = it.r0; r < it.r1 && ok; ++r, ++cnt) {
        const int q = resident ? q_base + r : q_made++;
        wait(B_QFULL + (q & 1), (q >> 1) & 1);
        const int cols = (min(it.nq - r * wa.tpt, wa.tpt) * wa.G + 15) & ~15;
        const uint32_t idesc = __shfl_sync(0xFFFFFFFFu, idesc_qk(cols), 0);
        const uint64_t qd =
            smem_desc(__shfl_sync(0xFFFFFFFFu, sbase + L::Q_OFF + (q & 1) * L::TILE, 0), 16, 1024);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          const int s = 2 * e + (cnt & 1);
          if (cnt >= 2) wait(B_SFREE + s, ((cnt >> 1) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = smem_desc(
              __shfl_sync(0xFFFFFFFFu, sbase + L::K_OFF + (e ? ks[1] : ks[0]) * L::TILE, 0), 16, 1024);
          const uint32_t sd = __shfl_sync(0xFFFFFFFFu, tm + 128 * s, 0);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint64_t off = (uint64_t)(((i >> 2) * BOX + (i & 3) * 32) >> 4);
            umma_f16_if(sd, kd + off, qd + off, idesc, i > 0, one);
          }
          commit(B_SFULL + s);
        }
        if (!resident) commit(B_QFREE + (q & 1));
      }
      if (!ok) break;
      commit(B_KFREE + ks[0]);
      commit(B_KFREE + ks[1]);
      if (resident && !it.keep_next)
        for (int r = 0; r < it.tiles; ++r) {
          // a tile that no item of the share needed has still to land before its buffer is free
          wait(B_QFULL + ((q_base + r) & 1), ((q_base + r) >> 1) & 1);
          commit(B_QFREE + ((q_base + r) & 1));
        }
    }
    commit(B_DRAIN);
    if (one) drain_wait(bar(B_DRAIN), 0u);
    __syncwarp();
  } else if (warp == W_Q) {
    // ------------------------------------------------------------ Q row tiles
    int made = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const Item it = *item_slot(n);
      item_done(n);
      if (it.b < 0) break;
      const bool resident = it.tiles <= 2;
      if (resident && it.keep) continue;
#pragma unroll 1
      for (int r = resident ? 0 : it.r0; r < (resident ? it.tiles : it.r1) && ok; ++r, ++made) {
        if (made >= 2) {
          const bool fr = bwait(bar(B_QFREE + (made & 1)), (uint32_t)(((made >> 1) - 1) & 1),
                                abort_flag);
          if (!__all_sync(0xFFFFFFFFu, fr)) {
            ok = false;
            break;
          }
        }
        if (lane == 0) {
          mbar_expect_tx(bar(B_QFULL + (made & 1)), (uint32_t)(NB * wa.G * wa.tpt * 128));
          for (int c = 0; c < NB; ++c)
            tma_load_3d(smem_u32(smem + L::Q_OFF + (made & 1) * L::TILE + c * BOX), &tmQ, 64 * c,
                        it.hk * wa.G, it.q0 + r * wa.tpt, bar(B_QFULL + (made & 1)));
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      for (int i = max(0, made - 2); i < made; ++i)
        drain_wait(bar(B_QFULL + (i & 1)), (uint32_t)((i >> 1) & 1));
    __syncwarp();
  } else if (warp == W_ITEM) {
    // ------------------------------------------------------------ items
    if (lane == 0) {
      PagedSeq s{0, 0, 0};
      int b = 0, hk = 0, i = 0, items = 0;
      int64_t at = 0;
      bool more = busy;
      auto next_sequence = [&]() {                     // from b on
        for (; b < nseq; ++b)
          if (extent(b, s) && ours(s) && (items = weight_items(s)) > 0) return true;
        return false;
      };
      if (busy) {
        b = first_b;
        more = next_sequence();
        const int64_t per_head = weight_units(s, shape);
        hk = (int)((x0 - first_before) / per_head);
        at = first_before + hk * per_head;
      }
      // the next item that begins in the share
      auto next = [&]() {
        Item it;
        it.b = -1;
        while (more && at < x1) {
          const WeightItem w = weight_item(s, i, shape);
          const bool here = at >= x0;
          if (here) {
            it.b = b;
            it.hk = hk;
            it.q0 = s.q0;
            it.nq = s.nq;
            it.n = s.n;
            it.k0 = w.k0;
            it.r0 = w.t0 / wa.tpt;
            it.r1 = w.t1 > w.t0 ? (w.t1 - 1) / wa.tpt + 1 : it.r0;
            it.tiles = s.nq > 0 ? (s.nq - 1) / wa.tpt + 1 : 0;
          }
          at += weight_cost(w, shape);
          if (++i == items) {
            i = 0;
            if (++hk == H) {
              hk = 0;
              ++b;
              more = next_sequence();
            }
          }
          if (here) break;
        }
        return it;
      };
      Item cur = next();
      cur.keep = 0;
      for (int n = 0;; ++n) {
        Item nx;
        nx.b = -1;
        if (cur.b >= 0) nx = next();
        nx.keep = nx.b >= 0 && nx.b == cur.b && nx.hk == cur.hk && nx.tiles <= 2;
        cur.keep_next = nx.keep;
        if (n >= ITEMS &&
            !bwait(bar(B_IFREE + n % ITEMS), (uint32_t)((n / ITEMS - 1) & 1), abort_flag))
          break;
        *item_slot(n) = cur;
        mbar_arrive(bar(B_IFULL + n % ITEMS));
        if (cur.b < 0) break;
        cur = nx;
      }
    }
    __syncwarp();
  } else if (warp >= W_RST) {
    // ------------------------------------------------------------ restore
    const int tid = threadIdx.x - W_RST * 32;
    int np = 0, st = 0, turn = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!item_wait(n)) break;
      const Item* it = item_slot(n);
      const int b = it->b, k0 = it->k0, len = it->n;
      item_done(n);
      if (b < 0) break;
#pragma unroll 1
      for (int e = 0; e < 2; ++e, ++np) {
        const int ks = np % KRING;
        bool got = bwait(bar(B_CFULL + st), (uint32_t)(turn & 1), abort_flag);
        if (np >= KRING)
          got = got && bwait(bar(B_KFREE + ks), (uint32_t)((np / KRING - 1) & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        restore_k<D>(smem_u32(smem + L::PART_OFF + st * L::PART),
                     smem_u32(smem + L::K_OFF + ks * L::TILE), lgb, len - k0 - e * kKeyTile, tid);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_CFREE + st));
          mbar_arrive(bar(B_KFULL + ks));
        }
        if (++st == wa.parts) {
          st = 0;
          ++turn;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int e = (warp - W_EXP) >> 2, quarter = warp & 3;
    const int m = 32 * quarter + lane;                 // the thread's position in its key tile, and
                                                       // the row whose log-sum-exp it fetches
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16);
    float* lse = lse_buf + e * 256;
    const int tok = m / wa.G, gh = m - tok * wa.G;
    const uint64_t sl2x2 = f2pack(wa.scale_log2, wa.scale_log2);
    int cnt = 0;                                       // row tiles
    // The log-sum-exp of row m of row tile r of an item: -inf for columns of no row.
    auto fetch = [&](const Item& it, int r) -> float {
      const int i = r * wa.tpt + tok;
      if (r >= it.r1 || tok >= wa.tpt || i >= it.nq) return -INFINITY;
      return a.lse_in[(int64_t)(it.q0 + i) * a.Hq + it.hk * wa.G + gh];
    };
    auto weight_at = [&](const Item& it) {
      return ((int64_t)it.b * H + it.hk) * a.acc_stride + it.k0 + e * kKeyTile + m;
    };
    auto fetch_old = [&](const Item& it) -> float {
      return a.acc && it.k0 + e * kKeyTile + m < it.n ? a.acc[weight_at(it)] : 0.0f;
    };
    float z_next = -INFINITY, old_next = 0.0f;         // of the next item, in flight
    bool ok = item_wait(0);
    if (ok && item_slot(0)->b >= 0) {
      z_next = fetch(*item_slot(0), item_slot(0)->r0);
      old_next = fetch_old(*item_slot(0));
    }
    for (int n = 0; ok; ++n) {
      const Item& it = *item_slot(n);                  // read where needed: no registers for it
      if (it.b < 0) break;
      const int t = it.k0 + e * kKeyTile + m;          // the thread's position
      const bool live = t < it.n;
      float z = z_next;
      const float old = old_next;
      if (!item_wait(n + 1)) break;
      const Item& nx = *item_slot(n + 1);
      if (nx.b >= 0) {
        z_next = fetch(nx, nx.r0);
        old_next = fetch_old(nx);
      }
      uint64_t sum2[2] = {f2pack(0.0f, 0.0f), f2pack(0.0f, 0.0f)};
#pragma unroll 1
      for (int r = it.r0; r < it.r1; ++r, ++cnt) {
        const int s = cnt & 1;
        // (the buffer's last readers have arrived at the other buffer's barrier since)
        // (-lse / ln 2; for a row of -inf, which adds nothing, a number that leaves 0 of finite scores)
        lse[128 * s + m] = z == -INFINITY ? kSilent : z * -1.4426950408889634f;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_ZFULL + 2 * e + s));
        z = fetch(it, r + 1);                          // in flight meanwhile
        // columns c0 .. c1 - 1 are rows that see the position
        const int ntok = min(it.nq - r * wa.tpt, wa.tpt), pos0 = it.n - it.nq + r * wa.tpt;
        const int64_t first = (int64_t)t - pos0;
        int64_t last = ntok;
        if (a.window != 0 && t >= a.sinks) last = min(last, (int64_t)t + a.window - pos0);
        const int c0 = (int)max((int64_t)0, min(first, (int64_t)ntok)) * wa.G;
        const int c1 = live ? (int)max((int64_t)0, last) * wa.G : 0;
        bool got = bwait(bar(B_ZFULL + 2 * e + s), (uint32_t)((cnt >> 1) & 1), abort_flag);
        got = got && bwait(bar(B_SFULL + 2 * e + s), (uint32_t)((cnt >> 1) & 1), abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t srow = lane_addr + 128 * (2 * e + s);
        const float* zr = lse + 128 * s;
        auto chunk = [&](const float (&v)[32], int c, auto columns) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 z4 = *reinterpret_cast<const float4*>(zr + 32 * c + i);
            const float2 x = f2unpack(ffma2(f2pack(v[i], v[i + 1]), sl2x2, f2pack(z4.x, z4.y)));
            const float2 y = f2unpack(ffma2(f2pack(v[i + 2], v[i + 3]), sl2x2, f2pack(z4.z, z4.w)));
            float p[4] = {ex2(x.x), ex2(x.y), ex2(y.x), ex2(y.y)};
            if (decltype(columns)::value == kHeard) {
              p[0] = z4.x != kSilent ? p[0] : 0.0f;
              p[1] = z4.y != kSilent ? p[1] : 0.0f;
              p[2] = z4.z != kSilent ? p[2] : 0.0f;
              p[3] = z4.w != kSilent ? p[3] : 0.0f;
            }
            if (decltype(columns)::value != kAll) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int col = 32 * c + i + k;
                p[k] = col >= c0 && col < c1 ? p[k] : 0.0f;
              }
            }
            sum2[0] = fadd2(sum2[0], f2pack(p[0], p[1]));
            sum2[1] = fadd2(sum2[1], f2pack(p[2], p[3]));
          }
        };
        float va[32], vb[32];
        const uint64_t before[2] = {sum2[0], sum2[1]};
        auto some = [&](auto columns) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (!__any_sync(0xFFFFFFFFu, c0 < 32 * c + 32 && c1 > 32 * c && c1 > c0)) continue;
            tmem_ld32(srow + 32 * c, va);
            tmem_wait_ld_dep(va);
            chunk(va, c, columns);
          }
        };
        if (__all_sync(0xFFFFFFFFu, c0 == 0 && c1 == 128)) {
          tmem_ld32(srow, va);
          tmem_wait_ld_dep(va);
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {             // the next load in flight
            tmem_ld32(srow + 32 * c + 32, vb);
            chunk(va, c, Columns<kAll>{});
            tmem_wait_ld_dep(vb);
            if (c == 0) tmem_ld32(srow + 64, va);
            chunk(vb, c + 1, Columns<kAll>{});
            tmem_wait_ld_dep(va);
          }
        } else {
          some(Columns<kSome>{});
        }
        // an infinity or NaN in Q or K: again, without what rows of -inf made of it
        const float2 now = f2unpack(fadd2(sum2[0], sum2[1]));
        if (__any_sync(0xFFFFFFFFu, !(now.x + now.y < INFINITY))) {
          sum2[0] = before[0];
          sum2[1] = before[1];
          some(Columns<kHeard>{});
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SFREE + 2 * e + s));
      }
      if (!ok) break;
      const float2 su = f2unpack(fadd2(sum2[0], sum2[1]));
      if (live) a.acc_out[weight_at(it)] = old + (su.x + su.y);
      item_done(n);
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
  e = cudaFuncSetAttribute(weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           L::bytes(L::depth()));
  done[dev] = e == cudaSuccess;
  return e;
}

template <int D>
cudaError_t launch_d(const PagedAttn& a, int nsm, cudaStream_t st) {
  using L = Smem<D>;
  cudaError_t e = prepare<D>();
  if (e != cudaSuccess || (e = get_encode()) != cudaSuccess) return e;
  WArgs wa;
  wa.a = a;
  wa.scale_log2 = a.scale * 1.4426950408889634f;
  wa.G = a.Hq / a.cache.H;
  wa.tpt = 128 / wa.G;
  wa.parts = L::depth();
  CUtensorMap tq{};                        // without rows no tile is loaded
  if (a.q_rows > 0) {
    e = make_map_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q, D, (uint64_t)a.Hq,
                    (uint64_t)a.q_rows, 2 * D, (uint64_t)a.q_stride * 2, 64, wa.G,
                    CU_TENSOR_MAP_SWIZZLE_128B, wa.tpt);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(weights_kernel<D>, dim3(std::max(nsm, 1)), dim3(THREADS), L::bytes(wa.parts), st,
                    tq, wa);
}

}  // namespace

// Sequences with few query rows go to the streaming kernel, the others here; a call whose rows are
// known to be few launches that alone.  (One token of 32 sequences of 2000 .. 4096 positions, 8 K/V
// heads: 36 us there with 1 to 8 query heads each and 50 us with 32, 72 us here with any.)
cudaError_t launch_attn_weights_paged(const PagedAttn& a, int d, int nsm, cudaStream_t st) {
  const cudaError_t e = launch_attn_weights_step(a, d, nsm, st);
  if (e != cudaSuccess || (int64_t)a.max_q * (a.Hq / a.cache.H) <= kStepRows) return e;
  return d == 128 ? launch_d<128>(a, nsm, st) : launch_d<64>(a, nsm, st);
}

cudaError_t weights_read_error(unsigned int* out) { return read_and_clear(g_weights_error, out); }

}  // namespace fg
