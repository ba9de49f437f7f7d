// The softmax weights that positions of the paged 4-bit cache receive, for sequences with few query
// rows (at most kStepRows rows of a K/V head's query heads): a stream over the K codes and statistics
// (sm_103a).  attn_weights_paged.cu has the sequences with more.
//
// The sums are those of that file: acc + sum exp(scale q . k^ - lse), with K^ = fp16(a + q (b - a) /
// 15) exactly as defined, so they are restored before the products, in registers: mma.sync m16n8k16 with
// 16 positions in its rows and 8 query rows in its columns.  A lane (gid, tig) holds 32 (d = 64: 16)
// channels of positions gid and gid + 8, as the codes lie; the products' index order follows, and
// Q's fragments are laid out for it in shared memory once per (sequence, K/V head).
//
// Work: blocks of 256 positions of one K/V head in one order, cut evenly among the CTAs; a warp takes
// 32 positions of a block, and copies those of the next one into shared memory meanwhile.
// Bound by instructions: 25 for every 8 codes of exact restoring are 400 of the 1150 that a warp takes
// for 32 positions of 128 channels, the turns, copies and sums around them the rest; then by HBM
// (0.5625 d bytes a position).  One token of 32 sequences of 2000 .. 4096 positions, 8 K/V heads, 4
// query heads each, 62 MB: 36 us, 1.7 TB/s (39 us with the codes loaded into registers as they are
// needed; 37 us with two CTAs per SM; 40 us with a warp's two tiles in code of their own).
#include <math.h>

#include <algorithm>

#include "attn_q4.cuh"
#include "paged_tc.cuh"
#include "q4_restore.cuh"

namespace fg {

__device__ unsigned int g_weights_step_error = 0;

namespace {

using q4attn::mma16816;

constexpr int kThreads = 256, kWarps = kThreads / 32, kCtasPerSm = 3;
constexpr int kBlock = kWarps * 32;        // positions
constexpr int kSets = kStepRows / 8;       // columns of 8 query rows

struct SArgs {
  PagedAttn a;
  float scale_log2;
  int G;
};

// (a called function: groups with infinities or NaN are rare)
__device__ __noinline__ uint4 restore8_any(uint32_t codes, uint32_t abw) {
  return restore8_fp16(codes, abw);
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t addr, uint32_t (&w)[N]) {
  static_assert(N == 2 || N == 4, "words of a lane");
  if constexpr (N == 4) {
    const uint4 v = paged::ld_shared_v4(addr);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) weights_step_kernel(const SArgs sa) {
  constexpr int NW = D / 32;               // code words of a position in a lane
  __shared__ uint4 qf[kSets * NW * 32];    // [set][word][lane]: 8 channels of query row 8 set + gid
  // -lse / ln 2 of the query rows; +inf: no row, or one that adds nothing
  __shared__ __align__(8) float zs[kStepRows];
  // two blocks of the warps' 32 positions: codes, then statistics
  constexpr int CODES = 16 * (D / 2), STATS = 16 * (D / 16);      // bytes of 16 positions
  __shared__ __align__(16) uint8_t stage[2][kWarps][2 * (CODES + STATS)];
  __shared__ int64_t warp_units[kWarps];
  __shared__ int first_b;
  __shared__ int64_t first_before;
  pdl_launch_dependents();
  pdl_wait();
  const PagedAttn& a = sa.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int nseq = a.cache.B, H = a.cache.H, G = sa.G;
  auto extent = [&](int b, PagedSeq& s) {
    return paged::extent_of(a, b, s) && s.n <= a.acc_stride && (int64_t)s.nq * G <= kStepRows;
  };
  auto blocks_of = [&](const PagedSeq& s) { return (int)(((int64_t)s.n + kBlock - 1) / kBlock); };

  // ---- the order of the work, and where this CTA's begins
  int64_t total = 0, before = 0, incl = 0, mine = 0;
  auto scan_round = [&](int b0) {
    const int b = b0 + threadIdx.x;
    PagedSeq s;
    mine = b < nseq && extent(b, s) ? (int64_t)H * blocks_of(s) : 0;
    if (blockIdx.x == 0 && b < nseq && (!paged::extent_of(a, b, s) || s.n > a.acc_stride))
      atomicOr(&g_weights_step_error, kErrExtent);
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_units[warp] = incl;
    __syncthreads();
    int64_t round = 0;
    for (int i = 0; i < kWarps; ++i) {
      const int64_t n = warp_units[i];
      if (i < warp) incl += n;
      round += n;
    }
    __syncthreads();
    return round;
  };
#pragma unroll 1
  for (int b0 = 0; b0 < nseq; b0 += kThreads) total += scan_round(b0);
  const int n_shares = (int)min((int64_t)gridDim.x, max((int64_t)1, total));
  if (total == 0 || (int)blockIdx.x >= n_shares) return;
  const Shares shares(total, n_shares);
  int64_t x = shares.first(blockIdx.x);
  const int64_t x1 = shares.first(blockIdx.x + 1);
#pragma unroll 1
  for (int b0 = 0; b0 < nseq; b0 += kThreads) {
    const int64_t round = nseq > kThreads ? scan_round(b0) : total;
    if (before + round > x) {
      if (before + incl > x && before + incl - mine <= x) {
        first_b = b0 + threadIdx.x;
        first_before = before + incl - mine;
      }
      break;
    }
    before += round;
  }
  __syncthreads();

  // ---- the blocks: `cur`, computed on; the one behind it, its codes in flight; and `ahead`, two
  // behind it, its page table entries in flight
  struct Cursor {
    PagedSeq s;
    int b, hk, i, blocks;
  };
  auto advance = [&](Cursor& c) {          // true: another (sequence, head)
    if (++c.i < c.blocks) return false;
    c.i = 0;
    if (++c.hk == H) {
      c.hk = 0;
      c.blocks = 0;
      while (c.blocks == 0 && ++c.b < nseq) c.blocks = extent(c.b, c.s) ? blocks_of(c.s) : 0;
    }
    return true;
  };
  // lanes 0, 1: the slots of the warp's two tiles of 16 (-1: a bad page; -2: behind the sequence)
  auto lookup = [&](const Cursor& c) -> int64_t {
    const int64_t p = (int64_t)c.i * kBlock + warp * 32 + lane * 16;
    return lane < 2 && p < c.s.n ? a.cache.slot(c.b, p) : -2;
  };
  // the tiles' codes and statistics, 16 bytes a lane and turn
  auto fetch = [&](int64_t slot, int head, int buf) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t sl = __shfl_sync(0xFFFFFFFFu, slot, t);
      if (sl >= 0) {
        const uint8_t* k = a.cache.block(sl, head, D);
        const int64_t at = sl & ((1 << a.cache.lg) - 1);
        const uint8_t* ab = k + ((int64_t)(D / 2) << a.cache.lg) + at * (D / 16);
        const uint32_t to = smem_u32(stage[buf][warp]) + t * CODES;
        k += at * (D / 2);
#pragma unroll
        for (int u = 0; u < CODES; u += 512) copy16(to + u + 16 * lane, k + u + 16 * lane);
        if (lane < STATS / 16)
          copy16(smem_u32(stage[buf][warp]) + 2 * CODES + t * STATS + 16 * lane, ab + 16 * lane);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Cursor cur;
  cur.b = first_b;
  extent(cur.b, cur.s);
  cur.blocks = blocks_of(cur.s);
  cur.hk = (int)((x - first_before) / cur.blocks);
  cur.i = (int)(x - first_before - (int64_t)cur.hk * cur.blocks);
  Cursor ahead = cur;
  int64_t slot = lookup(ahead);
  if (lane < 2 && slot == -1) atomicOr(&g_weights_step_error, kErrExtent);
  unsigned here = __ballot_sync(0xFFFFFFFFu, slot >= 0);           // tiles of `cur` that are there
  fetch(slot, ahead.hk, 0);
  int head1 = 0;                           // the next block's head
  if (x + 1 < x1) {
    advance(ahead);
    slot = lookup(ahead);
    head1 = ahead.hk;
  }
  bool fresh = true;                       // Q of another (sequence, head) than before
  int buf = 0;
#pragma unroll 1
  for (; x < x1; ++x, buf ^= 1) {
    const int p0 = cur.i * kBlock + warp * 32, b = cur.b, hk = cur.hk;
    const PagedSeq s = cur.s;
    unsigned there = 0;                    // the next block's tiles
    if (x + 1 < x1) {
      if (lane < 2 && slot == -1) atomicOr(&g_weights_step_error, kErrExtent);
      there = __ballot_sync(0xFFFFFFFFu, slot >= 0);
      fetch(slot, head1, buf ^ 1);
      if (x + 2 < x1) {
        advance(ahead);
        slot = lookup(ahead);
        head1 = ahead.hk;
      }
    }
    if (fresh) {
      // Q of the K/V head's rows: row r is token r / G, head r % G
      __syncthreads();
      const int rows = s.nq * G;
      for (int u = threadIdx.x; u < kSets * NW * 32; u += kThreads) {
        const int l = u & 31, w = (u >> 5) % NW, row = 8 * (u / (32 * NW)) + (l >> 2);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows)
          v = *reinterpret_cast<const uint4*>(a.q + (int64_t)(s.q0 + row / G) * a.q_stride +
                                              (int64_t)(hk * G + row % G) * D +
                                              (l & 3) * (8 * NW) + 8 * w);
        qf[u] = v;
      }
      if (threadIdx.x < kStepRows) {
        const int row = threadIdx.x;
        float z = -INFINITY;
        if (row < rows) z = a.lse_in[(int64_t)(s.q0 + row / G) * a.Hq + hk * G + row % G];
        zs[row] = z * -1.4426950408889634f;
      }
      __syncthreads();
    }
    const int nq = s.nq, n = s.n;
    const int rows = nq * G, pos0 = n - nq;
    if (x + 1 < x1)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // ---- products and sums
    // every row sees all of the warp's positions
    const bool all_see = a.window == 0 && p0 + 31 <= pos0;
    // (a loop, so that its instructions stay near)
    const int64_t out0 = ((int64_t)b * H + hk) * a.acc_stride + p0 + gid;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      float sum[2] = {}, old[2];           // what positions gid and gid + 8 receive, and received
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int o = 16 * t + 8 * r;
        old[r] = tig == 0 && a.acc && p0 + gid + o < n ? a.acc[out0 + o] : 0.0f;
      }
      if (here >> t & 1u) {
        uint4 k0[NW], k1[NW];
        const uint32_t codes = smem_u32(stage[buf][warp]) + t * CODES + gid * (D / 2) + tig * (4 * NW);
        const uint32_t stats = smem_u32(stage[buf][warp]) + 2 * CODES + t * STATS + gid * (D / 16) +
                               (D == 128 ? 4 * (tig >> 1) : 0);
        uint32_t w0[NW], w1[NW];
        load_words<NW>(codes, w0);
        load_words<NW>(codes + 8 * (D / 2), w1);
        const uint32_t ab0 = paged::ld_shared(stats), ab1 = paged::ld_shared(stats + 8 * (D / 16));
        const GroupFp16 g0(ab0), g1(ab1);
        if (__all_sync(0xFFFFFFFFu, g0.plain && g1.plain)) {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            k0[w] = g0.restore(w0[w]);
            k1[w] = g1.restore(w1[w]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            k0[w] = restore8_any(w0[w], ab0);
            k1[w] = restore8_any(w1[w], ab1);
          }
        }
        const int tp = p0 + 16 * t + gid;    // the lane's positions: tp and tp + 8
#pragma unroll 1
        for (int set = 0; 8 * set < rows; ++set) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const uint4 q = qf[(set * NW + w) * 32 + lane];
            mma16816(c, k0[w].x, k1[w].x, k0[w].y, k1[w].y, q.x, q.y);
            mma16816(c, k0[w].z, k1[w].z, k0[w].w, k1[w].w, q.z, q.w);
          }
          // c[2 r + e]: position tp + 8 r, query row 8 set + 2 tig + e
          const float2 z = *reinterpret_cast<const float2*>(zs + 8 * set + 2 * tig);
          if (all_see) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float y0 = ex2(fmaf(c[2 * r], sa.scale_log2, z.x));
              const float y1 = ex2(fmaf(c[2 * r + 1], sa.scale_log2, z.y));
              sum[r] += (z.x != INFINITY ? y0 : 0.0f) + (z.y != INFINITY ? y1 : 0.0f);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = 8 * set + 2 * tig + e, pos = pos0 + row / G;
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if ((e ? z.y : z.x) != INFINITY && visible(tp + 8 * r, pos, a.window, a.sinks))
                  sum[r] += ex2(fmaf(c[2 * r + e], sa.scale_log2, e ? z.y : z.x));
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = sum[r];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        const int o = 16 * t + 8 * r;
        if (tig == 0 && p0 + gid + o < n) a.acc_out[out0 + o] = old[r] + v;
      }
    }
    here = there;
    fresh = x + 1 < x1 && advance(cur);
    __syncwarp();                          // the stage is read; the turn after next copies into it
  }
}

}  // namespace

cudaError_t launch_attn_weights_step(const PagedAttn& a, int d, int nsm, cudaStream_t st) {
  const SArgs sa{a, a.scale * 1.4426950408889634f, a.Hq / a.cache.H};
  const dim3 grid((unsigned)std::max(1, nsm) * kCtasPerSm);
  return launch_pdl(d == 128 ? weights_step_kernel<128> : weights_step_kernel<64>, grid,
                    dim3(kThreads), 0, st, sa);
}

cudaError_t weights_step_read_error(unsigned int* out) {
  return read_and_clear(g_weights_step_error, out);
}

}  // namespace fg
