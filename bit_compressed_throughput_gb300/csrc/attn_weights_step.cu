// The softmax weights that positions of the paged 4-bit cache receive, for sequences with few query
// rows (at most kStepRows rows of a K/V head's query heads): a stream over the K codes and statistics
// (sm_103a).  attn_weights_paged.cu has the sequences with more.
//
// The sums are those of that file: acc + sum exp(scale q . k^ - lse), with K^ = fp16(a + q (b - a) / 15)
// exactly as defined, so they are restored before the products, in registers: mma.sync m16n8k16 with
// 16 positions in its rows and 8 query rows in its columns.  A lane (gid, tig) holds 32 (d = 64: 16)
// channels of positions gid and gid + 8, as the codes lie; the products' index order follows, and
// Q's fragments are laid out for it in shared memory once per (sequence, K/V head).
//
// Work: blocks of 256 positions of one K/V head in one order, cut evenly among the CTAs; a warp takes
// 32 positions of a block.  Bound by HBM (0.5625 d bytes a position) and by the restoring's
// instructions, about 25 per 8 codes.
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

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) weights_step_kernel(const SArgs sa) {
  constexpr int NW = D / 32;               // code words of a position in a lane
  __shared__ uint4 qf[kSets * NW * 32];    // [set][word][lane]: 8 channels of query row 8 set + gid
  __shared__ __align__(8) float zs[kStepRows];          // -lse / ln 2; -inf: no row, or one that sees nothing
  __shared__ int64_t warp_units[kWarps];
  __shared__ int first_b;
  __shared__ int64_t first_before;
  pdl_launch_dependents();
  pdl_wait();
  const PagedAttn& a = sa.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int nseq = a.cache.B, H = a.cache.H, G = sa.G;
  auto extent = [&](int b, PagedSeq& s) {
    return paged::extent_of(a, b, s) && s.n <= a.acc_stride && s.nq * G <= kStepRows;
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

  // ---- the blocks
  int b = first_b;
  PagedSeq s;
  extent(b, s);
  int blocks = blocks_of(s);
  int hk = (int)((x - first_before) / blocks);
  int i = (int)(x - first_before - (int64_t)hk * blocks);
  bool fresh = true;                       // Q of another (sequence, head) than before
  // the slot of the warp's tile `tile` of block i (-1: a bad page; -2: behind the sequence)
  auto slot_of = [&](int tile) -> int64_t {
    const int64_t p = (int64_t)i * kBlock + warp * 32 + tile * 16;
    return p < s.n ? a.cache.slot(b, p) : -2;
  };
  int64_t slot = lane < 2 ? slot_of(lane) : -2;
#pragma unroll 1
  for (; x < x1; ++x) {
    const int p0 = i * kBlock + warp * 32;
    const int64_t sl[2] = {__shfl_sync(0xFFFFFFFFu, slot, 0), __shfl_sync(0xFFFFFFFFu, slot, 1)};
    if (lane == 0 && (sl[0] == -1 || sl[1] == -1)) atomicOr(&g_weights_step_error, kErrExtent);
    // codes and statistics of the lane's four positions, and what they received before
    uint4 kw[2][2];
    uint32_t ab[2][2];
    float old[2][2];
    const int64_t out0 = ((int64_t)b * H + hk) * a.acc_stride + p0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gid + 8 * r;
        kw[t][r] = make_uint4(0, 0, 0, 0);
        ab[t][r] = 0u;
        old[t][r] = 0.0f;
        if (sl[t] < 0) continue;
        const uint8_t* k = a.cache.block(sl[t], hk, D);
        const int64_t at = (sl[t] & ((1 << a.cache.lg) - 1)) + row;
        const uint8_t* c = k + at * (D / 2) + tig * (4 * NW);
        if constexpr (D == 128) {
          kw[t][r] = ldg_nc_v4(c);
        } else {
          const uint2 u = __ldg(reinterpret_cast<const uint2*>(c));
          kw[t][r] = make_uint4(u.x, u.y, 0, 0);
        }
        ab[t][r] = __ldg(reinterpret_cast<const uint32_t*>(k + ((int64_t)(D / 2) << a.cache.lg)) +
                         at * (D / 64) + (D == 128 ? tig >> 1 : 0));
        if (tig == 0 && a.acc && p0 + 16 * t + row < s.n) old[t][r] = a.acc[out0 + 16 * t + row];
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
        zs[row] = z == -INFINITY ? z : z * -1.4426950408889634f;
      }
      __syncthreads();
    }
    // the next block, and the page table's answer for it in flight
    const int nq = s.nq, n = s.n;
    const int rows = nq * G, pos0 = n - nq;
    fresh = false;
    if (++i == blocks) {
      i = 0;
      fresh = true;
      if (++hk == H) {
        hk = 0;
        blocks = 0;
        while (blocks == 0 && ++b < nseq) blocks = extent(b, s) ? blocks_of(s) : 0;
      }
    }
    if (x + 1 < x1) slot = lane < 2 ? slot_of(lane) : -2;
    // ---- products and sums
    float sum[2][2] = {};
    // every row sees all of the warp's positions
    const bool all_see = a.window == 0 && p0 + 31 <= pos0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (sl[t] < 0) continue;
      uint4 k0[NW], k1[NW];
      const uint32_t w0[4] = {kw[t][0].x, kw[t][0].y, kw[t][0].z, kw[t][0].w};
      const uint32_t w1[4] = {kw[t][1].x, kw[t][1].y, kw[t][1].z, kw[t][1].w};
      const GroupFp16 g0(ab[t][0]), g1(ab[t][1]);
      if (__all_sync(0xFFFFFFFFu, g0.plain && g1.plain)) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          k0[w] = g0.restore(w0[w]);
          k1[w] = g1.restore(w1[w]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          k0[w] = restore8_any(w0[w], ab[t][0]);
          k1[w] = restore8_any(w1[w], ab[t][1]);
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
            sum[t][r] += (8 * set + 2 * tig < rows ? y0 : 0.0f) +
                         (8 * set + 2 * tig + 1 < rows ? y1 : 0.0f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * set + 2 * tig + e, pos = pos0 + row / G;
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (row < rows && visible(tp + 8 * r, pos, a.window, a.sinks))
                sum[t][r] += ex2(fmaf(c[2 * r + e], sa.scale_log2, e ? z.y : z.x));
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = sum[t][r];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        const int o = 16 * t + 8 * r + gid;
        if (tig == 0 && p0 + o < n) a.acc_out[out0 + o] = old[t][r] + v;
      }
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
