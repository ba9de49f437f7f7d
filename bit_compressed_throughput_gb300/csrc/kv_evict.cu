// Smaller caches: every K/V head of a sequence keeps its newest positions and the heaviest of the
// others, moved in order into pages of their own (sm_103a).
//
// Selection, a CTA per (sequence, head), or four that share its positions where such pairs are few and
// long (they add up their counts through one another's shared memory): the weights' order keys are
// 32-bit numbers, and three passes over them, histograms of 11, 11 and 10 bits, find the key of the
// last one that stays and how many equal ones do.  (11 bits of a weight are its exponent and two bits
// more, so that the threads of a warp rarely meet in one bin.)  Then every warp counts what stays of
// its part of the positions, and lists it behind what the warps before it have.  Ties go to the lower
// position.
// Moving: a position's K and V codes and statistics, copied as they are, 16 bytes a thread.
// Bound by HBM: the weights once, 2 * 1.125 d bytes per kept position; by latency where a call has few
// (sequence, head) pairs.  16 sequences of 2000 .. 4096 positions cut to 1024, 8 heads, 38 MB of
// positions read and written: 16 us; 4 of 20,001 .. 32,001 cut to 8192, 75 MB: 43 us.  (The weights
// held in shared memory between the passes: 58 us against 52 at that stage.)
#include <algorithm>

#include "attn_q4.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "gemm_tc.cuh"
#include "paged.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_evict_error = 0;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

constexpr int kBins = 2048;

constexpr int kShare = 4;                  // CTAs of a pair of its own

// Keys of equal weights are equal: -0 takes +0's, and every NaN the largest.
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t k = q4attn::order_key_f32(w);
  return isnan(w) ? 0xFFFFFFFFu : (k == 0x7FFFFFFFu ? 0x80000000u : k);
}
// A word of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}

template <int CL>
__global__ void __launch_bounds__(kThreads) select_kernel(const Evict a) {
  __shared__ int hist[kBins];
  __shared__ int2 warp_counts[kWarps];
  __shared__ int2 totals;                  // of the CTA's positions: that stay for sure, equal ones
  __shared__ int found[2];
  const int rank = CL == 1 ? 0 : (int)cluster_ctarank();
  auto together = [&]() {                  // all threads of the pair's CTAs
    if (CL == 1) __syncthreads(); else cluster_sync_all();
  };
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x / CL, b = blockIdx.y, H = a.src.H;
  int n = a.lens[b];
  if (n < 0 || n > a.src.cap() || n > a.acc_stride) {
    if (threadIdx.x == 0) atomicOr(&g_evict_error, kErrExtent);
    n = 0;
  }
  const int64_t row = (int64_t)b * H + head;
  const float* acc = a.acc + row * a.acc_stride;
  int32_t* kept = a.kept + row * a.keep;
  float* acc_out = a.acc_out + row * a.keep;
  const int left = min(n, a.keep);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.dst_lens[b] = left;
  for (int i = left + rank * kThreads + threadIdx.x; i < a.keep; i += CL * kThreads) {
    kept[i] = -1;
    acc_out[i] = 0.0f;
  }
  if (n <= a.keep) {
    for (int i = rank * kThreads + threadIdx.x; i < n; i += CL * kThreads) {
      kept[i] = i;
      acc_out[i] = acc[i];
    }
    return;
  }
  const int old = n - a.recent;            // recent <= keep < n
  int want = a.keep - a.recent;            // of the first `old`
  const bool none = want == 0;
  // the CTA's positions
  const int share = ((n + CL - 1) / CL + 31) & ~31;
  const int n0 = min(n, rank * share), n1 = min(n, n0 + share);
  // the key of the want-th largest: bits 21 and up, 10 .. 20, 0 .. 9
  uint32_t prefix = 0;
  if (!none) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const int above = pass == 0 ? 32 : (pass == 1 ? 21 : 10);      // bits that are settled
      for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 8
      for (int i = n0 + threadIdx.x; i < min(n1, old); i += kThreads) {
        const uint32_t k = key_of(acc[i]);
        if (pass == 0 || (k >> above) == prefix) atomicAdd(&hist[k >> shift & mask], 1);
      }
      together();
      // bins from the top, two a thread: the one in which the want-th falls
      const int b1 = (int)mask - 2 * (int)threadIdx.x, b0 = b1 - 1;
      int c1 = 0, c0 = 0;
#pragma unroll
      for (int r = 0; r < CL; ++r) {
        if (b1 >= 0) c1 += CL == 1 ? hist[b1] : ld_cluster(&hist[b1], r);
        if (b0 >= 0) c0 += CL == 1 ? hist[b0] : ld_cluster(&hist[b0], r);
      }
      int incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) warp_counts[warp].x = incl;
      __syncthreads();
      int before = incl - c0 - c1;
      for (int i = 0; i < warp; ++i) before += warp_counts[i].x;
      if (before < want && before + c1 >= want) {
        found[0] = b1;
        found[1] = before;
      } else if (before + c1 < want && before + c1 + c0 >= want) {
        found[0] = b0;
        found[1] = before + c1;
      }
      together();                          // (the counts are read by others, too)
      prefix = prefix << (pass == 0 ? 0 : (pass == 1 ? 11 : 10)) | (uint32_t)found[0];
      want -= found[1];
    }
  }
  // larger keys stay, and the first `want` equal ones; a warp has positions i0 .. i1 - 1
  const int per = ((share + kWarps - 1) / kWarps + 31) & ~31;
  const int i0 = min(n1, n0 + warp * per), i1 = min(n1, i0 + per);
  int2 cnt = make_int2(0, 0);              // that stay for sure; equal ones
#pragma unroll 4
  for (int base = i0; base < i1; base += 32) {         // the same turns for every lane
    const int i = base + lane;
    const uint32_t k = i < old && i < i1 && !none ? key_of(acc[i]) : 0u;
    const bool sure = i < i1 && (i >= old || (!none && k > prefix));
    const bool same = i < i1 && i < old && !none && k == prefix;
    cnt.x += __popc(__ballot_sync(0xFFFFFFFFu, sure));
    cnt.y += __popc(__ballot_sync(0xFFFFFFFFu, same));
  }
  __syncthreads();
  if (lane == 0) warp_counts[warp] = cnt;
  __syncthreads();
  int sure_before = 0, equal = 0;
  for (int i = 0; i < warp; ++i) {
    sure_before += warp_counts[i].x;
    equal += warp_counts[i].y;
  }
  if (CL > 1) {
    if (threadIdx.x == kThreads - 1)
      totals = make_int2(sure_before + cnt.x, equal + cnt.y);
    together();
    for (int r = 0; r < rank; ++r) {
      sure_before += ld_cluster(&totals.x, r);
      equal += ld_cluster(&totals.y, r);
    }
  }
  int at = sure_before + min(equal, want);
#pragma unroll 4
  for (int base = i0; base < i1; base += 32) {         // the same turns for every lane
    const int i = base + lane;
    const float w = i < i1 ? acc[i] : 0.0f;
    const uint32_t k = key_of(w);
    const bool sure = i < i1 && (i >= old || (!none && k > prefix));
    const bool same = i < i1 && i < old && !none && k == prefix;
    const unsigned eq = __ballot_sync(0xFFFFFFFFu, same), below = (1u << lane) - 1u;
    const bool stays = sure || (same && equal + __popc(eq & below) < want);
    const unsigned st = __ballot_sync(0xFFFFFFFFu, stays);
    if (stays) {
      kept[at + __popc(st & below)] = i;
      acc_out[at + __popc(st & below)] = w;
    }
    at += __popc(st);
    equal += __popc(eq);
  }
  if (CL > 1) together();                  // others may still read this CTA's totals
}

// 16 bytes of codes a thread (2 * D / 32 threads a position: K, then V), and a statistics word of it
// each; kMoves positions in flight.
constexpr int kMoves = 4;
template <int D>
__global__ void __launch_bounds__(256) move_kernel(const Evict a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int TPP = D / 16, PER = 256 / TPP;           // threads per position, positions a turn
  const int u = threadIdx.x % TPP, which = u / (TPP / 2), c = u % (TPP / 2);
  const int head = blockIdx.y, b = blockIdx.z, H = a.src.H;
  const int64_t row = (int64_t)b * H + head;
  const int n = a.dst_lens[b];
  const int64_t ab = (int64_t)(D / 2) << a.src.lg, v = which * a.src.half_bytes(D);
  const int mask = (1 << a.src.lg) - 1;
  const int first = blockIdx.x * PER * kMoves + threadIdx.x / TPP;
  int64_t s[kMoves], d[kMoves];
#pragma unroll
  for (int j = 0; j < kMoves; ++j) {
    const int i = first + j * PER;
    s[j] = i < n ? a.kept[row * a.keep + i] : -1;
  }
#pragma unroll
  for (int j = 0; j < kMoves; ++j) {
    const int i = first + j * PER;
    if (i >= n) continue;
    d[j] = a.dst.slot(b, i);
    s[j] = a.src.slot(b, s[j]);
    if (s[j] < 0 || d[j] < 0) {
      if (u == 0) atomicOr(&g_evict_error, kErrExtent);
      s[j] = -1;
    }
  }
  uint4 x[kMoves];
  uint32_t w[kMoves];
#pragma unroll
  for (int j = 0; j < kMoves; ++j)
    if (s[j] >= 0) {
      const uint8_t* f = a.src.block(s[j], head, D) + v;
      const int64_t p = s[j] & mask;
      x[j] = *reinterpret_cast<const uint4*>(f + p * (D / 2) + 16 * c);
      if (c < D / 64) w[j] = reinterpret_cast<const uint32_t*>(f + ab)[p * (D / 64) + c];
    }
#pragma unroll
  for (int j = 0; j < kMoves; ++j)
    if (s[j] >= 0) {
      uint8_t* g = a.dst.block(d[j], head, D) + v;
      const int64_t p = d[j] & mask;
      *reinterpret_cast<uint4*>(g + p * (D / 2) + 16 * c) = x[j];
      if (c < D / 64) reinterpret_cast<uint32_t*>(g + ab)[p * (D / 64) + c] = w[j];
    }
}

}  // namespace

cudaError_t launch_kv_evict(const Evict& a, int d, int nsm, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kShare;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // four CTAs where the pairs leave most SMs idle and may be long (4 sequences of 8 heads, 20001 ..
  // 32001 positions: 52 us with one CTA each, selection and move, 43 with four; 128 pairs of 4096: 16)
  const bool few = (int64_t)a.src.H * a.src.B * kShare <= nsm &&
                   std::min<int64_t>(a.src.cap(), a.acc_stride) >= 4096;
  cfg.numAttrs = few ? 2 : 1;
  cfg.gridDim = dim3(a.src.H * (few ? kShare : 1), a.src.B);
  cudaError_t e = few ? cudaLaunchKernelEx(&cfg, select_kernel<kShare>, a)
                      : cudaLaunchKernelEx(&cfg, select_kernel<1>, a);
  if (e != cudaSuccess) return e;
  const int per = 256 / (d / 16) * kMoves;
  return launch_pdl(d == 128 ? move_kernel<128> : move_kernel<64>,
                    dim3((a.keep + per - 1) / per, a.src.H, a.src.B), dim3(256), 0, st, a);
}

cudaError_t evict_read_error(unsigned int* out) { return read_and_clear(g_evict_error, out); }

}  // namespace fg
