// Smaller caches: every K/V head of a sequence keeps its newest positions and the heaviest of the
// others, moved in order into pages of their own (sm_103a).
//
// Selection, a CTA per (sequence, head): the weights' order keys are 32-bit numbers, and four
// passes over them, a histogram of 8 bits each, find the key of the last one that stays and how many
// equal ones do; a last pass lists the positions in order.  Ties go to the lower position.
// Moving: a position's K and V codes and statistics, copied as they are.
#include <algorithm>

#include "attn_q4.cuh"
#include "fg_common.cuh"
#include "fg_internal.h"
#include "paged.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_evict_error = 0;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// The block's sum of `mine`, and the sum of the threads before this one.
__device__ __forceinline__ int block_scan(int mine, int* warp_sums, int* before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int total = 0, base = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) base = total;
    total += warp_sums[i];
  }
  *before = base + incl - mine;
  return total;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const Evict a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kWarps];
  __shared__ int found[2];
  pdl_launch_dependents();
  pdl_wait();
  const int head = blockIdx.x, b = blockIdx.y, H = a.src.H;
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
  if (head == 0 && threadIdx.x == 0) a.dst_lens[b] = left;
  for (int i = left + threadIdx.x; i < a.keep; i += kThreads) {
    kept[i] = -1;
    acc_out[i] = 0.0f;
  }
  if (n <= a.keep) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      kept[i] = i;
      acc_out[i] = acc[i];
    }
    return;
  }
  const int old = n - a.recent;            // recent <= keep < n
  int want = a.keep - a.recent;            // of the first `old`
  // the key of the want-th largest, 8 bits at a time
  uint32_t prefix = 0;
  for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < old; i += kThreads) {
      const uint32_t k = q4attn::order_key_f32(acc[i]);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[k >> shift & 255u], 1);
    }
    __syncthreads();
    // bins from the top: the one in which the want-th falls
    const int bin = 255 - (int)threadIdx.x;
    int before, mine = threadIdx.x < 256 ? hist[bin] : 0;
    block_scan(mine, warp_sums, &before);
    if (threadIdx.x < 256 && before < want && before + mine >= want) {
      found[0] = bin;
      found[1] = before;
    }
    __syncthreads();
    prefix = prefix << 8 | (uint32_t)found[0];
    want -= found[1];
  }
  // larger keys stay, and the first `want` equal ones
  const bool none = a.keep == a.recent;
  int at = 0, equal = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t k = i < old && !none ? q4attn::order_key_f32(acc[i]) : 0;
    const bool same = i < old && !none && k == prefix;
    int before;
    const int equals = block_scan(same, warp_sums, &before);
    const bool stays = i < n && (i >= old || (!none && (k > prefix || (same && equal + before < want))));
    const int stay = block_scan(stays, warp_sums, &before);
    if (stays) {
      kept[at + before] = i;
      acc_out[at + before] = acc[i];
    }
    at += stay;
    equal += equals;
  }
}

// A warp per kept position.
template <int D>
__global__ void __launch_bounds__(256) move_kernel(const Evict a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y, b = blockIdx.z, H = a.src.H;
  const int64_t row = (int64_t)b * H + head;
  const int n = a.dst_lens[b];
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8) {
    const int t = a.kept[row * a.keep + i];
    const int64_t s = a.src.slot(b, t), d = a.dst.slot(b, i);
    if (s < 0 || d < 0) {
      if (lane == 0) atomicOr(&g_evict_error, kErrExtent);
      continue;
    }
    const int64_t sp = s & ((1 << a.src.lg) - 1), dp = d & ((1 << a.src.lg) - 1);
    const int64_t ab = (int64_t)(D / 2) << a.src.lg;
    for (int w = 0; w < 2; ++w) {
      const uint8_t* f = a.src.block(s, head, D) + w * a.src.half_bytes(D);
      uint8_t* g = a.dst.block(d, head, D) + w * a.src.half_bytes(D);
      if (lane < D / 8)
        reinterpret_cast<uint32_t*>(g + dp * (D / 2))[lane] =
            reinterpret_cast<const uint32_t*>(f + sp * (D / 2))[lane];
      if (lane < D / 64)
        reinterpret_cast<uint32_t*>(g + ab)[dp * (D / 64) + lane] =
            reinterpret_cast<const uint32_t*>(f + ab)[sp * (D / 64) + lane];
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(const Evict& a, int d, int nsm, cudaStream_t st) {
  cudaError_t e = launch_pdl(select_kernel, dim3(a.src.H, a.src.B), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(d == 128 ? move_kernel<128> : move_kernel<64>,
                    dim3(std::min((a.keep + 7) / 8, 64), a.src.H, a.src.B), dim3(256), 0, st, a);
}

cudaError_t evict_read_error(unsigned int* out) { return read_and_clear(g_evict_error, out); }

}  // namespace fg
