// Prefill attention over fp16 K/V rows of sequences of different lengths, with a sliding window,
// first positions that stay visible, and query heads that share K/V heads (sm_103a).
//
// Sequence b has nq = q_off[b+1] - q_off[b] query rows and nk = kv_off[b+1] - kv_off[b] K/V rows;
// query row r is position i = nk - nq + r (the newest positions), and
//   out_r,hq = sum_t softmax_t(scale * q_r,hq . k_t) v_t   over the t that i sees,
// K/V head hq / G of G = Hq / Hkv query heads each; a row that sees nothing gets zeros.
//
// One warp per (query row, query head): a lane holds d/32 channels, one key at a time.
#include <math.h>

#include "fg_common.cuh"
#include "fg_internal.h"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_prefill_window_error = 0;

namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads)
prefill_window_kernel(const PrefillWindow a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && (!offsets_ok(a.q_off, a.nseq, a.q_rows, threadIdx.x, kThreads) ||
                          !offsets_ok(a.kv_off, a.nseq, a.kv_rows, threadIdx.x, kThreads)))
    atomicOr(&g_prefill_window_error, kErrExtent);
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)a.q_rows * a.Hq) return;
  const int row = (int)(item / a.Hq), hq = (int)(item - (int64_t)row * a.Hq);
  const int b = sequence_of_row(a.q_off, a.nseq, row);
  if (b < 0) return;
  const int q0 = a.q_off[b], nq = a.q_off[b + 1] - q0;
  const int k0 = a.kv_off[b], nk = a.kv_off[b + 1] - k0;
  if (row < q0 || row >= q0 + nq || k0 < 0 || nk < 0 || k0 + nk > a.kv_rows) return;
  const int i = nk - nq + (row - q0), hk = hq / (a.Hq / a.Hkv);
  float qv[C], acc[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    qv[c] = h2f(a.q[(int64_t)row * a.q_stride + hq * D + lane * C + c]) * a.scale;
    acc[c] = 0.0f;
  }
  const int w0 = (a.window == 0) ? 0 : max(0, i + 1 - a.window);
  for (int t = 0; t <= i; ++t) {
    if (t < w0 && t >= a.sinks) {
      t = w0 - 1;
      continue;
    }
    const int64_t at = (int64_t)(k0 + t) * a.kv_stride + hk * D + lane * C;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(qv[c], h2f(a.k[at + c]), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float mn = fmaxf(m, s);
    const float corr = (m == -INFINITY) ? 0.0f : expf(m - mn), p = expf(s - mn);
    l = l * corr + p;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(acc[c], corr, p * h2f(a.v[at + c]));
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    a.out[(int64_t)row * a.out_stride + hq * D + lane * C + c] = f2h(i >= 0 ? acc[c] / l : 0.0f);
}

}  // namespace

cudaError_t launch_prefill_attn_window(const PrefillWindow& a, int d, int, cudaStream_t st) {
  const unsigned grid = (unsigned)(((int64_t)a.q_rows * a.Hq + kThreads / 32 - 1) / (kThreads / 32));
  return launch_pdl(d == 128 ? prefill_window_kernel<128> : prefill_window_kernel<64>, dim3(grid),
                    dim3(kThreads), 0, st, a);
}

cudaError_t prefill_window_read_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_prefill_window_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_prefill_window_error, &zero, sizeof(unsigned int));
}

}  // namespace fg
