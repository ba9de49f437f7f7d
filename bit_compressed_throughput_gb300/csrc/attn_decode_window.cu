// Decode attention over the 4-bit cache for sequences of different lengths, with a sliding
// window, first positions that stay visible, and query heads that share K/V heads (sm_103a).
//
// The query of sequence b is its newest position i = lens[b] - 1:
//   out_hq = sum_t softmax_t(scale * q_hq . k^_t) v^_t   over the t that i sees,
// K/V head hq / G of G = Hq / H query heads each; a sequence of length 0 sees nothing and gets
// zeros.
//
// One warp per (sequence, query head): a lane holds d/32 channels, one position at a time.
#include <math.h>

#include "fg_common.cuh"
#include "fg_internal.h"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_decode_window_error = 0;

namespace {

constexpr int kThreads = 256;

template <int D>
__device__ __forceinline__ void restore_lane(const uint8_t* codes, const uint32_t* ab, int64_t slot,
                                             int lane, float (&x)[D / 32]) {
  constexpr int C = D / 32;
  uint32_t w;
  if (C == 4)
    w = *reinterpret_cast<const uint16_t*>(codes + slot * (D / 2) + lane * 2);
  else
    w = codes[slot * (D / 2) + lane];
  const uint32_t abw = ab[slot * (D / 64) + lane * C / 64];
  const float af = h2f((uint16_t)(abw & 0xFFFFu)), bf = h2f((uint16_t)(abw >> 16));
  const float s = __fdiv_rn(__fsub_rn(bf, af), 15.0f);
#pragma unroll
  for (int c = 0; c < C; ++c)
    x[c] = h2f(f2h(__fadd_rn(af, __fmul_rn((float)((w >> (4 * c)) & 0xF), s))));
}

template <int D>
__global__ void __launch_bounds__(kThreads)
decode_window_kernel(const uint16_t* __restrict__ q, int64_t q_stride, int Hq, const fg_kvcache kv,
                     const int32_t* __restrict__ lens, int window, int sinks, float scale,
                     uint16_t* __restrict__ out, int64_t out_stride) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= (int64_t)kv.B * Hq) return;
  const int b = (int)(item / Hq), hq = (int)(item - (int64_t)b * Hq);
  int len = lens[b];
  if (len < 0 || len > kv.cap) {
    if (lane == 0) atomicOr(&g_decode_window_error, kErrExtent);
    len = 0;
  }
  const int64_t slot0 = ((int64_t)b * kv.H + hq / (Hq / kv.H)) * kv.cap;
  float qv[C], acc[C], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    qv[c] = h2f(q[(int64_t)b * q_stride + (int64_t)hq * D + lane * C + c]) * scale;
    acc[c] = 0.0f;
  }
  const int w0 = (window == 0) ? 0 : max(0, len - window);
  for (int t = 0; t < len; ++t) {
    if (t < w0 && t >= sinks) {
      t = w0 - 1;
      continue;
    }
    float k[C], v[C], s = 0.0f;
    restore_lane<D>(kv.k_codes, kv.k_ab, slot0 + t, lane, k);
    restore_lane<D>(kv.v_codes, kv.v_ab, slot0 + t, lane, v);
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(qv[c], k[c], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const float mn = fmaxf(m, s);
    const float corr = (m == -INFINITY) ? 0.0f : expf(m - mn), p = expf(s - mn);
    l = l * corr + p;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(acc[c], corr, p * v[c]);
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    out[(int64_t)b * out_stride + (int64_t)hq * D + lane * C + c] =
        f2h(len > 0 ? acc[c] / l : 0.0f);
}

}  // namespace

size_t decode_attn_window_ws_bytes(const fg_kvcache&, int32_t) { return 0; }

cudaError_t launch_decode_attn_window(const uint16_t* q, int64_t q_stride, int32_t Hq,
                                      const fg_kvcache& kv, const int32_t* lens, int32_t window,
                                      int32_t sinks, float scale, uint16_t* out,
                                      int64_t out_stride, void*, int, cudaStream_t st) {
  const unsigned grid = (unsigned)(((int64_t)kv.B * Hq + kThreads / 32 - 1) / (kThreads / 32));
  auto* kernel = (kv.h / kv.H == 128) ? decode_window_kernel<128> : decode_window_kernel<64>;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, q, q_stride, Hq, kv, lens, window,
                    sinks, scale, out, out_stride);
}

cudaError_t decode_window_read_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_decode_window_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_decode_window_error, &zero, sizeof(unsigned int));
}

}  // namespace fg
