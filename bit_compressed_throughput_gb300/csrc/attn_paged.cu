// Attention of the newest tokens of every sequence over the paged 4-bit cache, and the softmax
// weights that cached positions receive (sm_103a): plain forms, a warp per query row and head, a
// warp per cached position.
#include <math.h>

#include "fg_common.cuh"
#include "fg_internal.h"
#include "paged.cuh"
#include "q4_restore.cuh"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_paged_attn_error = 0;

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float restored(uint32_t code, uint32_t abw) {
  const float2 ab = unpack_h2(abw);
  const float s = __fdiv_rn(__fsub_rn(ab.y, ab.x), 15.0f);
  return h2f(f2h(__fadd_rn(ab.x, __fmul_rn((float)code, s))));
}
// Whether sequence b's extents fit; its query rows, first row and length.
struct Extent {
  int q0, nq, n;
};
__device__ __forceinline__ bool extent_of(const PagedAttn& a, int b, Extent& e) {
  const int q0 = a.q_off[b], q1 = a.q_off[b + 1], n = a.lens[b];
  if (q0 < 0 || q0 > q1 || q1 > a.q_rows || q1 - q0 > a.max_q || n < 0 || n > a.cache.cap())
    return false;
  e = Extent{q0, q1 - q0, n};
  return true;
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

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const PagedAttn a) {
  __shared__ float qs[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  if (w >= (int64_t)a.q_rows * a.Hq) return;
  const int row = (int)(w / a.Hq), hq = (int)(w % a.Hq), hk = hq / (a.Hq / a.cache.H);
  const int b = sequence_of_row(a.q_off, a.cache.B, row);
  Extent e;
  if (b < 0) return;
  if (!extent_of(a, b, e)) {
    atomicOr(&g_paged_attn_error, kErrExtent);
    return;
  }
  const int i = e.n - e.nq + row - e.q0;
  const uint16_t* q = a.q + row * a.q_stride + (int64_t)hq * D;
  for (int j = lane; j < D; j += 32) qs[warp][j] = h2f(q[j]) * a.scale;
  __syncwarp();
  constexpr int C = D / 32;
  float m = -INFINITY, l = 0.0f, o[C] = {};
  for (int t0 = 0; t0 <= i; t0 += 32) {
    const int t = t0 + lane;
    const bool vis = visible(t, i, a.window, a.sinks);
    float s = -INFINITY;
    const uint32_t* ab;
    if (vis) {
      const uint8_t* k = row_of<D>(a.cache, b, hk, t, 0, &ab);
      s = 0.0f;
      for (int j = 0; k && j < D / 2; ++j)
        s += qs[warp][2 * j] * restored(k[j] & 15u, ab[j / 32]) +
             qs[warp][2 * j + 1] * restored(k[j] >> 4, ab[j / 32]);
    }
    float mx = s;
    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    mx = fmaxf(mx, m);
    const float ref = mx == -INFINITY ? 0.0f : mx, corr = __expf(m - ref);
    const float p = vis ? __expf(s - ref) : 0.0f;
    l = l * corr + p;
    m = mx;
    for (int c = 0; c < C; ++c) o[c] *= corr;
    for (int u = 0; u < 32; ++u) {
      if (!__shfl_sync(0xFFFFFFFFu, vis, u)) continue;
      const float pu = __shfl_sync(0xFFFFFFFFu, p, u);
      const uint8_t* v = row_of<D>(a.cache, b, hk, t0 + u, 1, &ab);
      for (int c = 0; v && c < C; ++c) {
        const int ch = lane * C + c;
        o[c] += pu * restored(v[ch / 2] >> (4 * (ch & 1)) & 15u, ab[ch / 64]);
      }
    }
  }
  for (int d = 1; d < 32; d <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  uint16_t* out = a.out + row * a.out_stride + (int64_t)hq * D;
  for (int c = 0; c < C; ++c) out[lane * C + c] = f2h(l == 0.0f ? 0.0f : o[c] / l);
  if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

// A warp per (sequence, K/V head, position): lanes take (row, head) pairs.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const PagedAttn a) {
  __shared__ float ks[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, hk = blockIdx.y, G = a.Hq / a.cache.H;
  Extent e;
  if (!extent_of(a, b, e) || e.n > a.acc_stride) {
    if (threadIdx.x == 0) atomicOr(&g_paged_attn_error, kErrExtent);
    return;
  }
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < e.n; t += (int64_t)gridDim.x * kWarps) {
    const uint32_t* ab;
    const uint8_t* k = row_of<D>(a.cache, b, hk, t, 0, &ab);
    __syncwarp();
    for (int j = lane; k && j < D; j += 32)
      ks[warp][j] = restored(k[j / 2] >> (4 * (j & 1)) & 15u, ab[j / 64]);
    __syncwarp();
    float sum = 0.0f;
    for (int64_t p = lane; p < (int64_t)e.nq * G; p += 32) {
      const int r = (int)(p / G), hq = hk * G + (int)(p % G), i = e.n - e.nq + r;
      if (!visible((int)t, i, a.window, a.sinks)) continue;
      const uint16_t* q = a.q + (e.q0 + r) * a.q_stride + (int64_t)hq * D;
      float s = 0.0f;
      for (int j = 0; j < D; ++j) s = fmaf(h2f(q[j]), ks[warp][j], s);
      sum += expf(s * a.scale - a.lse_in[(int64_t)(e.q0 + r) * a.Hq + hq]);
    }
    for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const int64_t at = ((int64_t)b * a.cache.H + hk) * a.acc_stride + t;
    if (lane == 0) a.acc_out[at] = (a.acc ? a.acc[at] : 0.0f) + sum;
  }
}

}  // namespace

size_t attn_paged_ws_bytes(const fg_kvpages& kv, int32_t Hq, int32_t max_q) { return 256; }

cudaError_t launch_attn_paged(const PagedAttn& a, int d, void* ws, int nsm, cudaStream_t st) {
  const int64_t warps = (int64_t)a.q_rows * a.Hq;
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps));
  if (d == 128) attend_kernel<128><<<grid, kWarps * 32, 0, st>>>(a);
  else attend_kernel<64><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_attn_weights_paged(const PagedAttn& a, int d, int nsm, cudaStream_t st) {
  const dim3 grid(64, a.cache.H, a.cache.B);
  if (d == 128) weights_kernel<128><<<grid, kWarps * 32, 0, st>>>(a);
  else weights_kernel<64><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t paged_attn_read_error(unsigned int* out) {
  return read_and_clear(g_paged_attn_error, out);
}

}  // namespace fg
