// Decode attention over the 4-bit cache's regions, one per (sequence, head): the kernels of
// attn_decode_window.cuh.
#include "attn_decode_window.cuh"

namespace fg {

__device__ unsigned int g_decode_window_error = 0;

namespace {

using namespace decode_window;

struct Regions {
  static constexpr bool kLse = false, kRestored = false;
  fg_kvcache kv;
  const int32_t* lens;
  int B, H;
  using Run = int64_t;                     // the next position, as a row of the cache

  static __device__ __forceinline__ unsigned int* error_word() { return &g_decode_window_error; }
  __device__ __forceinline__ int64_t row(int b) const { return b; }
  __device__ __forceinline__ bool misfit(int b) const {
    const int len = lens[b];
    return len < 0 || len > kv.cap;
  }
  // A sequence's length, 0 when it does not fit the cache.
  __device__ __forceinline__ int length(int b) const {
    const int len = lens[b];
    return (len < 0 || len > kv.cap) ? 0 : len;
  }
  __device__ __forceinline__ bool blind(int b) const { return length(b) == 0; }
  __device__ __forceinline__ void begin(Run& r, int b, int hk, int pos) const {
    r = ((int64_t)b * H + hk) * kv.cap + pos;
  }
  template <int D>
  __device__ __forceinline__ void copy(Run& r, int tiles, uint32_t slot, uint32_t bar) const {
    using R = Ring<D, false>;
    constexpr int NG = D / 64;
    const uint32_t rows = tiles * kTilePos;            // whole tiles: never past cap
    if ((threadIdx.x & 31) == 0) {
      // the slot was last read through the generic proxy; order that before the copy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_expect_tx(bar, rows * 2 * (R::ROW_CODE + R::ROW_AB));
      bulk_copy(slot, kv.k_codes + r * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(slot + R::KAB_OFF, kv.k_ab + r * NG, rows * R::ROW_AB, bar);
      bulk_copy(slot + R::V_OFF, kv.v_codes + r * R::ROW_CODE, rows * R::ROW_CODE, bar);
      bulk_copy(slot + R::VAB_OFF, kv.v_ab + r * NG, rows * R::ROW_AB, bar);
    }
    r += rows;
  }
};

}  // namespace

size_t decode_attn_window_ws_bytes(const fg_kvcache& kv, int32_t Hq) {
  const int G = Hq / kv.H, heads = set_heads(G, false);
  return workspace_bytes<false>((int64_t)kv.B * kv.H * ((G + heads - 1) / heads), kv.cap, heads,
                         kv.h / kv.H, kMaxSms);
}

cudaError_t launch_decode_attn_window(const uint16_t* q, int64_t q_stride, int32_t Hq,
                                      const fg_kvcache& kv, const int32_t* lens, int32_t window,
                                      int32_t sinks, float scale, uint16_t* out,
                                      int64_t out_stride, void* ws, int nsm, cudaStream_t st) {
  const int G = Hq / kv.H, heads = set_heads(G, false);
  Args a;
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.G = G;
  a.nhb = (G + heads - 1) / heads;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.lse = nullptr;
  return launch_sets(a, Regions{kv, lens, kv.B, kv.H}, (int64_t)kv.B * kv.H * a.nhb, kv.cap,
                     kv.h / kv.H, ws, nsm, st);
}

cudaError_t decode_window_read_error(unsigned int* out) {
  return read_and_clear(g_decode_window_error, out);
}

}  // namespace fg
