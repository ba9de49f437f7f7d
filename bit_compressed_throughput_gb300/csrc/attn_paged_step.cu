// Attention of single new tokens over the paged 4-bit cache: the streaming kernels of
// attn_decode_window.cuh, for the sequences of a call that have one query row and at most
// kStepHeads query heads per K/V head (attn_paged.cu has the others).
//
// With so few rows a key tile's restoring would cost the tensor-core kernel more than its bytes; here
// the codes go into the products as they are, and the bytes are what counts.  The page table comes 32
// entries at a time, a lane each, and a slot's four copies are issued by a lane each.  16 contexts of
// 9000 .. 32,760, 8 K/V heads of 128 channels, 4 query heads each, 384 MB: 93 us, 4.1 TB/s; 84 us with
// one query head each.
#include "attn_decode_window.cuh"
#include "paged.cuh"

namespace fg {

__device__ unsigned int g_paged_step_error = 0;

namespace {

using namespace decode_window;

struct Pages {
  static constexpr bool kLse = true;
  PagedCache pc;
  const int32_t *q_off, *lens;
  int q_rows, max_q;
  int B, H;
  // The next position, and the page table's entries page0 + lane of its sequence.
  struct Run {
    int b, hk, pos, page0;
    int32_t entry;
  };

  static __device__ __forceinline__ unsigned int* error_word() { return &g_paged_step_error; }
  __device__ __forceinline__ int64_t row(int b) const { return q_off[b]; }
  __device__ __forceinline__ bool misfit(int b) const {
    const int q0 = q_off[b], q1 = q_off[b + 1], n = lens[b];
    return q0 < 0 || q0 > q1 || q1 > q_rows || q1 - q0 > max_q || n < 0 || n > pc.cap();
  }
  __device__ __forceinline__ bool single(int b) const {
    return q_off[b + 1] - q_off[b] == 1 && !misfit(b);
  }
  __device__ __forceinline__ int length(int b) const { return single(b) ? lens[b] : 0; }
  __device__ __forceinline__ bool blind(int b) const { return single(b) && lens[b] == 0; }
  __device__ __forceinline__ void load(Run& r) const {
    r.page0 = r.pos >> pc.lg;
    const int64_t p = (int64_t)r.page0 + (threadIdx.x & 31);
    r.entry = p < pc.table_stride ? pc.table[r.b * pc.table_stride + p] : -1;
  }
  __device__ __forceinline__ void begin(Run& r, int b, int hk, int pos) const {
    r.b = b;
    r.hk = hk;
    r.pos = pos;
    load(r);
  }
  // A lane per copy: K codes, V codes, K and V statistics of each tile, or of both where they lie in
  // one page.
  template <int D>
  __device__ __forceinline__ void copy(Run& r, int tiles, uint32_t slot, uint32_t bar) const {
    using R = Ring<D>;
    const int lane = threadIdx.x & 31;
    if (((r.pos + (tiles - 1) * kTilePos) >> pc.lg) - r.page0 >= 32) load(r);
    const int page = r.pos >> pc.lg, second = (r.pos + kTilePos) >> pc.lg;
    const int32_t e0 = __shfl_sync(0xFFFFFFFFu, r.entry, page - r.page0);
    const int32_t e1 = __shfl_sync(0xFFFFFFFFu, r.entry, tiles > 1 ? second - r.page0 : 0);
    const bool ok0 = e0 >= 0 && e0 < pc.pages;
    const bool ok1 = tiles > 1 && e1 >= 0 && e1 < pc.pages;
    const bool joined = tiles > 1 && second == page;
    if (lane == 0 && !(ok0 && (ok1 || tiles == 1))) atomicOr(&g_paged_step_error, kErrExtent);
    // the slot was last read through the generic proxy; order that before the copies
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (lane == 0) mbar_expect_tx(bar, (ok0 + ok1) * kTilePos * 2 * (R::ROW_CODE + R::ROW_AB));
    __syncwarp();
    const int tile = lane >> 2, kind = lane & 3;       // kind: 0, 1 codes of K, V; 2, 3 statistics
    if (lane < 8 && (tile ? ok1 && !joined : ok0)) {
      const int32_t e = tile ? e1 : e0;
      const int64_t p = (r.pos + tile * kTilePos) & ((1 << pc.lg) - 1);
      const uint8_t* src = pc.block((int64_t)e << pc.lg, r.hk, D) + (kind & 1) * pc.half_bytes(D);
      const uint32_t rows = joined ? 2 * kTilePos : kTilePos;
      if (kind < 2)
        bulk_copy(slot + (kind ? R::V_OFF : 0) + tile * kTilePos * R::ROW_CODE,
                  src + p * R::ROW_CODE, rows * R::ROW_CODE, bar);
      else
        bulk_copy(slot + (kind == 3 ? R::VAB_OFF : R::KAB_OFF) + tile * kTilePos * R::ROW_AB,
                  src + ((int64_t)R::ROW_CODE << pc.lg) + p * R::ROW_AB, rows * R::ROW_AB, bar);
    }
    r.pos += tiles * kTilePos;
  }
};

int sets_of(int G) { return (G + set_heads(G) - 1) / set_heads(G); }

}  // namespace

size_t attn_paged_step_ws_bytes(const fg_kvpages& kv, int32_t Hq) {
  const int G = Hq / kv.H;
  // any number of sequences, of any length: as many shares as the largest grid has warps
  return workspace_bytes(1 << 20, 1 << 20, set_heads(G), kv.h / kv.H, kMaxSms);
}

cudaError_t launch_attn_paged_step(const PagedAttn& a, int d, void* ws, int nsm, cudaStream_t st) {
  const int G = a.Hq / a.cache.H;
  Args s;
  s.q = a.q;
  s.out = a.out;
  s.q_stride = a.q_stride;
  s.out_stride = a.out_stride;
  s.G = G;
  s.nhb = sets_of(G);
  s.window = a.window;
  s.sinks = a.sinks;
  s.scale_log2 = a.scale * 1.4426950408889634f;
  s.lse = a.lse;
  const Pages kv{a.cache, a.q_off, a.lens, a.q_rows, a.max_q, a.cache.B, a.cache.H};
  return launch_sets(s, kv, (int64_t)a.cache.B * a.cache.H * s.nhb, (int)a.cache.cap(), d, ws, nsm,
                     st);
}

cudaError_t paged_step_read_error(unsigned int* out) {
  return read_and_clear(g_paged_step_error, out);
}

}  // namespace fg
