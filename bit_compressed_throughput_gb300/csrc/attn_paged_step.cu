// Attention of single new tokens over the paged 4-bit cache: the streaming kernels of
// attn_decode_window.cuh, for the sequences of a call that have one query row and at most
// kStepHeads query heads per K/V head (attn_paged.cu has the others).
//
// With so few rows most of a row tile of the tensor-core kernel would be empty; here up to 8 heads
// are the columns of mma.sync products over values restored in registers, to the fp16 numbers that
// the tensor-core kernel restores, too: a position counts the same for a token and for a piece.  The
// page table comes 32 entries at a time, a lane each, and a slot's copies are issued by a lane each.
//
// Bound by instructions: 1570 for 32 positions of 128 channels, about 900 of them exact restoring.  16
// contexts of 9000 .. 32,760, 8 K/V heads of 128 channels, 384 MB: 178 us with 1 or 4 query heads each,
// 182 us with 8, 2.2 TB/s.  (Products over the codes as they are, weights times (b - a) / 15, took 84,
// 93 and 171 us, but K and V are not rounded to fp16 then: relative error of the outputs 3.7e-4 ..
// 4.8e-4, now 2.1e-4, their own rounding.  One fused multiply-add per value instead of the format's two
// roundings: 5% faster, neighbours.  16 warps of 128 registers gained nothing.)
#include "attn_decode_window.cuh"
#include "paged.cuh"

namespace fg {

__device__ unsigned int g_paged_step_error = 0;

namespace {

using namespace decode_window;

struct Pages {
  static constexpr bool kLse = true, kRestored = true;
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
  // A lane per copy: K codes, V codes, K and V statistics of the slot's tiles, those of one page at
  // once.
  template <int D>
  __device__ __forceinline__ void copy(Run& r, int tiles, uint32_t slot, uint32_t bar) const {
    using R = Ring<D, true>;
    const int lane = threadIdx.x & 31, tile = lane >> 2, kind = lane & 3;  // 0, 1: codes of K, V
    if (((r.pos + (tiles - 1) * kTilePos) >> pc.lg) - r.page0 >= 32) load(r);
    const int pos = r.pos + min(tile, tiles - 1) * kTilePos;
    const int32_t e = __shfl_sync(0xFFFFFFFFu, r.entry, (pos >> pc.lg) - r.page0);
    const bool ok = tile < tiles && e >= 0 && e < pc.pages;
    const unsigned oks = __ballot_sync(0xFFFFFFFFu, ok);
    if (lane == 0) {
      if (__popc(oks) != 4 * tiles) atomicOr(&g_paged_step_error, kErrExtent);
      // the slot was last read through the generic proxy; order that before the copies
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_expect_tx(bar, __popc(oks) * (kTilePos / 2) * (R::ROW_CODE + R::ROW_AB));
    }
    __syncwarp();
    const int in_page = pos & ((1 << pc.lg) - 1);
    if (ok && (tile == 0 || in_page == 0)) {           // the first of its page
      const uint8_t* src = pc.block((int64_t)e << pc.lg, r.hk, D) + (kind & 1) * pc.half_bytes(D);
      const uint32_t rows = min((tiles - tile) * kTilePos, (1 << pc.lg) - in_page);
      if (kind < 2)
        bulk_copy(slot + (kind ? R::V_OFF : 0) + tile * kTilePos * R::ROW_CODE,
                  src + in_page * R::ROW_CODE, rows * R::ROW_CODE, bar);
      else
        bulk_copy(slot + (kind == 3 ? R::VAB_OFF : R::KAB_OFF) + tile * kTilePos * R::ROW_AB,
                  src + ((int64_t)R::ROW_CODE << pc.lg) + in_page * R::ROW_AB, rows * R::ROW_AB, bar);
    }
    r.pos += tiles * kTilePos;
  }
};

int sets_of(int G) { return (G + set_heads(G, true) - 1) / set_heads(G, true); }

}  // namespace

size_t attn_paged_step_ws_bytes(const fg_kvpages& kv, int32_t Hq) {
  const int G = Hq / kv.H;
  // any number of sequences, of any length: as many shares as the largest grid has warps
  return workspace_bytes<true>(1 << 20, 1 << 20, set_heads(G, true), kv.h / kv.H, kMaxSms);
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
