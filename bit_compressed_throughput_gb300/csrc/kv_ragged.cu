// Ragged K/V cache: rows of sequences of different lengths quantised into the 4-bit cache at
// each sequence's own position, and ranges of cached positions restored to fp16 rows (sm_103a).
//
// Rows row_off[b] .. row_off[b+1]-1 belong to sequence b and are positions pos[b], pos[b] + 1, ..
// The format is the cache's (include/fg.h): 64 consecutive channels of a row share (a, b), codes
// q = rint((x - a) 15 / (b - a)) in binary32, restored as fp16(a + q ((b - a) / 15)).
//
// Both are bound by HBM: 2 bytes of fp16 and 0.5625 bytes of codes and statistics per element.
// Work split: 8 lanes per group of 64, in row order.
#include "fg_common.cuh"
#include "fg_internal.h"
#include "ragged.cuh"

namespace fg {

__device__ unsigned int g_ragged_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kGroupsPerCta = kThreads / 8;

struct RaggedArgs {
  const int32_t* row_off;
  const int32_t* pos;
  int rows, B, H, d, cap;
  int64_t stride;      // elements between the fp16 rows
};

// Cache slot ((b*H + head)*cap + position) of row `row` and head `head`, or -1.
__device__ __forceinline__ int64_t slot_of(const RaggedArgs& a, int row, int head) {
  const int b = sequence_of_row(a.row_off, a.B, row);
  if (b < 0) return -1;
  const int64_t t = (int64_t)row - a.row_off[b];
  const int64_t p = a.pos[b] + t;
  if (t < 0 || row >= a.row_off[b + 1]) return -1;
  if (a.pos[b] < 0 || p >= a.cap) {
    atomicOr(&g_ragged_error, kErrExtent);
    return -1;
  }
  return ((int64_t)b * a.H + head) * a.cap + p;
}

__global__ void __launch_bounds__(kThreads)
append_kernel(const RaggedArgs a, const uint16_t* __restrict__ k_new,
              const uint16_t* __restrict__ v_new, const fg_kvcache kv) {
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 &&
      !offsets_ok(a.row_off, a.B, a.rows, threadIdx.x, kThreads))
    atomicOr(&g_ragged_error, kErrExtent);
  const int gpr = a.H * (a.d >> 6), gph = a.d >> 6;
  const int64_t grp = (int64_t)blockIdx.x * kGroupsPerCta + (threadIdx.x >> 3);
  const int sub = threadIdx.x & 7;
  const int row = (int)(grp / gpr), gi = (int)(grp - (int64_t)row * gpr);
  const int64_t slot = (row < a.rows) ? slot_of(a, row, gi / gph) : -1;
  const uint16_t* src = blockIdx.y ? v_new : k_new;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (slot >= 0) v = ldg_nc_v4(src + (int64_t)row * a.stride + gi * 64 + sub * 8);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t mm = q4_minmax8(w);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mm = __vminu2(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
  const uint32_t abw = q4_ab_word(mm);
  const uint32_t c = q4_codes8_checked_x2(w, q4_group(abw));
  if (slot >= 0) {
    const int gs = gi % gph;
    uint8_t* codes = blockIdx.y ? kv.v_codes : kv.k_codes;
    uint32_t* ab = blockIdx.y ? kv.v_ab : kv.k_ab;
    reinterpret_cast<uint32_t*>(codes + slot * (a.d >> 1) + gs * 32)[sub] = c;
    if (sub == 0) ab[slot * gph + gs] = abw;
  }
}

__global__ void __launch_bounds__(kThreads)
read_kernel(const RaggedArgs a, const fg_kvcache kv, uint16_t* __restrict__ k_out,
            uint16_t* __restrict__ v_out) {
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 &&
      !offsets_ok(a.row_off, a.B, a.rows, threadIdx.x, kThreads))
    atomicOr(&g_ragged_error, kErrExtent);
  uint16_t* out = blockIdx.y ? v_out : k_out;
  if (!out) return;
  const int gpr = a.H * (a.d >> 6), gph = a.d >> 6;
  const int64_t grp = (int64_t)blockIdx.x * kGroupsPerCta + (threadIdx.x >> 3);
  const int sub = threadIdx.x & 7;
  const int row = (int)(grp / gpr), gi = (int)(grp - (int64_t)row * gpr);
  if (row >= a.rows) return;
  const int64_t slot = slot_of(a, row, gi / gph);
  if (slot < 0) return;
  const int gs = gi % gph;
  const uint8_t* codes = blockIdx.y ? kv.v_codes : kv.k_codes;
  const uint32_t* ab = blockIdx.y ? kv.v_ab : kv.k_ab;
  const uint32_t c = reinterpret_cast<const uint32_t*>(codes + slot * (a.d >> 1) + gs * 32)[sub];
  const uint32_t abw = ab[slot * gph + gs];
  const float af = h2f((uint16_t)(abw & 0xFFFFu)), bf = h2f((uint16_t)(abw >> 16));
  const float s = __fdiv_rn(__fsub_rn(bf, af), 15.0f);
  uint32_t o[4];
#pragma unroll
  for (int n = 0; n < 4; ++n)
    o[n] = pack_h2(__fadd_rn(af, __fmul_rn((float)((c >> (8 * n)) & 0xF), s)),
                   __fadd_rn(af, __fmul_rn((float)((c >> (8 * n + 4)) & 0xF), s)));
  reinterpret_cast<uint4*>(out + (int64_t)row * a.stride + gi * 64)[sub] =
      make_uint4(o[0], o[1], o[2], o[3]);
}

RaggedArgs args_of(const int32_t* row_off, const int32_t* pos, int32_t rows, int64_t stride,
                   const fg_kvcache& kv) {
  return RaggedArgs{row_off, pos, rows, kv.B, kv.H, kv.h / kv.H, kv.cap, stride};
}

}  // namespace

cudaError_t launch_kv_append_ragged(const uint16_t* k_new, const uint16_t* v_new,
                                    int64_t row_stride, int32_t rows, const int32_t* row_off,
                                    const int32_t* pos, const fg_kvcache& kv, cudaStream_t st) {
  const int64_t ng = (int64_t)rows * (kv.h / 64);
  const dim3 grid((unsigned)((ng + kGroupsPerCta - 1) / kGroupsPerCta), 2);
  return launch_pdl(append_kernel, grid, dim3(kThreads), 0, st,
                    args_of(row_off, pos, rows, row_stride, kv), k_new, v_new, kv);
}

cudaError_t launch_kv_read_ragged(const fg_kvcache& kv, const int32_t* row_off, const int32_t* pos,
                                  int32_t rows, uint16_t* k_out, uint16_t* v_out,
                                  int64_t row_stride, cudaStream_t st) {
  const int64_t ng = (int64_t)rows * (kv.h / 64);
  const dim3 grid((unsigned)((ng + kGroupsPerCta - 1) / kGroupsPerCta), 2);
  return launch_pdl(read_kernel, grid, dim3(kThreads), 0, st,
                    args_of(row_off, pos, rows, row_stride, kv), kv, k_out, v_out);
}

cudaError_t ragged_read_error(unsigned int* out) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_ragged_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_ragged_error, &zero, sizeof(unsigned int));
}

}  // namespace fg
