/*
 * fg.h -- C ABI of libfg, the GB300 (sm_103a) engine for one OPT-style decoder layer
 * over 4-bit group-compressed weights and KV cache, run over a block of sequences.
 *
 * The method (FlexGen):
 *  - Weights and the KV cache are stored as 4-bit codes, grouped 64 elements at a
 *    time -- along the output channel for weights, along the hidden dimension for
 *    K/V -- with the group minimum a and maximum b kept per group, and are restored
 *    to FP16 before any compute; INT4 is a storage format, not an INT4 matmul.
 *    [FlexGen review (jaehun.me), section "4-bit 압축은 정수 연산 가속과 같은가",
 *     restating paper §5; "论文阅读：FlexGen" (blog.gzher.com) §3.4]
 *  - One layer is applied to every GPU batch of a block (B = g*m sequences) before the
 *    next layer's weights are used; generation is a prefill over the prompt that builds
 *    the KV cache, then decode steps that add one token per sequence.
 *    [FlexGen paper explainer, "Compute Schedule" and Algorithm 1; Figure 2]
 *
 * Storage formats (the pages leave them open; these are this library's):
 *  - fp16 values are IEEE binary16 bit patterns (uint16_t).
 *  - codes: element 2i in the low nibble, element 2i+1 in the high nibble of byte i,
 *    along the grouped (contiguous) dimension.
 *  - group statistics: one uint32_t per group of 64, the fp16 bits of a in the low
 *    half and of b in the high half.
 *  - code q = rint((x - a) * 15 / (b - a)) in IEEE binary32 with one rounding per
 *    operation (subtract, multiply by 15, divide), round half to even, clamped to
 *    [0, 15]; a and b are the group min and max (-0 ordered below +0); a constant
 *    group (b - a == 0) stores all-zero codes.  Restoring: fp16(a + q * ((b - a) / 15)).
 *  - weight W[K][N] (K = input channel, N = output channel): codes [K][N/2] bytes,
 *    ab [K][N/64] words, row-major, groups of 64 consecutive n at fixed k.
 *  - KV cache of one layer: codes [B][H][cap][d/2] bytes and ab [B][H][cap][d/64]
 *    words for K and for V, groups of 64 consecutive hidden channels (a group never
 *    straddles two heads since d is 64 or 128).
 *
 * Conventions for every call:
 *  - Pointers marked "device" are device memory owned by the caller; the library
 *    never allocates, frees or keeps them.  Work is enqueued asynchronously on
 *    `stream` (a cudaStream_t passed as void*; NULL = the legacy default stream).
 *  - Arguments are validated on the host before any launch; a bad argument returns a
 *    negative fg_status and launches nothing.  Validation touches no CUDA API, so it
 *    can be exercised on a machine without a GPU.
 *  - Device pointers must be 16-byte aligned.
 *  - A failed launch returns FG_ERR_CUDA; fg_last_error() gives the CUDA message
 *    (thread-local).  FG_ERR_ARCH: the current device is not sm_103.
 *  - Every device wait inside a kernel is bounded; a wait that runs out sets a device
 *    error word that fg_check_device_error() reads (FG_ERR_TIMEOUT).
 */
#ifndef FG_H_
#define FG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FG_OK = 0,
  FG_ERR_ARG = -1,        /* null pointer, misaligned pointer, bad enum */
  FG_ERR_SHAPE = -2,      /* a dimension outside the supported set */
  FG_ERR_WORKSPACE = -3,  /* workspace smaller than the matching *_workspace_bytes() */
  FG_ERR_CUDA = -4,       /* a CUDA call or launch failed (see fg_last_error) */
  FG_ERR_ARCH = -5,       /* current device is not compute capability 10.3 */
  FG_ERR_CAPACITY = -6,   /* KV cache position out of range */
  FG_ERR_TIMEOUT = -7     /* a bounded device wait ran out (kernel result invalid) */
} fg_status;

/* A 4-bit group-compressed weight W[K][N]. codes: device [K][N/2]; ab: device [K][N/64]. */
typedef struct {
  const uint8_t* codes;
  const uint32_t* ab;
  int64_t K;
  int64_t N;
} fg_q4mat;

/* The INT4 KV cache of one layer (device buffers, layout above). */
typedef struct {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint32_t* k_ab;
  uint32_t* v_ab;
  int32_t B;    /* sequences */
  int32_t cap;  /* positions per sequence, a multiple of 16 (whole 16-position tiles) */
  int32_t h;    /* hidden size */
  int32_t H;    /* heads; d = h / H must be 64 or 128 */
} fg_kvcache;

/* The INT4 KV cache of one layer in pages, for sequences that share one pool of memory.  blocks:
 * device [pages][H][page * 9 * d / 8] bytes; the block of one page and head holds K codes
 * [page][d/2], K ab [page][d/64] words, V codes, V ab, with the codes and statistics of above.
 * Which pages a sequence has stands in a page table of the call: device int32 [nseq][table_stride],
 * position p of sequence b being position p % page of page table[b][p / page].  The host never
 * reads it; entries of positions that a call does not touch may hold anything, and one that names
 * no page where a call needs it is reported by fg_check_device_error() (FG_ERR_CAPACITY).
 * table_stride * page < 2^31 - 65536; nseq <= 65535. */
typedef struct {
  uint8_t* blocks;
  int32_t pages;  /* pages of the pool */
  int32_t page;   /* positions per page: a power of two, 16 .. 1024 */
  int32_t h;      /* hidden size */
  int32_t H;      /* heads; d = h / H must be 64 or 128 */
} fg_kvpages;

/* Rotary positions: a row at position p turns pairs of the first `rot` channels of a head,
 *   y0 = x0 c - x1 s,  y1 = x0 s + x1 c,  (c, s) = angles[p][j], j < rot/2,
 * pairs (j, j + rot/2), or (2j, 2j + 1) when interleaved; every product and sum is rounded to
 * binary32, the result to fp16. */
typedef struct {
  const float* angles;  /* device [positions][rot/2][2], 16-byte aligned (fg_rope_table) */
  const int32_t* pos;   /* device [nseq]: the position of each sequence's first row */
  int32_t positions;    /* rows of the table */
  int32_t rot;          /* channels of a head that turn: a multiple of 16, at most d */
  int32_t interleaved;  /* 0 or 1 */
} fg_rope_rows;

typedef struct {
  int32_t h;      /* hidden size, multiple of 256, at most 16384 */
  int32_t H;      /* heads */
  int32_t d;      /* head dim, 64 or 128, h == H*d */
  int32_t f;      /* FFN width, multiple of 256; 0 = attention block without the MLP */
  float ln_eps;   /* LayerNorm epsilon */
} fg_dims;

/* One pre-LN decoder layer: h1 = x + Attn(LN1(x)) Wo + bo; y = h1 + ReLU(LN2(h1) W1 + b1) W2 + b2
 * with [Q|K|V] = LN1(x) Wqkv + bqkv. Weights K-major (W[in][out]); wqkv is [h][3h] with
 * columns q | k | v. All vectors fp16, device; biases may be NULL (zero).
 * w1/w2/b1/b2/ln2_* unused when f == 0. */
typedef struct {
  fg_q4mat wqkv, wo, w1, w2;
  const uint16_t *bqkv, *bo, *b1, *b2;
  const uint16_t *ln1_g, *ln1_b, *ln2_g, *ln2_b;
} fg_layer;

/* Epilogues of fg_dequant_gemm_q4. */
enum { FG_EPI_NONE = 0, FG_EPI_RELU = 1, FG_EPI_RESIDUAL = 2 };

/* ---------------------------------------------------------------------- quantise */

/* Group-wise 4-bit quantisation of fp16 x[rows][cols] (groups of 64 along cols), as
 * defined above.  x, codes [rows][cols/2], ab [rows][cols/64]: device.
 * cols % 64 == 0, rows >= 0 (rows == 0 is a no-op).  Bit-exact with the definition.
 * [FlexGen review (jaehun.me), "4-bit 압축은 정수 연산 가속과 같은가"] */
int fg_quantize_g64(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes,
                    uint32_t* ab, void* stream);

/* Restore fp16 y[rows][cols] = fp16(a + q * ((b - a) / 15)) (binary32, one rounding per
 * operation).  The standalone restore; the GEMM and attention restore in registers.
 * [same passage: values are restored to FP16 before compute] */
int fg_dequant_g64(const uint8_t* codes, const uint32_t* ab, int64_t rows, int64_t cols,
                   uint16_t* y, void* stream);

/* ---------------------------------------------------------------------- GEMM */

/* Y[M][N] = epi(X[M][K] * W^ + bias) with W^ the fp16 restoration of W, fp32 accumulate.
 * epi: FG_EPI_NONE; FG_EPI_RELU (max(.,0)); FG_EPI_RESIDUAL (+ residual[M][N]).
 * X, bias (nullable, [N]), residual (FG_EPI_RESIDUAL only), Y: device fp16, row-major,
 * leading dimensions K (X) and N (Y, residual).  K % 16 == 0, N % 256 == 0 (one output tile
 * of group statistics is one 16-byte row), M >= 0.
 * Y may alias residual.  ws: device scratch of at least fg_gemm_workspace_bytes(M,K,N)
 * bytes (split-K partial sums when M is small; with M > 256 a 4-byte unit counter that the
 * call zeroes on `stream` before its kernel); NULL allowed when that is 0.  Two calls in
 * flight at once on different streams need workspaces of their own.
 * [FlexGen review (jaehun.me), "4-bit 압축은 정수 연산 가속과 같은가": restore to FP16
 *  before compute, not an INT4 matmul; FlexGen paper explainer, "Cost Model and Policy
 *  Search": the four h x h and two h x h2 weight matrices of a layer] */
int fg_dequant_gemm_q4(const uint16_t* X, int64_t M, const fg_q4mat* W, const uint16_t* bias,
                       int epilogue, const uint16_t* residual, uint16_t* Y, void* ws,
                       size_t ws_bytes, void* stream);
/* Scratch bytes fg_dequant_gemm_q4 needs for an M x K by K x N product (split-K fp32
 * partials when M is small, and 256 bytes for the unit counter of the many-token plans;
 * 0 when neither applies).  Host computation only; the pages have no counterpart (their
 * GEMMs run in PyTorch). */
size_t fg_gemm_workspace_bytes(int64_t M, int64_t K, int64_t N);

/* The QKV projection with the KV quantise-and-append in its epilogue:
 *   Y[M][3h] = X[M][K] * W^[K][3h] + bias   (columns: Q, then K, then V),
 * and for every row r = b*T + t (sequence b of the cache, t < T) the K and V columns of
 * row r, rounded to fp16 as Y holds them, are quantised in groups of 64 (the same codes
 * and (a, b) as fg_kv_append_q4 gives for those rows) and written at position pos + t.
 * One launch (two when M is small enough for a split-K sum): the fp16 K/V are not read
 * back from memory.  h = kv->h, a multiple of 128; W->N == 3h; M == kv->B * T; T >= 1;
 * pos + T <= kv->cap; kv->B * kv->H * kv->cap < 2^31.  Y is still written in full (prefill attention reads the fp16 K/V).
 * ws as for fg_dequant_gemm_q4.  Errors as fg_dequant_gemm_q4, plus FG_ERR_CAPACITY.
 * [FlexGen review (jaehun.me), "4-bit 압축은 정수 연산 가속과 같은가": K/V grouped 64
 *  along the hidden dimension] */
int fg_dequant_gemm_q4_kv(const uint16_t* X, int64_t M, const fg_q4mat* W, const uint16_t* bias,
                          uint16_t* Y, const fg_kvcache* kv, int32_t T, int32_t pos, void* ws,
                          size_t ws_bytes, void* stream);

/* A GEMM whose output rows also pass through the pre-LN LayerNorm of the next sub-layer:
 *   Y = epilogue(X * W^ + bias)   (as fg_dequant_gemm_q4),
 *   Y_ln[r] = (Y[r] - mean) / sqrt(var + ln_eps) * ln_gamma + ln_beta   over the N values of
 *   row r of Y as stored (fp16), fp32 mean and population variance (as fg_layernorm).
 * When the plan splits K (few rows) the split-K reduce sums the partials, applies the
 * epilogue, stores Y and normalises the row in the same kernel (one CTA per row); otherwise
 * the GEMM is followed by the LayerNorm kernel.  N <= 16384; Y_ln must not alias Y (it
 * may alias nothing the GEMM reads).  ws as for fg_dequant_gemm_q4.  Errors as
 * fg_dequant_gemm_q4.  [OPT decoder layer as a pre-LN block; FlexGen paper explainer,
 *  "Computation Delegation": the layer's GEMMs and attention on the GPU] */
int fg_dequant_gemm_q4_ln(const uint16_t* X, int64_t M, const fg_q4mat* W, const uint16_t* bias,
                          int epilogue, const uint16_t* residual, uint16_t* Y,
                          const uint16_t* ln_gamma, const uint16_t* ln_beta, float ln_eps,
                          uint16_t* Y_ln, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------- KV cache */

/* Quantise new keys and values into the cache at positions pos .. pos+T-1 of every
 * sequence.  k_new, v_new: device fp16, row (b, t) at (b*T + t) * row_stride elements,
 * h contiguous values per row (row_stride >= h, a multiple of 8; lets K/V be read in
 * place from a [rows][3h] QKV buffer).  T >= 0; pos >= 0; pos + T <= cap.
 * Codes and statistics are bit-exact with fg_quantize_g64 on the same rows.
 * [FlexGen review (jaehun.me), "4-bit 압축은 정수 연산 가속과 같은가": KV grouped
 *  along the hidden dimension; FlexGen paper explainer, Figure 2: each decode step
 *  extends the cache] */
int fg_kv_append_q4(const uint16_t* k_new, const uint16_t* v_new, int64_t row_stride,
                    int32_t T, int32_t pos, const fg_kvcache* kv, void* stream);

/* Ragged append: sequences of different lengths, each at a position of its own.  Rows
 * row_off[b] .. row_off[b+1]-1 of k_new and v_new (h contiguous values per row, rows row_stride
 * elements apart: >= h, a multiple of 8) are quantised into positions pos[b], pos[b]+1, .. of
 * sequence b, with the codes and statistics fg_kv_append_q4 gives for those rows; everything
 * else in the cache stays as it was.  `rows`: the rows k_new and v_new hold (< 2^31 - 64); rows
 * before row_off[0] or from row_off[B] on are not used.  row_off: device int32 [B+1], 0 <=
 * row_off[b] <= row_off[b+1] <= rows; pos: device int32 [B], 0 <= pos[b], pos[b] + (rows of b) <=
 * cap.  The host never reads the two arrays, so their values are checked on the device: a row that
 * does not fit is not written, and fg_check_device_error() returns FG_ERR_CAPACITY.
 * rows == 0 or kv->B == 0 is a no-op.  The pages process blocks of equal prompts and have no
 * counterpart. */
int fg_kv_append_q4_ragged(const uint16_t* k_new, const uint16_t* v_new, int64_t row_stride,
                           int32_t rows, const int32_t* row_off, const int32_t* pos,
                           const fg_kvcache* kv, void* stream);

/* The inverse: positions pos[b], pos[b]+1, .. of sequence b restored to fp16 (the values of
 * fg_dequant_g64) into rows row_off[b] .. row_off[b+1]-1 of k_out and v_out, for prefill
 * attention over what the cache holds.  Arguments as fg_kv_append_q4_ragged; k_out or v_out may
 * be NULL (that half is not read); rows that overlap are refused (column blocks of one buffer do
 * not).  Rows outside every sequence, and rows that do not fit, stay as they were.  [FlexGen
 * review (jaehun.me), "4-bit 압축은 정수 연산 가속과 같은가": values are restored to FP16 before
 * compute] */
int fg_kv_read_q4_ragged(const fg_kvcache* kv, const int32_t* row_off, const int32_t* pos,
                         int32_t rows, uint16_t* k_out, uint16_t* v_out, int64_t row_stride,
                         void* stream);

/* ---------------------------------------------------------------------- paged cache */

/* angles[p][j] = gain * (cos, sin)(p * w_j) for p < positions, j < rot/2, computed in 64 bits and
 * rounded once.  w_j = base^(-2j/rot), stretched for contexts longer than those of `original`
 * positions: with r = original * w_j / 2 pi turns within them, w_j stays where r >= high, is divided
 * by `factor` where r <= low, and goes over linearly in r between; original = 0 divides every w_j.
 * factor = 1: no stretching.  rot even; 0 <= low <= high where original > 0.  A table is made once
 * and serves every call (and every layer). */
int fg_rope_table(float* angles, int32_t positions, int32_t rot, double base, double factor,
                  int32_t original, double low, double high, double gain, void* stream);

/* Rotary positions of packed rows: rows row_off[b] .. row_off[b+1]-1 of x are positions
 * rope->pos[b], rope->pos[b] + 1, .. of sequence b; every one of `heads` heads of d channels is
 * turned, channels behind the first rot are copied.  transpose = 1 turns by the transposed matrix
 * (s negated): the gradient of the call, given the gradient of its output, and with a gain of 1 its
 * inverse.  x, y: device fp16, rows x_stride and y_stride elements apart (>= heads * d, multiples of
 * 8); y may be x with the same stride; any other overlap of their rows is refused.  d in {64, 128}.
 * Extents are checked on the device as in fg_kv_append_q4_ragged: a row whose position the table
 * does not hold is not written.  The pages' models learn absolute positions; no counterpart. */
int fg_rope(const uint16_t* x, int64_t x_stride, int32_t rows, int32_t heads, int32_t d,
            const int32_t* row_off, int32_t nseq, const fg_rope_rows* rope, int32_t transpose,
            uint16_t* y, int64_t y_stride, void* stream);

/* fg_kv_append_q4_ragged into pages: rows row_off[b] .. row_off[b+1]-1 of k_new and v_new go to
 * positions pos[b], pos[b] + 1, .. of sequence b.  rope (nullable): K is turned first, as fg_rope
 * would, and quantised from the fp16 values that gives; rope->pos NULL means pos (they differ once
 * a cache has been made smaller).  Two rows that name the same place of the same page are a fault of
 * the caller (one of them is stored). */
int fg_kv_append_q4_paged(const uint16_t* k_new, const uint16_t* v_new, int64_t row_stride,
                          int32_t rows, const int32_t* row_off, const int32_t* pos,
                          const fg_rope_rows* rope, const fg_kvpages* kv, const int32_t* table,
                          int64_t table_stride, int32_t nseq, void* stream);

/* fg_kv_read_q4_ragged from pages. */
int fg_kv_read_q4_paged(const fg_kvpages* kv, const int32_t* table, int64_t table_stride,
                        int32_t nseq, const int32_t* row_off, const int32_t* pos, int32_t rows,
                        uint16_t* k_out, uint16_t* v_out, int64_t row_stride, void* stream);

/* Attention of the newest tokens of every sequence over its pages, one token or many: sequence b
 * has query rows q_off[b] .. q_off[b+1]-1 (nq of them, at most max_q) and lens[b] cached positions,
 * those of its query rows included (append first); query row r of them is position
 * i = lens[b] - nq + r, and
 *   out[row][hq*d + j] = sum_t softmax_t(scale * q_row,hq . K^_hk,t) V^_hk,t,j   over the visible t
 * (visible: as stated below for the windowed calls), hk = hq / (Hq / H), Hq a multiple of H, at
 * most 128 times H, nseq * Hq * (table_stride * page / 16 + 2) at most 2^40.  K^ and V^ are the
 * fp16 values that fg_kv_read_q4_paged gives.  A row that sees nothing gets 0.
 * lse (nullable): device fp32 [q_rows][Hq], the logarithm of the row's sum of exp(score), -inf for
 * a row that sees nothing.  q, out: device fp16, q_rows rows q_stride and out_stride elements apart
 * (>= Hq*d, multiples of 8); out may be q with the same stride; any other overlap of q, out and lse
 * is refused.
 * q_off: device int32 [nseq+1], not decreasing, within 0 .. q_rows; lens: device int32 [nseq], at
 * most what a row of the table names; checked on the device (the rows of a sequence that does not
 * fit stay as they were; those of one with a bad page hold nothing of use;
 * fg_check_device_error() returns FG_ERR_CAPACITY).  Rows outside every sequence stay as they were.
 * Values of positions that a row does not see never reach it, not even infinities and NaN.  ws:
 * device scratch of at least fg_attn_paged_workspace_bytes(kv, Hq, max_q) bytes, whatever the
 * lengths; two calls in flight at once need workspaces of their own. */
int fg_attn_q4kv_paged(const uint16_t* q, int64_t q_stride, int32_t q_rows, const int32_t* q_off,
                       int32_t max_q, int32_t Hq, const fg_kvpages* kv, const int32_t* table,
                       int64_t table_stride, const int32_t* lens, int32_t nseq, int32_t window,
                       int32_t sinks, float scale, uint16_t* out, int64_t out_stride, float* lse,
                       void* ws, size_t ws_bytes, void* stream);
/* Scratch bytes of fg_attn_q4kv_paged (planned for up to 192 SMs).  Host computation only; 0 for
 * invalid arguments. */
size_t fg_attn_paged_workspace_bytes(const fg_kvpages* kv, int32_t Hq, int32_t max_q);

/* The softmax weights that cached positions receive from given queries:
 *   acc_out[b][hk][t] = acc[b][hk][t] + sum exp(scale * q_row,hq . K^_hk,t - lse[row][hq])
 * over sequence b's query rows that see t and the query heads of hk, for t < lens[b]; everything
 * else of acc_out stays as it was.  acc (nullable: zeros) and acc_out: device fp32
 * [nseq][H][acc_stride], lens[b] <= acc_stride; acc_out may be acc, and any other overlap of it with
 * acc, lse or q is refused.  K^: the codes restored to fp16.  lse: as fg_attn_q4kv_paged
 * gives it; rows of -inf add nothing.  Sums are taken in one order whatever else runs.  The other
 * arguments as there. */
int fg_attn_weights_q4_paged(const uint16_t* q, int64_t q_stride, int32_t q_rows,
                             const int32_t* q_off, int32_t max_q, int32_t Hq, const fg_kvpages* kv,
                             const int32_t* table, int64_t table_stride, const int32_t* lens,
                             int32_t nseq, int32_t window, int32_t sinks, float scale,
                             const float* lse, const float* acc, float* acc_out,
                             int64_t acc_stride, void* stream);

/* Caches of at most `keep` positions: every K/V head of sequence b keeps its last `recent`
 * positions (<= keep) and, of the others, the keep - recent with the largest acc (equal ones: the
 * lower position first; NaN orders above +inf), or everything when lens[b] <= keep.  What stays is
 * moved, in order of position, to positions 0, 1, .. of the pages that dst_table names: pages of the
 * same pool that no sequence of `table` uses (afterwards the old pages are free).  kept: device
 * int32 [nseq][H][keep], the positions that stay, -1 behind them; acc_out: device fp32
 * [nseq][H][keep], their acc, 0 behind them; dst_lens: device int32 [nseq], min(lens[b], keep).
 * Heads keep different positions: a cached position no longer says when its token came, so later
 * rows give fg_kv_append_q4_paged a rope->pos of their own, and the attention's window and sinks
 * count cached positions, the ones that stayed, from then on.  keep <= dst_stride * page
 * (FG_ERR_CAPACITY).  acc as in fg_attn_weights_q4_paged.  kept, acc_out and dst_lens may overlap
 * neither one another nor acc, lens and the tables. */
int fg_kv_evict_q4_paged(const fg_kvpages* kv, const int32_t* table, int64_t table_stride,
                         int32_t nseq, const int32_t* lens, const float* acc, int64_t acc_stride,
                         int32_t keep, int32_t recent, const int32_t* dst_table,
                         int64_t dst_stride, int32_t* kept, float* acc_out, int32_t* dst_lens,
                         void* stream);

/* ---------------------------------------------------------------------- attention */

/* Decode attention of one new token per sequence over cache positions 0 .. len-1:
 * out[b][hd*d + j] = sum_t softmax_t(scale * q_b,hd . K^_b,hd,t) V^_b,hd,t,j with K^, V^
 * the fp16 restorations of the cached codes.  q: device fp16, row b at b*q_stride
 * elements; out: device fp16 [B][h].  1 <= len <= cap.  ws: device scratch of at least
 * fg_decode_attn_workspace_bytes(kv, len) bytes (split-sequence partials).
 * [FlexGen paper explainer, "Computation Delegation": decoding attention is I/O bound
 *  over the KV cache] */
int fg_decode_attn_q4kv(const uint16_t* q, int64_t q_stride, const fg_kvcache* kv, int32_t len,
                        float scale, uint16_t* out, void* ws, size_t ws_bytes, void* stream);
/* Scratch bytes fg_decode_attn_q4kv needs (split-sequence partials, planned for up to 192
 * SMs; 0 when no split is planned).  Host computation only; no counterpart on the pages. */
size_t fg_decode_attn_workspace_bytes(const fg_kvcache* kv, int32_t len);

/* Decode attention exactly as fg_decode_attn_q4kv, for callers that cannot allocate
 * device memory -- code that must not call cudaMalloc (a region that forbids allocation,
 * an external allocator that owns all device memory, a host runtime that can only pass
 * existing buffers through) and so cannot supply the split-sequence workspace.  Its
 * scratch is a fixed array of FG_DECODE_ATTN_STATIC_SCRATCH_BYTES in device global
 * memory defined by the library itself (held on every GPU that loads the library until
 * the process exits); the call allocates nothing.  The caller still passes q, the cache
 * and out.  A call whose split scratch (fg_decode_attn_workspace_bytes) would exceed the
 * array returns FG_ERR_WORKSPACE without launching, and fg_last_error() says so.
 * The first call on a device looks up the array's device address for that device; make
 * that first call before any stream capture.  All calls share the array: calls that
 * overlap on the GPU race on it.  No part of it needs to start at zero; each call writes
 * every byte it reads.  The paper has no counterpart of this entry point. */
#define FG_DECODE_ATTN_STATIC_SCRATCH_BYTES (4u << 20)
int fg_decode_attn_q4kv_static(const uint16_t* q, int64_t q_stride, const fg_kvcache* kv,
                               int32_t len, float scale, uint16_t* out, void* stream);

/* Top-K sparse decode attention over the same cache: the scores of all positions
 * 0 .. len-1 come from the 4-bit K and the softmax runs over all of them, but only the k
 * positions with the highest scores contribute their values:
 *   out[b][hd*d + j] = sum_{t in top-k(b,hd)} p_t V^_b,hd,t,j   (no renormalisation)
 * with equal scores at the k-th place going to the lower position.  1 <= k <= len <= cap,
 * d in {64, 128}, (len + k) * 4 + 1024 bytes <= 227 KB.  q, out as fg_decode_attn_q4kv.  sel
 * (nullable): device int32 [B][H][k] receiving the selected positions in increasing
 * position order.  ws: device scratch of at least fg_decode_attn_topk_workspace_bytes(kv,
 * len) bytes (the scores).
 * [论文阅读：FlexGen, §3.4: optional sparse attention that loads only the top 10% of the value
 *  cache; FlexGen paper explainer, §3.3: Top-K sparse attention cuts I/O volume] */
int fg_decode_attn_q4kv_topk(const uint16_t* q, int64_t q_stride, const fg_kvcache* kv,
                             int32_t len, int32_t k, float scale, uint16_t* out, int32_t* sel,
                             void* ws, size_t ws_bytes, void* stream);
size_t fg_decode_attn_topk_workspace_bytes(const fg_kvcache* kv, int32_t len);

/* Causal prefill attention over fp16 Q/K/V read from a QKV buffer qkv[nseq*s][3h]
 * (columns q | k | v, head hd at hd*d): out[nseq*s][h] fp16, position i attends over
 * positions 0..i of its own sequence, scores scaled by `scale`.  d in {64, 128}, scale > 0,
 * nseq <= 65535, nseq * s < 2^31; qkv and out device pointers, 16-byte aligned (FG_ERR_ARG
 * otherwise).  nseq == 0 or s == 0 is a no-op.
 * [FlexGen paper explainer, Figure 2: the prefill step processes all prompt tokens] */
int fg_prefill_attn(const uint16_t* qkv, int32_t nseq, int32_t s, int32_t H, int32_t d,
                    float scale, uint16_t* out, void* stream);

/* What a query sees in the two windowed calls: position i sees position t of its sequence when
 *   t <= i  and  (window == 0  or  t > i - window  or  t < sinks),
 * i.e. the newest `window` positions up to its own (0: all of them) and the first `sinks`
 * positions, which stay visible however far the window has moved.
 *
 * Decode attention over the 4-bit cache for sequences of different lengths: the query of
 * sequence b is its newest cached position i = lens[b] - 1, and
 *   out[b][hq*d + j] = sum_t softmax_t(scale * q_b,hq . K^_b,hk,t) V^_b,hk,t,j   over the visible t,
 * query head hq reading K/V head hk = hq / (Hq / H): Hq query heads, a multiple of the cache's H.
 * K^ and V^ enter the sums as a + q*((b-a)/15), not rounded to fp16 first.  A sequence of length
 * 0 sees nothing: its output is 0.  q: device fp16, row b at b*q_stride; out: device fp16, row b
 * at b*out_stride (both strides >= Hq*d, multiples of 8); out may be q itself, with the same
 * stride; any other overlap of their rows is refused.  Hq <= 65536, B*Hq*(cap/16 + 2) <= 2^40.
 * lens: device int32 [B], 0 <= lens[b] <= cap, checked on the device (a length that does not fit counts
 * as 0, and fg_check_device_error() returns FG_ERR_CAPACITY).  window, sinks >= 0.  ws: device
 * scratch of at least fg_decode_attn_window_workspace_bytes(kv, Hq) bytes, whatever the lengths
 * and the window; it needs no initialisation.  Two calls in flight at once need workspaces of
 * their own.  Reads the sequences' visible 16-position tiles only.  The pages attend over whole
 * caches of one length and have no counterpart. */
int fg_decode_attn_q4kv_window(const uint16_t* q, int64_t q_stride, int32_t Hq,
                               const fg_kvcache* kv, const int32_t* lens, int32_t window,
                               int32_t sinks, float scale, uint16_t* out, int64_t out_stride,
                               void* ws, size_t ws_bytes, void* stream);
/* Scratch bytes of fg_decode_attn_q4kv_window (planned for up to 192 SMs).  Host computation
 * only; 0 for invalid arguments. */
size_t fg_decode_attn_window_workspace_bytes(const fg_kvcache* kv, int32_t Hq);

/* Prefill attention over fp16 rows for sequences of different lengths: sequence b has query rows
 * q_off[b] .. q_off[b+1]-1 and K/V rows kv_off[b] .. kv_off[b+1]-1 (nq and nk of them); its query
 * rows are its newest positions, row r of them being position i = nk - nq + r, and
 *   out[row][hq*d + j] = sum_t softmax_t(scale * q_row,hq . k_hk,t) v_hk,t,j   over the visible t,
 * hk = hq / (Hq / Hkv).  A row that sees nothing (nk < nq) gets 0.  With nq == nk this is a whole
 * prompt (q, k and v may be column blocks of one QKV buffer), with nq < nk a piece of one against
 * what was before it (fg_kv_read_q4_ragged).  q, out: device fp16, q_rows rows, q_stride and
 * out_stride elements apart (>= Hq*d, multiples of 8); k, v: device fp16, kv_rows rows, kv_stride
 * elements apart (>= Hkv*d, a multiple of 8).  q_off, kv_off: device int32 [nseq+1], not
 * decreasing, within 0 .. q_rows and 0 .. kv_rows; checked on the device (the output of a sequence
 * that does not fit stays as it was, and fg_check_device_error() returns FG_ERR_CAPACITY).  Rows
 * of out outside every sequence stay as they were.  d in {64, 128}; Hq a multiple of Hkv, at most
 * 65536; rows of out that overlap rows of q, k or v are refused.  Values of keys that a row does not see never reach it,
 * not even infinities and NaN.  nseq == 0 or q_rows == 0 is a no-op; with kv_rows == 0, k and v may
 * be NULL.  The pages' prompts have one length and no window; no counterpart. */
int fg_prefill_attn_window(const uint16_t* q, int64_t q_stride, int32_t q_rows,
                           const int32_t* q_off, const uint16_t* k, const uint16_t* v,
                           int64_t kv_stride, int32_t kv_rows, const int32_t* kv_off, int32_t nseq,
                           int32_t Hq, int32_t Hkv, int32_t d, int32_t window, int32_t sinks,
                           float scale, uint16_t* out, int64_t out_stride, void* stream);

/* ---------------------------------------------------------------------- LayerNorm */

/* y[rows][h] = (x - mean) / sqrt(var + eps) * gamma + beta, fp32 statistics (population
 * variance), fp16 in and out.  x, gamma, beta, y: device fp16 (gamma, beta [h]); h % 64
 * == 0, h <= 16384, eps > 0; rows == 0 is a no-op.  The pages name no normalisation: this
 * is the pre-LN of the OPT decoder layer the workloads specify (LN1 before attention, LN2
 * before the MLP); the pages have no counterpart of the call itself. */
int fg_layernorm(const uint16_t* x, int64_t rows, int32_t h, const uint16_t* gamma,
                 const uint16_t* beta, float eps, uint16_t* y, void* stream);

/* ---------------------------------------------------------------------- layer */

/* Prefill of one layer over a block of m GPU batches of g sequences each, prompt length s:
 * x, y: device fp16 [m][g][s][h] (y may alias x).  GPU batch k is processed in full
 * (M = g*s rows per GEMM) before batch k+1; its K/V are quantised into `kv` positions
 * 0..s-1 of sequences k*g .. k*g+g-1.  kv->B == g*m, s <= kv->cap.  When g*s > 128 the
 * call first restores the layer's four weight matrices to fp16 in `ws` (once for the m GPU
 * batches) and its GEMMs read those instead of restoring the codes tile by tile; the results
 * are those of the 4-bit weights either way.
 * ws: device scratch of at least fg_layer_workspace_bytes(dims, g, m, s) bytes.
 * [FlexGen paper explainer, Algorithm 1 (a layer over every GPU batch of the block);
 *  Figure 2 (prefill builds the cache); FlexGen review, "4-bit 압축은 정수 연산 가속과
 *  같은가": weights restored to FP16 before compute] */
int fg_layer_prefill(const fg_dims* dims, const fg_layer* layer, fg_kvcache* kv,
                     const uint16_t* x, uint16_t* y, int32_t g, int32_t m, int32_t s,
                     void* ws, size_t ws_bytes, void* stream);

/* One decode step of one layer for the whole block: x, y: device fp16 [m][g][h] = [B][h]
 * (y may alias x), one launch per operation with M = B rows so each weight is read once
 * per step.  pos is the cache length before the step: the new K/V are appended at pos
 * and attention runs over positions 0..pos.  pos + 1 <= kv->cap.
 * [FlexGen paper explainer, Algorithm 1 and Figure 2] */
int fg_layer_decode(const fg_dims* dims, const fg_layer* layer, fg_kvcache* kv,
                    const uint16_t* x, uint16_t* y, int32_t g, int32_t m, int32_t pos,
                    void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes for fg_layer_prefill with prompts up to s_max and for fg_layer_decode
 * with caches up to s_max positions (the larger of the two uses): per GPU batch of g
 * sequences the LayerNorm output, the [g*s][3h] QKV, the attention output, h1 and the
 * [g*s][f] FFN activation, plus GEMM split-K partials, the layer's weights restored to fp16
 * for a prefill of more than 128 rows (2*(4h^2 + 2hf) bytes) and, for decode over the whole
 * block of g*m sequences, the split-sequence attention partials.  Returns 0 for invalid dims
 * or g, m, s_max <= 0.  A pure host computation (no CUDA call).
 * [FlexGen paper explainer, "Compute Schedule": a layer runs over every GPU batch of the
 *  block, so the scratch is sized by g, m and the sequence length, not by the stack] */
size_t fg_workspace_bytes(const fg_dims* dims, int32_t g, int32_t m, int32_t s_max);
/* The same value as fg_workspace_bytes, under the name of the layer calls it sizes. */
size_t fg_layer_workspace_bytes(const fg_dims* dims, int32_t g, int32_t m, int32_t s_max);

/* ---------------------------------------------------------------------- runtime */

const char* fg_status_string(int status);
const char* fg_last_error(void);
/* Synchronise `stream`, read and clear the device error words: FG_OK, FG_ERR_TIMEOUT, or
 * FG_ERR_CAPACITY when a call met lengths, positions or offsets in a device array that do not
 * fit its buffers.  fg_last_error() names the kernels of either kind; FG_ERR_TIMEOUT is the status
 * when both happened. */
int fg_check_device_error(void* stream);

/* Per-kernel timing with CUDA events recorded around every launch on its stream.
 * kind: one of FG_K_* below.  fg_prof_query synchronises the recorded events and
 * returns the launch count, total milliseconds and the algorithmic work of those
 * launches (bytes for HBM-bound kinds, flops for the GEMM and prefill attention). */
enum {
  FG_K_QUANT = 0, FG_K_DEQUANT = 1, FG_K_GEMM = 2, FG_K_GEMM_REDUCE = 3,
  FG_K_KV_APPEND = 4, FG_K_DECODE_ATTN = 5, FG_K_DECODE_COMBINE = 6,
  FG_K_PREFILL_ATTN = 7, FG_K_LAYERNORM = 8,
  FG_K_GEMM_STREAM = 9,   /* the weight-streaming GEMM (M <= 128): work counted in bytes */
  FG_K_DECODE_ATTN_TOPK = 10,   /* both kernels of the top-K attention: bytes */
  FG_K_GEMM_PAIR = 11,   /* the tiled GEMM on CTA pairs (many tokens): flops */
  FG_K_GEMM_PAIR_F16W = 12,   /* the CTA-pair GEMM on weights restored to fp16 (layer
                                 prefill): flops */
  /* work of the calls whose extents the host does not see is counted for the most that their
   * host arguments allow: every row of the buffers, sequences that fill the cache (of which
   * decode attention counts the window and the first positions).  A rate made from it is an upper
   * bound, near the truth for full buffers only */
  FG_K_KV_READ = 13,             /* fg_kv_read_q4_ragged: bytes */
  FG_K_DECODE_ATTN_WINDOW = 14,  /* fg_decode_attn_q4kv_window, all its kernels: bytes */
  FG_K_PREFILL_ATTN_WINDOW = 15, /* fg_prefill_attn_window: bytes of its rows (not its flops: how
                                    many pairs are visible stands in the device arrays) */
  FG_K_ROPE = 16,                /* fg_rope: bytes */
  FG_K_ATTN_PAGED = 17,          /* fg_attn_q4kv_paged, all its kernels: bytes */
  FG_K_ATTN_WEIGHTS = 18,        /* fg_attn_weights_q4_paged: bytes */
  FG_K_KV_EVICT = 19,            /* fg_kv_evict_q4_paged, both kernels: bytes */
  FG_K_COUNT = 20
};
int fg_prof_enable(int on);
int fg_prof_reset(void);
int fg_prof_query(int kind, int64_t* launches, double* ms, double* work);
const char* fg_kernel_name(int kind);

#ifdef __cplusplus
}
#endif
#endif /* FG_H_ */
