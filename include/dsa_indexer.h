/*
 * dsa_indexer.h -- C ABI of the GB300 (sm_103a) DSA indexer paged
 * MQA-logits library, libdsa_indexer.so.
 *
 * The operation.  For every row r (a decode request, or a prefill query
 * token) and every cached key position t in [0, W*64):
 *
 *     out[r, t] = scale(t) * sum_{h<64} w[r, h] * max(0, q[r, h, :] . k(t))
 *                                                      if t <  seqlens[r]
 *     out[r, t] = -inf                                 if t >= seqlens[r]
 *
 * The per-head dot, the ReLU, the per-head weights and the per-position
 * scale are the ingredients listed on "The Dispatch Wire: Connecting a
 * Triton Indexer Kernel to Production Inference", section "The Road to This
 * Message".  The -inf rule is the "inf-pattern" criterion of "The Final Gate:
 * Validating a Custom Triton Indexer Kernel Before Production Deployment",
 * section "What the Test Output Reveals".  The output shape is fixed
 * ([rows, W*64]) and work past seqlens[r] is skipped inside the kernel, so a
 * call can be captured in a CUDA graph and replayed with new lengths and
 * block tables: "The Moment the Context-Length Tax Vanished: Committing the
 * O(actual) Triton Indexer", section "The Commit: Engineering as Narrative".
 *
 * The key cache.  Keys live in physical pages of 64 positions x D = 128
 * values.  Position t of row r is slot (t % 64) of physical page
 * block_table[r][t / 64] (the page table of "The Final Gate ...", section
 * "Assumptions and Knowledge Required").  Page p starts at
 * (char*)kcache + p * page_stride_bytes and holds its 64 key rows
 * position-major (D values per position, contiguous):
 *   DSA_KV_FP8_E4M3  OCP e4m3 ("e4m3fn") bytes, 128 bytes per position.  The
 *                    fused page of "The Dispatch Wire ...", section "The
 *                    Reasoning and Decision-Making", is 8,448 bytes: 8,192
 *                    bytes of keys then 64 fp32 scales, i.e.
 *                    page_stride_bytes = 8448 and kscale = kcache + 8192.
 *   DSA_KV_BF16      bf16, 256 bytes per position, 16,384 bytes per page,
 *                    no quantisation ("The Dispatch Decision: Wiring a Triton
 *                    Kernel into Production", section "The Problem That Led
 *                    Here"); pass kscale = NULL for scale 1.
 * kscale, when not NULL, is the address of page 0's 64 fp32 scales; page p's
 * are at (char*)kscale + p * page_stride_bytes.  NULL means scale(t) = 1.
 *
 * Common rules for the indexer entry points.
 *   Memory.   Every pointer except `stream` is a DEVICE pointer owned by the
 *             caller (the varlen prefill's request offsets are host data).
 *             The library allocates nothing, never synchronises and
 *             launches one kernel per call on `stream` (a cudaStream_t;
 *             NULL = legacy default stream); the top-k calls launch two, the
 *             varlen prefill one per 128 requests.  All calls are legal inside
 *             stream capture.  Every kernel is launched with
 *             programmatic dependent launch allowed: its set-up may overlap
 *             the tail of the previous kernel in the stream, but it reads no
 *             argument array before that kernel has completed.
 *   Shapes.   Only H = 64, D = 128 and page_size = 64 are supported
 *             (DSA_ERR_UNSUPPORTED otherwise).  W >= 1.  Rows may be 0 (no
 *             launch, DSA_OK).
 *   Layouts.  q: bf16 [rows, 64, 128] contiguous.  w: fp32 [rows, 64]
 *             contiguous.  block_table: int32, row r at
 *             block_table + r * bt_stride, W entries used (bt_stride = 0
 *             means every row shares row 0; otherwise bt_stride >= W).
 *             seqlens: int32 [rows].  out: fp32, row r at
 *             out + r * out_stride, W*64 entries written (out_stride >=
 *             W*64).
 *   Alignment. q, kcache and out 16-byte aligned; kscale 16-byte aligned;
 *             page_stride_bytes a multiple of 16 and at least the key bytes
 *             of a page (8,192 fp8, 16,384 bf16); out_stride a multiple of
 *             4 (DSA_ERR_MISALIGNED otherwise).
 *   Host errors.  Invalid arguments are reported by the return value and
 *             nothing is launched.  A launch failure returns DSA_ERR_CUDA.
 *   Data errors (found by the kernel; never a trap or a fault):
 *             - seqlens[r] > W*64: the whole row is written NaN, status
 *               DSA_ERR_BAD_SEQLEN;
 *             - a block-table entry outside [0, num_pages) that a valid
 *               position needs: that page's valid positions are NaN, status
 *               DSA_ERR_BAD_PAGE;
 *             - an internal wait that does not complete within its bound:
 *               the affected outputs are NaN, status DSA_ERR_TIMEOUT.
 *             The status is stored with atomicMax into *dev_status when
 *             dev_status is not NULL; the library never clears it (zero it
 *             before the call to read a fresh status).  seqlens[r] <= 0 is
 *             not an error: the row is all -inf.  Entries of the block table
 *             at or past ceil(seqlens[r] / 64) are never used as page ids and
 *             may hold any value (decode may load the first entries of a row
 *             before it knows the row's length; all W entries of every row
 *             must therefore be readable memory).
 */
#ifndef DSA_INDEXER_H
#define DSA_INDEXER_H

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_INDEXER_ABI_VERSION 1

typedef enum {
  DSA_KV_FP8_E4M3 = 0,
  DSA_KV_BF16 = 1
} dsa_kv_dtype_t;

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,
  DSA_ERR_UNSUPPORTED = 2,
  DSA_ERR_MISALIGNED = 3,
  DSA_ERR_CUDA = 4,
  DSA_ERR_TIMEOUT = 5,
  DSA_ERR_BAD_PAGE = 6,
  DSA_ERR_BAD_SEQLEN = 7,
  DSA_ERR_BAD_POSITION = 8
} dsa_status_t;

/*
 * Decode: B requests, one query token each.  Row b uses q[b], w[b], block
 * table row b and length seqlens[b].  The grid is fixed by (B, W) alone, so
 * the launch does not depend on the lengths: "The Dispatch Wire ...",
 * section "The Reasoning and Decision-Making" (one program per request and
 * page, early exit past the request's length).
 */
int dsa_indexer_logits_decode(const void* q, const float* w,
                              const void* kcache, const void* kscale,
                              long long page_stride_bytes, int num_pages,
                              int kv_dtype, const int* block_table,
                              long long bt_stride, const int* seqlens, int B,
                              int H, int D, int page_size, int W, float* out,
                              long long out_stride, int* dev_status,
                              void* stream);

/*
 * Prefill: n_q query tokens.  Query i uses q[i], w[i], block-table row i
 * (bt_stride = 0: all queries share row 0, the one-request prefill of "The
 * Dispatch Decision ...", section "The Problem That Led Here") and length
 * seqlens[i] = its causal limit + 1.  Keys are read page by page from the
 * cache: no gathered copy is made.  A shared row (bt_stride = 0) runs the
 * query-tile kernel, which reuses each key tile for four query tokens (fp8
 * keys: the query is split into two e4m3 terms, as in decode).  Per-query
 * rows (bt_stride >= W: several requests in one call, or multi-token
 * decode) run the decode kernel with one row per query token; there
 * n_q <= 65535 (DSA_ERR_UNSUPPORTED otherwise).  Range (query-tile kernel,
 * bf16 keys): half of the heads
 * take their ReLU as a saturating multiply by 2^-64 with the weight scaled
 * by 2^64, so results are defined for |w[i, h]| < 2^64 and per-head dots
 * |q . k| < 2^64.
 */
int dsa_indexer_logits_prefill(const void* q, const float* w,
                               const void* kcache, const void* kscale,
                               long long page_stride_bytes, int num_pages,
                               int kv_dtype, const int* block_table,
                               long long bt_stride, const int* seqlens,
                               int n_q, int H, int D, int page_size, int W,
                               float* out, long long out_stride,
                               int* dev_status, void* stream);

/*
 * Prefill of several requests in one call, with a table row per request:
 * the query tokens of request b are rows [cu_q[b], cu_q[b+1]) of q, w,
 * seqlens and out, and read the keys through block-table row b
 * (block_table + b * bt_stride; bt_stride >= W, or 0 for one row shared by
 * all requests).  Query i may see the positions t < seqlens[i] (its causal
 * limit + 1), as in dsa_indexer_logits_prefill; positions past it hold
 * -inf.  No gathered per-query copy of the keys is made ("The Dispatch
 * Decision ...", section "The Problem That Led Here": the materialised
 * [query tokens, pages, ...] gather is what ran out of memory).
 *
 * cu_q is a HOST array of n_req + 1 offsets: cu_q[0] = 0, non-decreasing
 * (DSA_ERR_INVALID_ARG otherwise, checked before any launch); n_q =
 * cu_q[n_req] rows in all.  The requests' query tiles run in one launch of
 * the query-tile kernel of dsa_indexer_logits_prefill (up to 128 requests a
 * launch; more run as further launches, in request order, on `stream`),
 * each tile reading its own request's table row, so requests of many tokens
 * reuse each key tile four times; requests of one or a few tokens are
 * better served by per-query rows.  Other arguments, layouts, alignment,
 * range and device errors as for dsa_indexer_logits_prefill.  DSA_ERR_CUDA
 * from a launch may leave the earlier groups of requests launched.
 */
int dsa_indexer_logits_prefill_varlen(const void* q, const float* w, const void* kcache,
                                      const void* kscale, long long page_stride_bytes,
                                      int num_pages, int kv_dtype, const int* block_table,
                                      long long bt_stride, const int* cu_q, int n_req,
                                      const int* seqlens, int H, int D, int page_size, int W,
                                      float* out, long long out_stride, int* dev_status,
                                      void* stream);

/* How the top-k decode computes its selection (dsa_indexer_topk_decode_form). */
typedef enum {
  DSA_TOPK_AUTO = 0,      /* the library's choice (today: two passes) */
  DSA_TOPK_TWO_PASS = 1,  /* the logits into the workspace, then a selection kernel */
  DSA_TOPK_FUSED = 2      /* selection in the decode epilogue, then a merge kernel */
} dsa_topk_form_t;

/*
 * Decode with top-k selection: for every request b, the k_top positions
 * t < seqlens[b] with the largest logits (the positions sparse attention
 * then reads), instead of the [B, W*64] logits.  topk_idx: int32, row b at
 * topk_idx + b * topk_stride (topk_stride >= k_top), the selected positions
 * in increasing order; a row with L <= k_top valid positions takes all of
 * them and pads with -1.  topk_val (nullable): their logits, same layout,
 * -inf for the padding.  Equal logits at the k-th place are taken in
 * position order.  workspace: device fp32 buffer of at least
 * B * W * 64 entries (16-byte aligned), owned by the caller; no -inf fill
 * is written anywhere.  Two kernel launches on `stream`, in one of two
 * forms (this entry point takes the two-pass one; the caller chooses with
 * dsa_indexer_topk_decode_form):
 *   two passes: the decode kernel writes the logits of the valid positions
 *     into the workspace, then the selection kernel (a cluster of two CTAs
 *     per request while 2 * B CTAs fit in one wave of one CTA per SM, else
 *     one CTA per request: a histogram pass, the k-th value's bin collected
 *     and ranked, an in-order write) reads them;
 *   fused: the decode kernel keeps the logits in shared memory, chunk by
 *     chunk of up to 32 pages of a row, and writes each chunk's best
 *     min(k_top, n) positions with their logits to the workspace; a merge
 *     kernel then selects each request's best among them.  No logit of the
 *     call is written to global memory.  It applies when k_top <= 2048 (a
 *     chunk: for k_top >= 2048 every chunk keeps all its positions and the
 *     merge does all the selecting), the
 *     decode takes its balanced form (W > 64 and B <= 384) and the
 *     workspace holds 4 * ceil((B + 1) / 4) + (C + B + ceil(B * W / 32)) *
 *     (4 + 2 * k_top) floats, C being the decode's persistent CTAs (two per
 *     SM).
 * Both forms take the same positions and return the same logits, bit for
 * bit: the logits come from the same arithmetic and the order is total.
 * Other arguments, checks and data errors as for dsa_indexer_logits_decode;
 * an over-long row selects nothing (all -1) and reports DSA_ERR_BAD_SEQLEN.
 */
int dsa_indexer_topk_decode(const void* q, const float* w, const void* kcache,
                            const void* kscale, long long page_stride_bytes, int num_pages,
                            int kv_dtype, const int* block_table, long long bt_stride,
                            const int* seqlens, int B, int H, int D, int page_size, int W,
                            int k_top, int* topk_idx, float* topk_val, long long topk_stride,
                            float* workspace, long long workspace_floats, int* dev_status,
                            void* stream);

/*
 * dsa_indexer_topk_decode with the form chosen by the caller (a
 * dsa_topk_form_t; DSA_ERR_INVALID_ARG for another value).  DSA_TOPK_FUSED
 * where the fused form does not apply returns DSA_ERR_UNSUPPORTED before
 * any launch.  The top-k is the logits' consumer: "The Dispatch Decision
 * ...", section "The Problem That Led Here".
 */
int dsa_indexer_topk_decode_form(const void* q, const float* w, const void* kcache,
                                 const void* kscale, long long page_stride_bytes, int num_pages,
                                 int kv_dtype, const int* block_table, long long bt_stride,
                                 const int* seqlens, int B, int H, int D, int page_size, int W,
                                 int k_top, int* topk_idx, float* topk_val, long long topk_stride,
                                 float* workspace, long long workspace_floats, int* dev_status,
                                 int form, void* stream);

/*
 * dsa_indexer_topk_decode without a caller workspace, for callers that
 * cannot allocate device memory for it (an allocator that is not theirs to
 * call, a memory pool fixed at start-up, code running inside another
 * library's allocation-free hot path).  The logits go to a fixed device
 * array of the library (24 Mi floats, 96 MiB per device); the call itself
 * allocates nothing.  With lazy module loading (the CUDA default) the array
 * is reserved on a device when this entry point is first used there; under
 * CUDA_MODULE_LOADING=EAGER every process that loads the library reserves
 * it on every device it creates a context on, whether or not it calls this.
 * B * W * 64 must not exceed 24 Mi (DSA_ERR_UNSUPPORTED otherwise, checked
 * before any device work).  The array is shared: calls on one device must
 * not overlap (use one stream, or order the streams), or they race.  The
 * first call with B > 0 on a device looks up the array's address (which may
 * load its module), so make one such call before capturing one in a CUDA
 * graph.  The pages have no counterpart: this is a convenience of the
 * library.  Every other argument is checked, and every result written, as
 * by dsa_indexer_topk_decode.
 */
int dsa_indexer_topk_decode_static(const void* q, const float* w, const void* kcache,
                                   const void* kscale, long long page_stride_bytes,
                                   int num_pages, int kv_dtype, const int* block_table,
                                   long long bt_stride, const int* seqlens, int B, int H, int D,
                                   int page_size, int W, int k_top, int* topk_idx,
                                   float* topk_val, long long topk_stride, int* dev_status,
                                   void* stream);

/*
 * Key-cache store: writes n new key rows into their cache slots, in the
 * page layouts above (the step before the indexer: its keys come from this
 * cache).  k: bf16 [n, 128], 16-byte aligned.  slot_mapping: int32 [n],
 * entry i = page * 64 + slot of row i; a negative entry skips the row.
 * kcache: the pool, page p at (char*)kcache + p * page_stride_bytes.
 *   DSA_KV_FP8_E4M3  page_stride_bytes >= 8448: the slot's 128 e4m3 codes
 *                    at page + slot * 128 and its fp32 scale s at
 *                    page + 8192 + slot * 4, with s = max_d |k[i, d]| / 448
 *                    (1 for an all-zero row) and code_d = e4m3(k[i, d] / s)
 *                    rounded to nearest even and saturated to +-448, every
 *                    step in fp32.  The pages give no quantisation rule; this
 *                    one maps the row's largest |k| to e4m3's largest finite
 *                    value, so k ~ code * s.
 *   DSA_KV_BF16      page_stride_bytes >= 16384: the row's 256 bytes at
 *                    page + slot * 256.
 * Host errors as for the indexer calls (D = 128, page_size = 64; k and
 * kcache 16-byte aligned, page_stride_bytes a multiple of 16).  A slot at or
 * past num_pages * 64 is skipped and DSA_ERR_BAD_PAGE stored into
 * *dev_status.  One kernel launch on `stream`; nothing is allocated.  Rows
 * with the same slot race (the last writer is unspecified).
 */
int dsa_kcache_store(const void* k, const int* slot_mapping, int n, void* kcache,
                     long long page_stride_bytes, int num_pages, int kv_dtype,
                     int D, int page_size, int* dev_status, void* stream);

/*
 * ---- Around the sparse attention: norm + rotation, latent cache, attention --
 *
 * The common rules above hold (device pointers, no allocation, no
 * synchronisation, programmatic dependent launch, host errors by return
 * value before any launch, data errors by atomicMax into *dev_status).
 * Strides are in elements of the array they belong to.  A rope_table is fp32
 * [max_pos, rot] contiguous: row t holds rot/2 cosines, then rot/2 sines, of
 * the angles of position t.  A rotation turns the pair (a, b) into
 * (a cos - b sin, b cos + a sin); pair i is (x[i], x[i + rot/2]), or
 * (x[2i], x[2i + 1]) when `interleaved` is not 0.
 */
typedef enum { DSA_BF16 = 0, DSA_FP16 = 1, DSA_FP32 = 2 } dsa_dtype_t;
typedef enum { DSA_NORM_NONE = 0, DSA_NORM_RMS = 1, DSA_NORM_LAYER = 2 } dsa_norm_t;

/*
 * Per-head norm of queries and keys, with the position rotation in the same
 * pass.  Row (t, h) of q starts at q + t * q_token_stride + h *
 * q_head_stride and holds D contiguous values (k alike); the results go to
 * q_out and k_out, which may be q and k themselves (same strides) but must
 * not overlap them in any other way.  Per row, every step in fp32 with one
 * rounding at the end:
 *   DSA_NORM_RMS    y = x * rsqrt(mean(x^2) + eps) * weight + bias
 *   DSA_NORM_LAYER  y = (x - mean) * rsqrt(var + eps) * weight + bias
 *   DSA_NORM_NONE   y = x (weights and biases unused)
 * then values [rot_offset, rot_offset + rot_dims) are rotated by
 * positions[t].  weight, bias: fp32 [D] per side, nullable (1 and 0).
 * positions NULL: no rotation.  Hq or Hk may be 0 (that side's pointers are
 * not used); sides of different norms take a call each.  8 <= D <= 256, a multiple of 8; rot_dims a multiple of 16
 * (interleaved: of 8), rot_offset of 8 (DSA_ERR_UNSUPPORTED).  Arrays and
 * rows 16-byte aligned, weights, biases and rope_table too
 * (DSA_ERR_MISALIGNED).  A position
 * outside [0, max_pos) is a data error: that token's rows are NaN, status
 * DSA_ERR_BAD_POSITION.
 */
int dsa_qk_norm_rope(const void* q, long long q_token_stride, long long q_head_stride, int Hq,
                     const void* k, long long k_token_stride, long long k_head_stride, int Hk,
                     int T, int D, int dtype, int norm, const float* q_weight,
                     const float* k_weight, const float* q_bias, const float* k_bias, float eps,
                     const int* positions, const float* rope_table, int max_pos, int rot_dims,
                     int rot_offset, int interleaved, void* q_out, long long qo_token_stride,
                     long long qo_head_stride, void* k_out, long long ko_token_stride,
                     long long ko_head_stride, int* dev_status, void* stream);

/*
 * The latent cache: per token one latent vector (latent_dim = 512 values)
 * and one rotated part (rope_dim = 64 values) that all heads share, in pages
 * of 64 tokens.
 *   DSA_KV_BF16      token s of a page: 576 bf16 values at page + s * 1152
 *                    (page_stride_bytes >= 73,728).
 *   DSA_KV_FP8_E4M3  512 e4m3 codes at page + s * 512, the rotated part as 64
 *                    bf16 at page + 32768 + s * 128, four fp32 scales at page
 *                    + 40960 + s * 16, one per 128 latent values
 *                    (page_stride_bytes >= 41,984).  Value = code * scale.
 *
 * Store: n new tokens into their slots (slot_mapping as for
 * dsa_kcache_store: page * 64 + slot, negative = skip, past the pool =
 * skipped with DSA_ERR_BAD_PAGE, equal slots race).  latent: bf16, row i at
 * latent + i * latent_stride; rope alike.  norm_weight (fp32 [512],
 * nullable): the latent is first normalised, c * rsqrt(mean(c^2) + eps) *
 * norm_weight.  positions (nullable): the rotated part is turned by
 * positions[i] (rope_table's rot = 64).  Every step is fp32.  The fp8 scale
 * of a group is 2^e with the smallest e for which its largest finite
 * magnitude is at most 448 * 2^e (e >= -126; 1 for a group of zeros), the codes
 * round to nearest even, infinities become +-448 and NaN stays NaN; a power
 * of two keeps code * scale exact in bf16.  A bad position makes the rotated
 * part NaN, status DSA_ERR_BAD_POSITION.
 */
int dsa_latent_store(const void* latent, long long latent_stride, const void* rope,
                     long long rope_stride, int n, int latent_dim, int rope_dim,
                     const float* norm_weight, float eps, const int* positions,
                     const float* rope_table, int max_pos, int interleaved,
                     const int* slot_mapping, void* cache, long long page_stride_bytes,
                     int num_pages, int kv_dtype, int page_size, int* dev_status, void* stream);

/*
 * Load: ranges of tokens back as packed bf16 rows of 576 values (latent,
 * then rotated part).  Output row i (out + i * out_stride) belongs to the
 * request r with cu_rows[r] <= i < cu_rows[r + 1] and holds its position
 * starts[r] + i - cu_rows[r] (starts NULL: 0), read through block-table row
 * r.  cu_rows: DEVICE int32 [n_req + 1], non-decreasing.  Rows i < n of no
 * request are zeros.  An fp8 value is code * scale rounded to bf16 (exact
 * for the scales that the store writes).  A position outside [0, W * 64)
 * gives a NaN row and DSA_ERR_BAD_SEQLEN, a page outside the pool a NaN row
 * and DSA_ERR_BAD_PAGE.
 */
int dsa_latent_load(const void* cache, long long page_stride_bytes, int num_pages, int kv_dtype,
                    int page_size, const int* block_table, long long bt_stride, int W,
                    const int* starts, const int* cu_rows, int n_req, int n, int latent_dim,
                    int rope_dim, void* out, long long out_stride, int* dev_status, void* stream);

/*
 * Attention over the latent cache in the absorbed form.  For row r (a decode
 * request, or a prefill query token) and head h < H:
 *     s[t] = scale * (q_latent[r, h] . c[t] + q_rope[r, h] . k[t])
 *     out[r, h, :] = sum_t softmax(s)[t] c[t],   lse[r, h] = log sum_t exp(s[t])
 * with c[t] the 512 latent values and k[t] the rotated part of position t of
 * the row's block-table row.  The visible positions are t < seqlens[r]
 * (idx NULL), or those of the row's selection list: entries idx[r * idx_stride
 * + j], j < min(k, seqlens[r]), k >= 1, that are not negative and below seqlens[r]
 * (the lists that the top-k calls write: valid entries first, then -1; an
 * entry that is repeated counts as often).  A row without a visible position
 * gives zeros and lse = -inf.
 *   q_latent  bf16 [rows, H, 512], q_rope bf16 [rows, H, 64] through their
 *             row and head strides, values contiguous; 1 <= H <= 128.
 *   out       bf16 [rows, H, 512] through its strides; lse fp32 [rows, H]
 *             contiguous, nullable.
 *   block_table, bt_stride, seqlens  as for the indexer calls (bt_stride = 0:
 *             all rows share row 0, a prompt of one request; prompts of several
 *             requests repeat a request's row for each of its query tokens).
 *   workspace fp32, at least dsa_latent_attention_workspace() floats for the
 *             current device, 16-byte aligned; calls that may overlap need
 *             one each.  What another call or kernel writes to it meanwhile
 *             leaves the results undefined, without an access out of range;
 *             where it is noticed the status is DSA_ERR_INVALID_ARG.
 * The softmax and all sums are fp32; the weights of the value product are
 * rounded to bf16.  With an fp8 cache latent queries, weights and tokens are
 * fp16 under scales of their own (a power of two per head, one per token from
 * its four scales, groups of zeros left out): exact for scales that are powers
 * of two within 2^22 of the token's largest; another scale is rounded as a
 * ratio and so are its products (2^-11 each); what lies further down is rounded
 * to 2^-32 of the largest scale or to 2^-125, and a group whose scale is 2^-32
 * of it or less counts as zeros.  Weights round by 2^-11 of themselves, and by
 * 2^-31 of the row's largest weight * scale where theirs is below 2^-20 of it.
 * A head's latent queries are exact down to 2^-29 of its largest, but for steps
 * of 2^-125 and of 2^-85 of its largest rotated one.  Two kernel launches, whose
 * shapes depend on rows and H, not on lengths, lists or tables: a captured call
 * may be replayed with others of those.
 * Data errors: seqlens[r] > W * 64 gives a NaN row and DSA_ERR_BAD_SEQLEN; a
 * visible position without a page in the pool a NaN row and
 * DSA_ERR_BAD_PAGE; a wait that runs out DSA_ERR_TIMEOUT and NaN rows.
 * rows * (idx ? ceil(k / 64) : W), W * 64 and num_pages * 64 must be below
 * 2^31 (DSA_ERR_UNSUPPORTED).
 */
int dsa_latent_attention(const void* q_latent, long long ql_row_stride, long long ql_head_stride,
                         const void* q_rope, long long qr_row_stride, long long qr_head_stride,
                         int rows, int H, int latent_dim, int rope_dim, float scale,
                         const void* cache, long long page_stride_bytes, int num_pages,
                         int kv_dtype, int page_size, const int* block_table, long long bt_stride,
                         int W, const int* seqlens, const int* idx, long long idx_stride, int k,
                         void* out, long long out_row_stride, long long out_head_stride,
                         float* lse, float* workspace, long long workspace_floats,
                         int* dev_status, void* stream);

/* Floats of workspace that dsa_latent_attention needs on the current device
 * (two partial rows of 64 heads and a split record per SM); -1 when there is
 * no device. */
long long dsa_latent_attention_workspace(void);

/* A static, human-readable name for a status code. */
const char* dsa_status_string(int status);

/* DSA_INDEXER_ABI_VERSION of the loaded library. */
int dsa_indexer_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_INDEXER_H */
