/*
 * colibri_attn.h - C ABI of the attention operators of a pre-norm decoder
 * block on a GB300 (sm_103a): what stands between two MoE layers of
 * colibri_moe.h.
 *
 *   append   queries and keys normalised per head, rotated to their
 *            positions, keys and values written to a paged cache: one pass
 *   prompt   attention of packed sequences of different lengths, grouped
 *            heads, causal or full, over the prompt's own rows or over pages
 *   decode   attention of one row per sequence over a paged cache, with a
 *            prefix that all sequences share read once
 *
 * No handle: every call works on the caller's buffers, allocates nothing,
 * runs on the current device ordered on `stream` (a cudaStream_t, NULL = the
 * legacy default stream) and returns without waiting, so it can be captured
 * into a CUDA graph (but for colibri_attention_check, which waits).  Argument checks run on the host before any CUDA call:
 * INVALID_ARG for pointers, sizes, strides and alignment that cannot be right,
 * UNSUPPORTED for shapes that this build does not run.  Every device pointer
 * belongs to the current device.  Calls that may overlap on the GPU must not
 * share a workspace; nothing in a workspace outlives its call and it needs no
 * initialisation.
 *
 * Common limits: dtype FP32 or BF16; head_dim 64 or 128; n_q_heads a multiple
 * of n_kv_heads, at most 128 query heads per key head; query head h reads key
 * head h / (n_q_heads / n_kv_heads).  Rows and heads start on 16-byte
 * boundaries: base pointers 16-byte aligned, strides multiples of 16 bytes.
 * Strides are in elements; a head's head_dim elements are contiguous.
 */
#ifndef COLIBRI_ATTN_H
#define COLIBRI_ATTN_H

#include "colibri_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Keys and values.  Element c of row r of head h of page p is at
 *   p * page_stride + h * head_stride + r * row_stride + c
 * of k and of v, so both [pages, heads, rows, dim] and [pages, rows, heads,
 * dim] storage (and views of larger tensors) are described by their strides.
 * page_size is a power of two from 8 to 65536 for a paged cache.  Packed keys
 * without pages (colibri_seqs_t.page_table NULL) are one page of page_size rows,
 * the keys of sequence b being rows seq_start[b] .. seq_start[b + 1] - 1.
 */
typedef struct {
    void* k;               /* device */
    void* v;               /* device */
    int64_t page_stride;
    int64_t head_stride;
    int64_t row_stride;
    int32_t num_pages;
    int32_t page_size;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t dtype;         /* colibri_dtype_t of k, v and of the call's other tensors */
} colibri_kv_pages_t;

/*
 * The sequences of a call.  Rows seq_start[b] .. seq_start[b + 1] - 1 of the
 * call's row tensors belong to sequence b; seq_start NULL means one row per
 * sequence (n_rows == n_seqs, row b is sequence b).  kv_len[b] counts the
 * sequence's keys including this call's rows, so its row i of n is at
 * position kv_len[b] - n + i; kv_len NULL means kv_len[b] = n.  Position t is
 * row t % page_size of page page_table[b * table_stride + t / page_size].
 * n_seqs may be 0 (a batch of nothing but padding): arrays without entries may
 * then be NULL, and outputs are left as they were.
 *
 * The arrays are read on the device, so their values are not checked by the
 * call; whatever they hold, every access stays in bounds: seq_start is cut to
 * 0 .. n_rows, rows at or behind seq_start[n_seqs] belong to no sequence and
 * their outputs are left as they were, a kv_len beyond the page table is cut
 * to it (and to 2^31 - 2^20) and a negative one is 0, a page id outside
 * 0 .. num_pages - 1 is never written and reads as rows of zeros.  They must
 * not change while a call that reads them runs.
 */
typedef struct {
    const int32_t* seq_start;    /* [n_seqs + 1] device, or NULL */
    const int32_t* kv_len;       /* [n_seqs] device, or NULL */
    const int32_t* page_table;   /* [n_seqs, table_stride] device, or NULL */
    int32_t n_seqs;
    int32_t n_rows;              /* rows of q, k, v and o */
    int32_t table_stride;        /* entries of a sequence's row of page_table */
} colibri_seqs_t;

/*
 * Rotary positions.  Pair i < rot_dim / 2 of a head at position t turns by
 * the angle t * freq[i]: (a, b) -> mscale * (a cos - b sin, b cos + a sin).
 * HALF pairs elements i and i + rot_dim / 2, INTERLEAVED 2 i and 2 i + 1; the
 * elements from rot_dim on are left alone.  rot_dim is a multiple of 16 up to
 * head_dim.  The angle is formed in 64-bit fixed point (a fraction of a turn):
 * before float32 rounding it is off by at most 2^-32 + t (freq 2^-55 + 2^-64) turns.
 */
typedef enum { COLIBRI_ROPE_HALF = 0, COLIBRI_ROPE_INTERLEAVED = 1 } colibri_rope_style_t;

typedef struct {
    const double* freq;    /* [rot_dim / 2] device, radians per position */
    int32_t rot_dim;
    int32_t style;         /* colibri_rope_style_t */
    float mscale;          /* factor of cos and sin; 1 where contexts are not scaled */
} colibri_rope_t;

/*
 * colibri_rope_frequencies - freq[i] = theta^(-2 i / rot_dim) on the host,
 * stretched for contexts `factor` times the trained one:
 *   NONE    as above
 *   LINEAR  every frequency divided by factor
 *   NTK     theta * factor^(rot_dim / (rot_dim - 2)) in theta's place
 *           (rot_dim > 2)
 *   YARN    by parts (Peng et al., 2023): pairs that turn at least beta_fast
 *           times in the trained context are kept, those that turn at most
 *           beta_slow times are divided by factor, a linear ramp between;
 *           *mscale = 0.1 ln(factor) + 1
 * *mscale is 1 for the others.  freq [rot_dim / 2] and mscale are host
 * memory.  INVALID_ARG: rot_dim not a positive multiple of 16, theta <= 1,
 * factor < 1, trained <= 0 or beta_fast <= beta_slow or beta_slow <= 0 (YARN).
 */
typedef enum {
    COLIBRI_ROPE_SCALE_NONE = 0,
    COLIBRI_ROPE_SCALE_LINEAR = 1,
    COLIBRI_ROPE_SCALE_NTK = 2,
    COLIBRI_ROPE_SCALE_YARN = 3
} colibri_rope_scaling_t;

colibri_status_t colibri_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling,
                                          double factor, int32_t trained, double beta_fast,
                                          double beta_slow, double* freq, float* mscale);

/*
 * colibri_append_qkv - the rows of a projection made ready for attention:
 *   q' = R(t) (q / sqrt(mean(q^2) + eps) * q_norm)   per head, into q_out
 *   k' = R(t) (k / sqrt(mean(k^2) + eps) * k_norm)   into the cache's keys
 *   v                                                into the cache's values
 * q_norm / k_norm NULL: that norm is left out; rope NULL: no rotation.
 * Arithmetic in float32, rounded once to dtype.
 *   q     [n_rows, n_q_heads, head_dim], q_stride elements from row to row
 *   k, v  [n_rows, n_kv_heads, head_dim]
 *   q_norm, k_norm [head_dim] dtype
 *   q_out [n_rows, n_q_heads, head_dim]; may be q (with the same stride),
 *         otherwise it must not overlap q, k or v, and the cache none of them
 * q, k, v and q_out may be column ranges of one tensor's rows (equal strides).  A row whose
 * position is negative or has no page is not stored in the cache (its q_out is
 * written).  Two rows of one call never name the same place of the cache
 * unless page_table names a page twice.
 */
colibri_status_t colibri_append_qkv(const colibri_kv_pages_t* cache, const colibri_seqs_t* seqs,
                                    const colibri_rope_t* rope, int32_t n_q_heads, const void* q,
                                    int64_t q_stride, const void* k, int64_t k_stride,
                                    const void* v, int64_t v_stride, const void* q_norm,
                                    const void* k_norm, float eps, void* q_out,
                                    int64_t q_out_stride, void* stream);

/*
 * colibri_qk_norm_rope - the same for rows that go to no cache: q' into q_out
 * and k' into k_out (each may be its input, with the same stride; other
 * overlaps as above).
 * seqs->page_table is not read.
 */
colibri_status_t colibri_qk_norm_rope(const colibri_seqs_t* seqs, const colibri_rope_t* rope,
                                      int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t dtype, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* q_norm,
                                      const void* k_norm, float eps, void* q_out,
                                      int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                      void* stream);

/*
 * Rotary positions of several axes, as the tokens of images and video have (time,
 * height, width): the position of row r of the call on axis x is
 * at[x * axis_stride + r], any int32, and pair i of a head turns by
 * at[axis[i] * axis_stride + r] * freq[i].  axis NULL: every pair by axis 0; an axis[i]
 * of n_axes or more counts as n_axes - 1.  n_axes is 1 to 8, axis_stride not negative
 * (0: the axes agree).  Places in the cache follow from the lengths as
 * ever.  Arrays are read on the device.
 */
typedef struct {
    const int32_t* at;     /* [n_axes][n_rows] device */
    const uint8_t* axis;   /* [rot_dim / 2] device, or NULL */
    int64_t axis_stride;
    int32_t n_axes;
} colibri_positions_t;

/*
 * colibri_append_qkv_at, colibri_qk_norm_rope_at - colibri_append_qkv and
 * colibri_qk_norm_rope with positions of their own for the rows (rope given);
 * positions NULL: those that follow from the lengths.
 */
colibri_status_t colibri_append_qkv_at(const colibri_kv_pages_t* cache, const colibri_seqs_t* seqs,
                                       const colibri_rope_t* rope, const colibri_positions_t* positions,
                                       int32_t n_q_heads, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride,
                                       const void* q_norm, const void* k_norm, float eps, void* q_out,
                                       int64_t q_out_stride, void* stream);
colibri_status_t colibri_qk_norm_rope_at(const colibri_seqs_t* seqs, const colibri_rope_t* rope,
                                         const colibri_positions_t* positions, int32_t n_q_heads,
                                         int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                         const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* q_norm, const void* k_norm, float eps, void* q_out,
                                         int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                         void* stream);

/*
 * colibri_attention_prompt - for row i of n of sequence b and query head h
 *   o = sum_j w_j v_j,  w = softmax_j(scale * q . k_j)
 * over the keys j < kv_len[b] (causal == 0) or j <= kv_len[b] - n + i (causal
 * != 0) of the head's key head.  A row that sees no key, or none
 * whose score is above -infinity, gets zeros.
 *   kv    a paged cache (seqs->page_table and kv_len given), or the prompt's
 *         own packed keys (page_table and kv_len NULL, num_pages 1,
 *         page_size n_rows)
 *   q, o  [n_rows, n_q_heads, head_dim]; o must not overlap q, k or v (column
 *         ranges of one tensor's rows may lie between each other)
 *   lse   [n_rows, n_q_heads] float32 or NULL: ln sum_j exp(scale * q . k_j),
 *         -infinity for a row that gets zeros
 *   scale positive, scale * log2(e) finite
 *   workspace  colibri_attention_prompt_workspace() bytes, 256-byte aligned;
 *         may be NULL where that is 0
 * Scores, maxima and sums are float32; for bf16 the weights are rounded to bf16
 * for the product with v, and sums are formed of weights up to 2^24, so
 * |v| * keys * 2^24 has to stay in float32's range.  Key rows beyond a sequence's
 * length may hold anything (NaN included).  Inside a sequence, and inside the part
 * of a shared prefix that some row sees, a non-finite value row may also reach rows
 * that do not see it, through a weight of 0.
 * Waits of the tensor-core kernel are bounded; rows whose wait gave up are
 * filled with NaN, and colibri_attention_check reports it.
 */
colibri_status_t colibri_attention_prompt_workspace(const colibri_kv_pages_t* kv,
                                                    const colibri_seqs_t* seqs,
                                                    int32_t n_q_heads, size_t* bytes);
colibri_status_t colibri_attention_prompt(const colibri_kv_pages_t* kv,
                                          const colibri_seqs_t* seqs, int32_t n_q_heads,
                                          const void* q, int64_t q_stride, float scale,
                                          int32_t causal, void* o, int64_t o_stride, float* lse,
                                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * colibri_attention_decode - attention of one row per sequence (seqs:
 * seq_start NULL, kv_len and page_table given) over all its kv_len[b] keys.
 * The first prefix_len keys of every sequence are those of prefix_table
 * [prefix_len / page_size] (device; prefix_len a multiple of page_size), read
 * once for the whole batch; page_table's entries for them are not read.  A prefix
 * of more than 2^31 - 2^20 keys is UNSUPPORTED.
 * prefix_len 0: no shared prefix (prefix_table NULL).  A sequence with
 * kv_len[b] <= prefix_len sees the prefix's first kv_len[b] keys, one with
 * kv_len[b] = 0 gets zeros.  Other arguments as colibri_attention_prompt.
 */
colibri_status_t colibri_attention_decode_workspace(const colibri_kv_pages_t* cache,
                                                    const colibri_seqs_t* seqs,
                                                    int32_t n_q_heads, int32_t prefix_len,
                                                    size_t* bytes);
colibri_status_t colibri_attention_decode(const colibri_kv_pages_t* cache,
                                          const colibri_seqs_t* seqs, int32_t n_q_heads,
                                          const void* q, int64_t q_stride, float scale,
                                          int32_t prefix_len, const int32_t* prefix_table,
                                          void* o, int64_t o_stride, float* lse, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * colibri_attention_check - wait for `stream` (of the current device; not while it
 * is being captured), then COLIBRI_ERR_TIMEOUT when a wait of a prompt or decode call
 * on this device gave up since the last check, whatever stream it ran on;
 * COLIBRI_ERR_CUDA for a CUDA error.
 */
colibri_status_t colibri_attention_check(void* stream);

/*
 * colibri_attention_waits - for later calls of the process: the bound of the
 * tensor-core kernel's waits in nanoseconds (0: 2 s, the default), and, for
 * failure-detection tests, the work item from which on a CTA's copies stop (1:
 * the first; 0: never).  Until it is called they are what COLIBRI_WAIT_LIMIT_NS and
 * COLIBRI_TEST_STALL_TMA said at the process's first attention call.
 */
colibri_status_t colibri_attention_waits(uint64_t limit_ns, int32_t stall);

/*
 * A cache held in 8 bits, for bf16 rows: a key or value element is code * scale, with
 * one scale for each block of `block` tokens of each key head.  Codes lie as the
 * elements of colibri_kv_pages_t do (strides in bytes, multiples of 16); the scale of
 * block j of head h of page p is at [(p * n_kv_heads + h) * (page_size / block) + j]
 * of k_scale and of v_scale.
 *   code   E4M3 numbers, or INT8 whole numbers
 *   block  16, 32 or 64, at most page_size
 * page_size is a power of two from 16 to 65536.  Attention takes any codes and any
 * scales that are finite and not negative; an E4M3 code that is no number (0x7f, 0xff) must
 * not stand where a row sees it.  What stands behind a sequence's last key may be anything, the scale of
 * a block without keys included.
 */
typedef enum { COLIBRI_CODE_E4M3 = 0, COLIBRI_CODE_INT8 = 1 } colibri_code_t;

typedef struct {
    void* k;               /* device */
    void* v;               /* device */
    float* k_scale;        /* device */
    float* v_scale;        /* device */
    int64_t page_stride;
    int64_t head_stride;
    int64_t row_stride;
    int32_t num_pages;
    int32_t page_size;
    int32_t n_kv_heads;
    int32_t head_dim;
    int32_t code;          /* colibri_code_t */
    int32_t block;
} colibri_kv_pages8_t;

/*
 * colibri_append_qkv8 - colibri_append_qkv(_at) of bf16 rows into such a cache.  q' goes
 * to q_out in bf16; k' and v go to their places as codes, rounded once from float32:
 *   code = round(x * (1 / scale)), to nearest, ties to even.
 * Of the elements x that the call brings to a block, let m be the largest magnitude.
 * A block that holds earlier rows of the sequence keeps its scale where m <= largest
 * code * scale (448, 127).  Otherwise its scale becomes the smallest power of two 2^e,
 * e >= -100, with m <= largest code * 2^e, and the codes of its earlier rows, if it has
 * any, become round(code * (old scale / scale)).  A block of a head that is given an
 * element that is not finite gets the scale NaN, and all its values are NaN until a
 * call writes the block from its first row on.
 * Blocks of the cache that get no row, and codes behind the call's last row, stay as
 * they are.  No two sequences of a call may append to one page.  k, v and the scales
 * must not overlap.
 */
colibri_status_t colibri_append_qkv8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                     const colibri_rope_t* rope, const colibri_positions_t* positions,
                                     int32_t n_q_heads, const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     const void* q_norm, const void* k_norm, float eps, void* q_out,
                                     int64_t q_out_stride, void* stream);

/*
 * colibri_values8 - the values of pages, code * scale in bf16: of page pages[i] (pages
 * [n_pages] device; NULL: page i) into k_out and v_out [n_pages, n_kv_heads, page_size,
 * head_dim].  An id that no page has gives zeros.
 */
colibri_status_t colibri_values8(const colibri_kv_pages8_t* cache, const int32_t* pages, int32_t n_pages,
                                 void* k_out, void* v_out, void* stream);

/*
 * colibri_attention_prompt8, colibri_attention_decode8 - colibri_attention_prompt over
 * pages (page_table and kv_len given) and colibri_attention_decode over an 8-bit cache; q
 * and o are bf16.  Codes enter the products as they are, scales and sums are float32.
 * Weights times value scales are rounded for the product with the codes: to bf16, or,
 * for one row per sequence and prompts of few rows (32 per sequence and key head on
 * average), to f16 on a reference of the row's largest such product, so that a key's
 * part below 2^-31 of that is lost.
 */
colibri_status_t colibri_attention_prompt8_workspace(const colibri_kv_pages8_t* cache,
                                                     const colibri_seqs_t* seqs, int32_t n_q_heads,
                                                     size_t* bytes);
colibri_status_t colibri_attention_prompt8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                           int32_t n_q_heads, const void* q, int64_t q_stride,
                                           float scale, int32_t causal, void* o, int64_t o_stride,
                                           float* lse, void* workspace, size_t workspace_bytes,
                                           void* stream);
colibri_status_t colibri_attention_decode8_workspace(const colibri_kv_pages8_t* cache,
                                                     const colibri_seqs_t* seqs, int32_t n_q_heads,
                                                     int32_t prefix_len, size_t* bytes);
colibri_status_t colibri_attention_decode8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                           int32_t n_q_heads, const void* q, int64_t q_stride,
                                           float scale, int32_t prefix_len, const int32_t* prefix_table,
                                           void* o, int64_t o_stride, float* lse, void* workspace,
                                           size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* COLIBRI_ATTN_H */
