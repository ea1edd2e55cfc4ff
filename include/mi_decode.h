/*
 * mi_decode.h -- C ABI of libmi_decode: the operators that stand beside the
 * projections in the decode step of a language model, for AMD Instinct MI355X
 * (gfx950).
 *
 *   mi_decode_w4_linear  linear layer with 4-bit weights and group scales, for
 *                        few tokens;
 *   mi_decode_kv_append  keys and values of new tokens into a paged 8-bit
 *                        cache, rotated by their positions on the way;
 *   mi_decode_kv_read    the values of a range of cached tokens;
 *   mi_decode_kv_attend  attention over that cache;
 *   mi_decode_rms_norm_f8     norm, with the residual's addition, into 8-bit
 *                             floats with a scale for 128 columns;
 *   mi_decode_f8_linear       linear layer of 8-bit floats with block scales,
 *                             for any number of tokens;
 *   mi_decode_kv_append_at    append with positions of its own for the rotation;
 *   mi_decode_kv_attend_tree  attention for a tree of drafted tokens;
 *   mi_decode_kv_keep         the drafted tokens that are kept move together;
 *   mi_decode_kv_copy         copies of pages.
 *
 * Conventions for every function:
 *   - Pointers are DEVICE pointers on the handle's device (the cache descriptor
 *     itself is a host struct); the caller owns them.  Sizes and strides count
 *     elements.  Activations are IEEE binary16 or bfloat16 (mi_decode_dtype_t).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Work
 *     is enqueued on it and the call returns without synchronising.  Nothing is
 *     allocated per call and nothing but kernels is enqueued, so every call may
 *     be captured into a graph.
 *   - No exception crosses the ABI; every failure is a status code, and no work
 *     is enqueued then.
 *   - mi_decode_kv_attend and mi_decode_kv_attend_tree keep partial results in
 *     the handle's workspace: launches of one handle that may run at the same
 *     time on different streams must use separate handles.  The other operators
 *     use no workspace.
 *   - Page tables, lengths and offsets are read by the kernels.  A page number
 *     outside 0 .. pages-1 is never followed: tokens on it are skipped (not
 *     appended, read as zeros, not attended to).  Lengths and offsets are
 *     clamped to the table's and the token arrays' extents.  Rows of outputs
 *     whose token belongs to no sequence (before cu[0], or from cu[batch] on)
 *     are not written.
 */
#ifndef MI_DECODE_H
#define MI_DECODE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mi_decode_ctx* mi_decode_handle_t;

typedef enum {
  MI_DECODE_OK = 0,
  MI_DECODE_ERR_INVALID_ARG = 1, /* null pointer, negative size, stride too small, size mismatch */
  MI_DECODE_ERR_UNSUPPORTED = 2, /* a size, type or alignment that no kernel takes */
  MI_DECODE_ERR_NO_DEVICE = 3,   /* no gfx950 device (or an inspection handle asked to launch) */
  MI_DECODE_ERR_HIP = 4          /* a HIP call failed; see mi_decode_last_hip_error */
} mi_decode_status_t;

typedef enum { MI_DECODE_F16 = 0, MI_DECODE_BF16 = 1 } mi_decode_dtype_t;
/* Codes of a cache: int8 -127..127, or e4m3 (OCP, largest value 448). */
typedef enum { MI_DECODE_INT8 = 0, MI_DECODE_E4M3 = 1 } mi_decode_code_t;

/* Flags of mi_decode_create. */
#define MI_DECODE_CREATE_NO_DEVICE 1u /* inspection handle: arguments are checked, nothing launches */

/* Create a handle on the current HIP device.  Allocates the workspace of
 * mi_decode_kv_attend and mi_decode_kv_attend_tree once (MI_DECODE_WORKSPACE_BYTES).  Returns OK,
 * INVALID_ARG (out NULL), NO_DEVICE or ERR_HIP (no memory). */
#define MI_DECODE_WORKSPACE_BYTES (64u << 20)
mi_decode_status_t mi_decode_create(mi_decode_handle_t* out, uint32_t flags);

/* Release a handle (NULL is a no-op).  Waits for nothing. */
mi_decode_status_t mi_decode_destroy(mi_decode_handle_t h);

/* The HIP device of a handle, or -1 (NULL, or an inspection handle). */
int mi_decode_device(mi_decode_handle_t h);

/* Human-readable name of a status.  Never NULL. */
const char* mi_decode_status_string(mi_decode_status_t s);

/* The hipError_t of the handle's last failed HIP call (0 if none). */
int mi_decode_last_hip_error(mi_decode_handle_t h);

/*
 * y[m][n] = round( sum_k x[m][k] * (c[n][k] - z[n][k / group]) * s[n][k / group] + bias[n] )
 * for 0 <= m < M, 0 <= n < N, 0 <= k < K: sums in binary32, one rounding to y's type.
 *   x [M, K] and y [M, N] of type dtype with unit-stride rows ldx >= K and
 *   ldy >= N apart (ldx at most 2^25, K at most 2^30); bias [N] of type dtype or NULL.
 *   qweight: the codes c, 0..15, in tiles of 16 rows by 128 columns, 1 KiB
 *   each: tile (n / 16, k / 128) is number (n / 16) * ceil(K / 128) + k / 128.
 *   Its 32-bit word 4 * l + j with l = 16 c + r holds row 16 (n / 16) + r,
 *   columns 128 (k / 128) + 32 j + 8 c + e for e = 0..7, at bit
 *   4 (e / 2) + 16 (e % 2).  One 16-byte load per lane then is the operand of
 *   four matrix instructions, and a whole wave's load is one contiguous KiB.
 *   Codes past N and past K may hold anything.
 *   scales [ceil(K / group)][16 ceil(N / 16)] of type dtype; zeros uint8 of
 *   the same shape (0..15), or NULL for 8 everywhere.
 *   group: a positive multiple of 32.
 * Any alignment of x, y and bias to their elements is taken; qweight must be
 * 16-byte aligned (UNSUPPORTED otherwise).  M == 0 or N == 0: nothing is done.
 * K == 0: y = bias, or 0.  y must not overlap any input.
 */
mi_decode_status_t mi_decode_w4_linear(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                       int64_t N, int64_t K, int64_t group, const void* x,
                                       int64_t ldx, const void* qweight, const void* scales,
                                       const void* zeros, const void* bias, void* y, int64_t ldy,
                                       void* stream);

/*
 * A paged cache of 8-bit keys and values.  k and v are [pages][kv_heads]
 * [page_size][head_dim] codes, contiguous and 16-byte aligned; k_scale and
 * v_scale are binary32 [pages][kv_heads].  A cached value is its code times
 * the scale of its page and head.  page_size is 16, 32, 64, 128 or 256;
 * head_dim is 64, 128 or 256.  Position p of sequence b lies in slot
 * p % page_size of page table[b * table_stride + p / page_size].
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t code; /* mi_decode_code_t */
} mi_decode_cache_t;

/* The tokens of a ragged batch and where they lie in the cache (host struct). */
typedef struct {
  const int32_t* table;  /* [batch][table_cols], rows table_stride apart */
  const int32_t* lens;   /* [batch], see each function */
  const int32_t* cu;     /* [batch + 1] first token of each sequence, cu[batch] = tokens; NULL: one token each */
  int64_t table_stride;
  int32_t table_cols;
  int32_t batch;
  int32_t tokens;
  int32_t max_tokens;    /* no sequence has more tokens than this in the call */
} mi_decode_batch_t;

/* 16-bit rows [tokens][heads][head_dim] whose last dimension is contiguous. */
typedef struct {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} mi_decode_rows_t;

/*
 * Append the batch's tokens: token i of sequence b takes position
 * lens[b] + i, where lens holds the tokens that the sequence already has.
 *   k, v: [tokens][kv_heads][head_dim] of type dtype.
 *   rope: binary32 [rope_rows][rot_dim], rot_dim / 2 cosines followed by
 *   rot_dim / 2 sines for each position, or NULL (no rotation).  The first
 *   rot_dim channels of k (and of q) are turned in pairs (i, i + rot_dim / 2),
 *   or (2 i, 2 i + 1) if interleaved:
 *       (a, b) -> (a cos - b sin, b cos + a sin).
 *   rot_dim: a multiple of 16, at most head_dim.  rope_rows must cover every
 *   position of the table (table_cols * page_size), else INVALID_ARG.
 *   q, q_out: [tokens][q_heads][head_dim] queries to be turned by the same
 *   angles, and where they go (may be q itself, then also in one buffer with k
 *   and v, but in none of their elements); q NULL or q_heads 0: none.
 * Scales.  For each page and head that receives tokens, with QMAX 127 (int8)
 * or 448 (e4m3): s' = max(s, max |x| / QMAX), where s is the page's scale if
 * the page already held tokens of the sequence and 0 if its first slot is
 * filled now.  New codes are x / s' rounded to nearest even (0 if s' is 0).
 * Where s' > s, the codes that the page held become round(code * s / s').  A
 * non-finite x leaves a non-finite scale: the page's values for that head read
 * as non-finite rather than wrong, until its first slot is filled again.
 * The same page must not receive tokens of two sequences in one call.  Tokens
 * past the table's end are skipped (their q is still turned, by the last row).
 */
mi_decode_status_t mi_decode_kv_append(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                       mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                       const mi_decode_rows_t* k, const mi_decode_rows_t* v,
                                       const float* rope, int64_t rope_rows, int32_t rot_dim,
                                       int32_t interleaved, int32_t q_heads,
                                       const mi_decode_rows_t* q, const mi_decode_rows_t* q_out,
                                       void* stream);

/*
 * The values of cached tokens: token i of sequence b is position lens[b] + i.
 * k_out and v_out: contiguous [tokens][kv_heads][head_dim] of type dtype,
 * each value code * scale in binary32 rounded once.  Tokens without a valid
 * page read as zeros.
 */
mi_decode_status_t mi_decode_kv_read(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                     void* k_out, void* v_out, void* stream);

/*
 * out = softmax(scale * q k^T + mask) v over the cache.  lens[b] is the number
 * of tokens that sequence b has in the cache, the batch's own included: its n
 * query tokens are the last n, so query i stands at position
 * p = lens[b] - n + i and sees position j where
 *     0 <= j <= p  and  (window == 0  or  j > p - window  or  j < sinks).
 * Query head h reads key-value head h / (q_heads / kv_heads).  A query that
 * sees nothing (p < 0, or no valid page) gives zeros.  What is not seen does
 * not enter the result, whatever its codes and scales are (NaN among them).
 * A query that sees a NaN code may be NaN in all its channels.
 *   max_len: no lens[b] is larger; used to plan the split of long sequences
 *   over workgroups, not for correctness.
 *   q, out: [tokens][q_heads][head_dim] of type dtype; q_heads a multiple of
 *   kv_heads.  out must not overlap an input.
 * Products take codes and binary16 queries exactly, bf16 queries too down to
 * 2^-32 of their row's largest channel (below, as a multiple of 2^-39 of it;
 * nothing below 2^-40), and softmax weights times their page's value scale in
 * 11 significant bits down to 2^-26 of the row's largest (below, as a multiple
 * of 2^-36 of it; nothing below 2^-37).  Sums and statistics are binary32.
 */
mi_decode_status_t mi_decode_kv_attend(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                       mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                       int64_t max_len, int32_t q_heads, const mi_decode_rows_t* q,
                                       const mi_decode_rows_t* out, float scale, int32_t window,
                                       int32_t sinks, void* stream);

/*
 * As mi_decode_kv_append, but token t of the call is turned by row
 * positions[t] of the rope table (int32 [tokens], clamped to 0 .. rope_rows - 1),
 * and so is its query; it still takes the place lens[b] + i in the cache.
 * Drafted tokens of a tree have the positions of their depths so, wherever they
 * lie.  rope_rows need not cover the table's positions.  positions NULL: as
 * mi_decode_kv_append.
 */
mi_decode_status_t mi_decode_kv_append_at(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                          mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                          const mi_decode_rows_t* k, const mi_decode_rows_t* v,
                                          const float* rope, int64_t rope_rows, int32_t rot_dim,
                                          int32_t interleaved, const int32_t* positions,
                                          int32_t q_heads, const mi_decode_rows_t* q,
                                          const mi_decode_rows_t* q_out, void* stream);

/*
 * Attention for drafted tokens, several continuations of a sequence at once.
 * As in mi_decode_kv_attend sequence b's n query tokens are the last n of its
 * lens[b] tokens in the cache; the c = lens[b] - n tokens before them are its
 * context.  Bit a % 32 of word a / 32 of row t of `seen` (int32
 * [tokens][seen_words], rows seen_stride apart) says whether token t of the
 * call sees its sequence's drafted token a, which may be itself; bits from n on
 * say nothing.  For a tree these are a token's ancestors and itself.  Token t sees
 *   - context position j < c where window == 0, or j > p - window, or j < sinks,
 *     with p = c + the number of drafted tokens other than itself that it sees
 *     (for a tree, the position of its depth);
 *   - drafted tokens by their bits alone, whatever the window is.  So a row of
 *     a tree with more levels than the window has tokens must not have the bits
 *     of ancestors at positions <= its own - window (and >= sinks), if it is to
 *     see what mi_decode_kv_attend would show it; p is then below its position
 *     and hides the same of the context, all but the sinks.
 * seen_words * 32 must be at least batch->max_tokens, and seen_stride at least
 * seen_words.  A query that sees nothing gives zeros.  Everything else is as in
 * mi_decode_kv_attend.
 */
mi_decode_status_t mi_decode_kv_attend_tree(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                            mi_decode_dtype_t dtype, const mi_decode_batch_t* batch,
                                            int64_t max_len, int32_t q_heads,
                                            const mi_decode_rows_t* q, const mi_decode_rows_t* out,
                                            const int32_t* seen, int64_t seen_stride,
                                            int32_t seen_words, float scale, int32_t window,
                                            int32_t sinks, void* stream);

/*
 * The drafted tokens that are kept move to the front of the drafts: token i of
 * sequence b, i < cu[b + 1] - cu[b], comes to position lens[b] + i from position
 * lens[b] + keep[cu[b] + i], where lens holds the tokens before the drafts.
 * All are as if they moved at once.  An entry with keep < i (so a negative
 * one), or whose source has no valid page, leaves its position as it is; a
 * position without a valid page is skipped.  Indices need not ascend, and one
 * may be there more than once.
 * Scales.  For each page and head that positions lens[b] .. lens[b] + n - 1 lie
 * on: s' = max(s, max |x| / QMAX) over the tokens x that come from other pages.
 * Codes become round(code * (s_source / s')), 0 where s' is 0: those that come,
 * and, where s' > s, those of all positions up to lens[b] + n - 1 that the page
 * holds.  s', the ratio and the product are binary64, and the product is rounded
 * to binary32 before the code's own rounding to nearest even, so that products
 * on the border between two codes, which simple ratios have, are not moved off
 * it by the ratio's error.  So a token that stays on its page keeps its code
 * unless the scale grows, and a NaN code then stays one.  A token from another page with a NaN
 * code or a scale that is not finite leaves a scale that is not finite, as in
 * mi_decode_kv_append.
 * Positions from lens[b] + n on hold no token of the sequence afterwards.
 * max_tokens: the most that a sequence keeps.  batch->cu NULL: one token each.
 * A page that the kept tokens come to or lie on must belong to one sequence and
 * be in its table once.
 */
mi_decode_status_t mi_decode_kv_keep(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     const mi_decode_batch_t* batch, const int32_t* keep,
                                     void* stream);

/*
 * Page dst[i] becomes a copy of page src[i], codes and scales of all heads, for
 * 0 <= i < pairs.  A pair with a page outside 0 .. pages - 1, or of a page with
 * itself, is skipped.  A page may be the source of several pairs; one that is
 * the destination of a pair must be in no other pair of the call (what it holds
 * afterwards is not defined then).
 */
mi_decode_status_t mi_decode_kv_copy(mi_decode_handle_t h, const mi_decode_cache_t* cache,
                                     const int32_t* src, const int32_t* dst, int64_t pairs,
                                     void* stream);

/*
 * For each row m of x [M][K], with r the row of `residual` (or nothing):
 *   t = round(x + r) in dtype,            which goes to `total`,
 *   y = t / sqrt(mean(t^2) + eps) * weight,
 *   scales[m][j] = max |y[k]| / 448        over 128 j <= k < 128 (j + 1), k < K,
 *   codes[m][k] = e4m3(y[k] / scales[m][k / 128])   to nearest even, 0 where the scale is 0.
 * Sums are binary32, and the square root's argument keeps its bits where squares
 * would leave binary32.  A block with a y that is not finite has a scale that
 * is not finite, so that it reads as non-finite rather than wrong.
 *   x, residual, total: of type dtype, rows ldx, ldr and ldt elements apart.
 *   residual NULL: t is x, and total must be NULL; total NULL: it is not wanted.
 *   weight [K] of type dtype, or NULL for 1.
 *   codes: e4m3 bytes, rows ldc >= K apart; scales: binary32, rows
 *   lds >= ceil(K / 128) apart.  eps: not negative, finite.
 * total may be x or residual themselves (the same pointer and row distance);
 * outputs may not overlap anything else.  Any alignment to elements is taken.
 * M == 0 or K == 0: nothing is done.
 */
mi_decode_status_t mi_decode_rms_norm_f8(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                         int64_t K, const void* x, int64_t ldx,
                                         const void* residual, int64_t ldr, const void* weight,
                                         float eps, void* codes, int64_t ldc, float* scales,
                                         int64_t lds, void* total, int64_t ldt, void* stream);

/*
 * y[m][n] = round( sum_j (xs[m][j] * ws[n / 128][j]) * sum_k x[m][k] w[n][k] + bias[n] )
 * with the inner sum over 128 j <= k < min(128 (j + 1), K), and one rounding to
 * dtype.  The matrix unit adds the products of 8 neighbouring columns (8 i to
 * 8 i + 7) in units of 2^-13 of the largest one's power of two and cuts off what is
 * below; all other sums, and the product of two scales, are binary32.
 *   x [M][K] and w [N][K]: e4m3 bytes, rows ldx and ldw >= K apart.
 *   xs [M][ceil(K / 128)] and ws [ceil(N / 128)][ceil(K / 128)]: binary32, rows
 *   ldxs and ldws apart.  bias [N] of type dtype, or NULL.  y: rows ldy >= N apart.
 * Any alignment to elements is taken; rows of x and w that begin and end at
 * multiples of 4 bytes are faster, and many rows at multiples of 16.
 * M == 0 or N == 0: nothing is done; K == 0: y = bias, or 0.
 * y must not overlap any input.
 */
mi_decode_status_t mi_decode_f8_linear(mi_decode_handle_t h, mi_decode_dtype_t dtype, int64_t M,
                                       int64_t N, int64_t K, const void* x, int64_t ldx,
                                       const float* xs, int64_t ldxs, const void* w, int64_t ldw,
                                       const float* ws, int64_t ldws, const void* bias, void* y,
                                       int64_t ldy, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MI_DECODE_H */
