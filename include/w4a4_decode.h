/*
 * w4a4_decode.h — C ABI of the operators of a decoding step (same library as
 * w4a4.h):
 *   w4a16_qlinear_forward  a projection of a few rows by 4-bit weights with
 *                          group scales, the activations not quantized;
 *   w4a4_cache_write       keys and values quantized to 4 or 8 bits as they
 *   w4a4_cache_read        are written into a paged cache, and read back;
 *   w4a4_cache_attention   attention of a batch over that cache, in which a
 *                          prefix shared by all sequences is computed once.
 *
 * Conventions: statuses, dtypes, streams and threads as in w4a4.h (every
 * call only enqueues work on `stream`, allocates nothing, keeps no pointer
 * past the call, and enqueues nothing when it returns a non-OK status).
 * Matrices are row-major with contiguous rows; `ld...` is the distance
 * between rows in elements (at least the row's length).  Index arrays are
 * contiguous int32 in device memory.  Weights, the cache and workspaces are
 * contiguous and aligned to 16 bytes.  Offsets are 64 bits wide.
 */
#ifndef W4A4_DECODE_H
#define W4A4_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "w4a4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace w4a16_qlinear_forward needs for up to M rows (0 if it
 * needs none or a size is 0 or negative).  Calls that share one workspace
 * must not overlap in time. */
size_t w4a16_qlinear_workspace_size(int64_t M, int64_t N, int64_t K);

/*
 * The projection without quantization of the activations, meant for few rows
 * (the weights are read once for every 64 rows):
 *   y[m, n] = sum_j w_scale[n, j] sum_{k in group j} x[m, k] q[n, k].
 *   x       [M, K] in x_dtype; rows aligned to 16 bytes (x and ldx).  K a
 *           positive multiple of 64, at most 16384, as in the layer; N at most
 *           16776960, M at most 4194240.
 *   wq      codes as written by w4a4_quantize_weight_int4 (-8 multiplies
 *           correctly as well) in w_layout: W4A4_WEIGHTS_ROWMAJOR or, with K a
 *           multiple of 128, W4A4_WEIGHTS_TILED; others are
 *           W4A4_ERR_UNSUPPORTED.  Weights prepared with a Hadamard block take
 *           rotated activations (w4a4_hadamard_rotate).
 *   w_scale [N] (w_group 0) or [N, K / w_group] in w_scale_dtype; w_group 0 or
 *           a multiple of 64 (tiled: of 128) dividing K.
 *   y       [M, N] in y_dtype; only its element's alignment is needed.
 *   The products are exact and the sums float32: fp16 activations meet the
 *   codes on the fp16 matrix instruction, float32 ones as three bfloat16 parts
 *   that add up to them (parts below 2^-133 are lost).  An infinity in x gives
 *   infinities or NaN in its row of y.  A row's result depends on that row
 *   only (M chooses the order of its sums) and is the same from call to call.
 *   workspace: at least w4a16_qlinear_workspace_size(M, N, K) bytes, or NULL
 *   where that is 0.
 */
int w4a16_qlinear_forward(const void* x, int x_dtype, int64_t ldx, const uint8_t* wq, int w_layout,
                          const void* w_scale, int w_scale_dtype, int64_t M, int64_t N, int64_t K,
                          int64_t w_group, void* y, int y_dtype, int64_t ldy, void* workspace,
                          size_t ws_bytes, void* stream);

/*
 * A cache of keys and values in pages.  For head h of the token in slot
 * p * page_size + o (offset o of page p):
 *   k, v              [pages, heads, page_size, head_dim * bits / 8] bytes:
 *                     codes of 4 bits (two's-complement nibbles, the even
 *                     channel in the low one) or 8 bits (int8);
 *   k_scale, v_scale  [pages, heads, page_size] float32: a value is its code
 *                     times its row's scale.
 * bits 4 or 8; head_dim 64, 128 or 256; page_size a power of two from 16 to
 * 65536; pages * page_size below 2^31.  The struct is read during the call
 * only.
 */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t pages, heads, page_size, head_dim;
  int bits;
} w4a4_cache;

/*
 * Quantizes the keys and values of T tokens into their slots: per token and
 * head s = max|x| / qmax in float32 (IEEE division; qmax 7 or 127), codes
 * clamp(rint(x / s), -qmax, qmax) with the quotient rounded to float32 and
 * ties to even; a zero scale gives all-zero codes (the quantizer of w4a4.h).
 *   k, v   [T, heads * head_dim] in dtype, rows ldk and ldv apart; only their
 *          element's alignment is needed.
 *   slots  [T]; a token whose slot is outside [0, pages * page_size) is not
 *          written.  A slot may occur once in a call (of tokens that share
 *          one, the slot holds a mixture).
 *   The input must be finite: a row holding a NaN or an infinity gets
 *   unspecified codes and scale.
 */
int w4a4_cache_write(const w4a4_cache* cache, const void* k, int64_t ldk, const void* v, int64_t ldv,
                     int dtype, const int32_t* slots, int64_t T, void* stream);

/*
 * The values in T slots (any order, repeated ones too): code times scale in
 * float32, rounded to dtype.
 *   k, v   [T, heads * head_dim] in dtype, rows ldk and ldv apart; one of
 *          them may be NULL (not read).  The rows of a slot outside
 *          [0, pages * page_size) become zero.
 */
int w4a4_cache_read(const w4a4_cache* cache, const int32_t* slots, int64_t T, void* k, int64_t ldk,
                    void* v, int64_t ldv, int dtype, void* stream);

/* Bytes of workspace w4a4_cache_attention needs for these sizes (0 if it
 * needs none or a size is outside its limits).  Smaller sizes may need more: a
 * workspace for several sizes has the largest of theirs.  Calls that share one
 * workspace must not overlap in time. */
size_t w4a4_cache_attention_workspace_size(const w4a4_cache* cache, int64_t tokens, int64_t q_heads,
                                           int64_t seqs, int64_t table_width, int64_t max_q,
                                           int64_t prefix_width);

/*
 * Attention of the queries of a batch over the cache:
 *   out[t, h] = sum_j p_j v_j,  p = softmax over the visible tokens j of
 *               scale * q[t, h] . k_j,
 * keys and values those of cache head h / (q_heads / heads).
 *   q       [tokens, q_heads * head_dim] in q_dtype, out the same in
 *           out_dtype; only their element's alignment is needed.  q_heads a
 *           multiple of the cache's heads.
 *   Sequence s has the cache tokens of positions [0, lengths[s]): position i
 *   is in page tables[s * table_width + i / page_size].  Lengths are taken
 *   between 0 and table_width * page_size.  Positions whose page is outside
 *   [0, pages) are not visible.
 *   q_start [seqs + 1], ascending from 0 to at most `tokens`: the queries of
 *           sequence s are rows [q_start[s], q_start[s + 1]), at most max_q
 *           (rows past max_q are not computed).  NULL: one row a sequence
 *           (tokens at least seqs, max_q 1).
 *   causal  non-zero: of n queries of a sequence of length L, query i sees
 *           positions up to L - n + i; zero: all positions.
 *   prefix_table [prefix_width], prefix_length [1]: pages of a prefix in
 *           front of all sequences, and its length (taken between 0 and
 *           prefix_width * page_size); every query sees all of it.  NULL and
 *           0: none.
 *   Sizes: q_heads at most 65536; table_width and prefix_width times page_size at
 *   most 2^30; tokens, and seqs, times q_heads below 2^31, seqs times heads below
 *   2^23, and the lesser of tokens and seqs times max_q, times q_heads, below 2^24
 *   (262144 queries of 64 heads); what is beyond is W4A4_ERR_UNSUPPORTED.
 *   Rows of q that belong to no sequence are not read, and those of out are
 *   left as they are.  A query that sees nothing gets zeros.
 *   Scores and sums are float32: codes are exact, queries enter under a power
 *   of two of their row, fp16 ones as they are (what is below 2^-31 of the
 *   row's largest may be lost) and float32 ones as a pair of fp16 values, and
 *   the probability times the value's scale as such a pair too (off by 2^-23 of
 *   itself or 2^-33 of the row's largest); products with 4-bit keys may be cut
 *   at 2^-22 of the largest of 32 channels.  Float32 outputs are about as close
 *   as those of the formula in float32 operations.  What masked positions hold
 *   has no effect.
 *   Ranges: |scale| times a row's largest query below 2^115, the sum of a score's
 *   |scale q k| below 2^120 (where a score passes 2^26, with values' scales below
 *   2^14), values' scales below 2^100.  In a row outside them infinities, NaN and
 *   zeros may come out.
 *   A row's result depends on its own sequence and the prefix only (the
 *   call's sizes and the lengths choose the order of its sums) and is the
 *   same from call to call.
 */
int w4a4_cache_attention(const w4a4_cache* cache, const void* q, int q_dtype, int64_t ldq,
                         int64_t tokens, int64_t q_heads, const int32_t* tables, int64_t seqs,
                         int64_t table_width, const int32_t* lengths, const int32_t* q_start,
                         int64_t max_q, int causal, const int32_t* prefix_table,
                         int64_t prefix_width, const int32_t* prefix_length, float scale, void* out,
                         int out_dtype, int64_t ldo, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A4_DECODE_H */
