/*
 * w4a4_block.h — C ABI of the operators that stand beside the W4A4 linear
 * layer in a transformer block (same library as w4a4.h):
 *   w4a4_adapter_add        low-rank adapters of many requests, added to the
 *                           output of one shared projection;
 *   w4a4_norm_residual      the norm after a block, its gate and residual
 *                           scale, the residual sum and the norm before the
 *                           next block, in one pass;
 *   w4a4_gated_activation   act(gate) * up between two projections.
 *
 * Conventions: statuses, dtypes, streams and threads as in w4a4.h (every
 * call only enqueues work on `stream`, allocates nothing, keeps no pointer
 * past the call, and enqueues nothing when it returns a non-OK status).
 * Matrices are row-major with contiguous rows; `ld...` is the distance
 * between rows in elements (at least the row's length).  Activations need
 * only their own element's alignment, except where an entry says more;
 * 16-byte-aligned rows are read in wide loads.  Weights, norm parameters and
 * workspaces are contiguous and aligned to 16 bytes.
 * Sizes: M (rows) may be 0 (nothing is enqueued).  Offsets are 64 bits wide.
 */
#ifndef W4A4_BLOCK_H
#define W4A4_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "w4a4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace w4a4_adapter_add needs for these sizes (0 if a size is
 * 0 or negative).  Calls that share one workspace must not overlap in time. */
size_t w4a4_adapter_workspace_size(int64_t M, int64_t K, int64_t rank);

/*
 * Adds to every row of a projection's output the low-rank term of that row's
 * own adapter.  For row m with a = index[m] in [0, adapters) and r = ranks[a]:
 *   out[m, n] = y[m, n] + scales[a] * sum_{j < r} t[j] Bt[a, n, j],
 *   t[j]      = sum_k x[m, k] At[a, j, k];
 * every other row: out[m] = y[m].
 *   x       [M, K] in x_dtype; rows aligned to 16 bytes (x and ldx).
 *           K a positive multiple of 64, at most 16384, as in the layer.
 *   At      [adapters, rank, K], Bt [adapters, N, rank] in x_dtype; rank in
 *           [1, 256], for fp16 a multiple of 8 (the layer's own limits);
 *           M at most 134217600, N at most 16776960.
 *   index   [M] int32 in device memory, any order; a value outside
 *           [0, adapters) means no adapter.
 *   ranks   [adapters] int32, or NULL (all `rank`).  Values are clamped to
 *           [0, rank]; At rows and Bt columns at or past ranks[a] are not
 *           used and may hold anything.
 *   scales  [adapters] float32, or NULL (all 1).
 *   y       [M, N] float32, or NULL (zero).  out [M, N] float32; out may
 *           equal y when ldo equals ldy.
 *   Both sums are float32 and t is not rounded to the factors' type: it stays
 *   float32, except that with 128 rows or more and fp16 factors the second
 *   product takes scales[a] t as a pair of fp16 values under powers of two per
 *   row and 32 or 64 ranks: off by 2^-22 of itself, or 2^-49 of the largest |t|
 *   of these ranks, whichever is more (float32's own rounding is 2^-24).  There
 *   an infinity among the factors in use may come out as NaN.
 *   A row's result depends on its own inputs only (not on the other rows'
 *   values; M and index choose the order of its sums) and is the same from call
 *   to call.
 *   workspace: at least w4a4_adapter_workspace_size(M, K, rank) bytes.
 */
int w4a4_adapter_add(const void* x, int x_dtype, int64_t ldx, const void* At, const void* Bt,
                     int64_t adapters, int64_t rank, const int32_t* index, const int32_t* ranks,
                     const float* scales, int64_t M, int64_t N, int64_t K, const float* y,
                     int64_t ldy, float* out, int64_t ldo, void* workspace, size_t ws_bytes,
                     void* stream);

typedef enum { W4A4_NORM_NONE = 0, W4A4_NORM_RMS = 1, W4A4_NORM_LAYER = 2 } w4a4_norm;

/*
 * The seam between two blocks, per row of C channels (1 <= C <= 16384):
 *   v = norm_post(y);  v *= gate[m / gate_rows];  h' = h + residual_scale * v;
 *   x = norm_pre(h').
 * A norm of v is v * (offset + w) + b after
 *   W4A4_NORM_RMS:    v / sqrt(mean(v^2) + eps);
 *   W4A4_NORM_LAYER:  (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps);
 *   W4A4_NORM_NONE:   v (w and b must be NULL).
 * A NULL w counts as offset + w = 1, a NULL b as 0.
 *   h      [M, C] in h_dtype, or NULL (zero); y [M, C] in y_dtype, or NULL
 *          (zero; then post_norm must be W4A4_NORM_NONE and gate NULL).  Not
 *          both NULL.
 *   gate   [ceil(M / gate_rows), C] in gate_dtype with row distance ldg, or
 *          NULL (one).  Row g serves rows [g gate_rows, (g + 1) gate_rows).
 *   post_w, post_b, pre_w, pre_b: [C] in p_dtype, or NULL.
 *   h_out  [M, C] in h_dtype, or NULL; may equal h when ldho equals ldh.
 *   x_out  [M, C] in x_dtype, or NULL (then pre_norm must be W4A4_NORM_NONE).
 *          x is formed from the float32 h', before it is rounded to h_dtype.
 * Sums and the values between the steps are float32; the variance is taken
 * over the centred values.
 */
int w4a4_norm_residual(const void* h, int h_dtype, int64_t ldh, const void* y, int y_dtype,
                       int64_t ldy, int post_norm, const void* post_w, const void* post_b,
                       const void* gate, int gate_dtype, int64_t ldg, int64_t gate_rows,
                       float residual_scale, int pre_norm, const void* pre_w, const void* pre_b,
                       int p_dtype, float offset, float eps, int64_t M, int64_t C, void* h_out,
                       int64_t ldho, void* x_out, int x_dtype, int64_t ldx, void* stream);

typedef enum {
  W4A4_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
  W4A4_ACT_GELU = 1,      /* g Phi(g), Phi the normal distribution function */
  W4A4_ACT_GELU_TANH = 2, /* g / 2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) */
  W4A4_ACT_RELU = 3       /* max(g, 0), NaN kept */
} w4a4_act;

/*
 * out[m, f] = act(gate[m, f]) * up[m, f], or act(gate[m, f]) with up NULL.
 *   gate, up  [M, F] in in_dtype with row distances ldg, ldu (the halves of
 *             one [M, 2F] projection, in either order, or two tensors).
 *   out       [M, F] in out_dtype.  Computed in float32, rounded once.
 */
int w4a4_gated_activation(const void* gate, int64_t ldg, const void* up, int64_t ldu, int in_dtype,
                          int act, int64_t M, int64_t F, void* out, int64_t ldo, int out_dtype,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A4_BLOCK_H */
