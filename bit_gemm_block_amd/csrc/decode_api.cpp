// decode_api.cpp — the C ABI declared in include/w4a4_decode.h: argument
// validation and stream-ordered launches.  No allocation happens here.
#include "w4a4_decode.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "block_internal.h"
#include "decode_internal.h"
#include "w4a4_internal.h"

namespace {

constexpr int64_t kMaxK = 16384;
// The grids' limits: 512 threads for 16 columns, 65535 workgroups of 64 rows.
constexpr int64_t kMaxN = 16776960;
constexpr int64_t kMaxM = int64_t{65535} * 64;
constexpr int64_t kMaxSlots = INT32_MAX;
constexpr int64_t kMaxTokens = int64_t{1} << 30;  // of a sequence or a prefix

bool dtype_ok(int d) { return d == W4A4_F32 || d == W4A4_F16; }
uintptr_t esize(int dtype) { return dtype == W4A4_F16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int status(hipError_t e) { return e == hipSuccess ? W4A4_OK : w4a4::hip_status(e); }

// The cache's sizes, and with `pointers` its addresses.
int check_cache(const w4a4_cache* c, bool pointers) {
  if (!c || c->pages <= 0 || c->heads <= 0 || c->page_size <= 0 || c->head_dim <= 0 || (c->bits != 4 && c->bits != 8))
    return W4A4_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->page_size < 16 || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)) != 0 || c->heads > 65536 || c->pages > kMaxSlots / c->page_size)
    return W4A4_ERR_UNSUPPORTED;
  if (!pointers) return W4A4_OK;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return W4A4_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return W4A4_ERR_MISALIGNED;
  return W4A4_OK;
}

int log2_of(int64_t v) {
  int r = 0;
  while ((int64_t{1} << r) < v) ++r;
  return r;
}

w4a4::CacheArgs cache_args(const w4a4_cache* c, const int32_t* slots, int64_t T) {
  w4a4::CacheArgs a{};
  a.codes[0] = c->k; a.codes[1] = c->v;
  a.scale[0] = c->k_scale; a.scale[1] = c->v_scale;
  a.slots = slots; a.T = T;
  a.heads = static_cast<int>(c->heads); a.page_log2 = log2_of(c->page_size);
  a.D = static_cast<int>(c->head_dim); a.bits = c->bits;
  a.slots_end = c->pages * c->page_size;
  return a;
}

// Fewer than 2^32 threads of eight elements each along a grid's x.
bool rows_fit(const w4a4_cache* c, int64_t T) {
  return T <= ((int64_t{1} << 32) - 256) / (c->heads * (c->head_dim / 8));
}

// Rows of N float32 partial sums that a projection of M rows writes.
int64_t w4a16_partial_rows(int64_t M, int64_t N, int64_t K) {
  const int parts = w4a4::w4a16_plan(M, N, K).parts;
  return parts > 1 ? parts * M : 0;
}

// Sizes of an attention call that its plan depends on.
int attention_sizes(const w4a4_cache* c, int64_t tokens, int64_t q_heads, int64_t seqs, int64_t width, int64_t max_q,
                    int64_t prefix_width, w4a4::AttentionArgs* a, w4a4::AttentionPlan* plan) {
  if (tokens < 0 || q_heads <= 0 || seqs < 0 || width < 0 || max_q <= 0 || prefix_width < 0)
    return W4A4_ERR_INVALID_ARG;
  if (q_heads % c->heads != 0) return W4A4_ERR_INVALID_ARG;
  max_q = max_q < tokens ? max_q : tokens > 0 ? tokens : 1;  // a sequence has no more queries than there are
  if (q_heads > 65536 || tokens > INT32_MAX / q_heads || seqs > INT32_MAX / q_heads ||
      width > kMaxTokens / c->page_size || prefix_width > kMaxTokens / c->page_size)
    return W4A4_ERR_UNSUPPORTED;
  a->pages = static_cast<int>(c->pages); a->heads = static_cast<int>(c->heads);
  a->page_log2 = log2_of(c->page_size); a->D = static_cast<int>(c->head_dim); a->bits = c->bits;
  a->tokens = static_cast<int>(tokens); a->q_heads = static_cast<int>(q_heads);
  a->group = w4a4::Divisor(static_cast<uint32_t>(q_heads / c->heads));
  a->by_heads = w4a4::Divisor(static_cast<uint32_t>(c->heads));
  a->seqs = static_cast<int>(seqs); a->width = width;
  a->max_q = static_cast<int>(max_q);
  a->prefix_width = prefix_width;
  return w4a4::attention_plan(*a, plan) ? W4A4_OK : W4A4_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

size_t w4a16_qlinear_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  // The most that M rows or fewer write: 64 rows may be cut into twice the parts of
  // 65.  With more 64s of rows there are no more parts.
  int64_t most = 0;
  for (int64_t m = 64;; m += 64) {
    const int64_t rows = w4a16_partial_rows(m < M ? m : M, N, K);
    most = rows > most ? rows : most;
    if (m >= M || rows == 0) break;
  }
  return static_cast<size_t>(most) * static_cast<size_t>(N) * 4;
}

int w4a16_qlinear_forward(const void* x, int x_dtype, int64_t ldx, const uint8_t* wq, int w_layout,
                          const void* w_scale, int w_scale_dtype, int64_t M, int64_t N, int64_t K, int64_t w_group,
                          void* y, int y_dtype, int64_t ldy, void* workspace, size_t ws_bytes, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(w_scale_dtype) || !dtype_ok(y_dtype) || M < 0 || N < 0 || K <= 0 ||
      w_group < 0 || ldx < K || ldy < N || w_layout < W4A4_WEIGHTS_ROWMAJOR || w_layout > W4A4_WEIGHTS_TILED_F6)
    return W4A4_ERR_INVALID_ARG;
  const bool tiled = w_layout == W4A4_WEIGHTS_TILED;
  const int64_t unit = tiled ? 128 : 64;
  if ((!tiled && w_layout != W4A4_WEIGHTS_ROWMAJOR) || K % unit != 0 || K > kMaxK || w_group % unit != 0 ||
      (w_group > 0 && K % w_group != 0) || M > kMaxM || N > kMaxN)
    return W4A4_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return W4A4_OK;
  const size_t need = static_cast<size_t>(w4a16_partial_rows(M, N, K)) * static_cast<size_t>(N) * 4;
  if (!x || !wq || !w_scale || !y || (need > 0 && !workspace)) return W4A4_ERR_INVALID_ARG;
  if (!aligned(x, 16) || (M > 1 && static_cast<uintptr_t>(ldx) * esize(x_dtype) % 16 != 0) || !aligned(wq, 16) ||
      !aligned(w_scale, 16) || !aligned(y, esize(y_dtype)) || !aligned(workspace, 16))
    return W4A4_ERR_MISALIGNED;
  if (ws_bytes < need) return W4A4_ERR_WORKSPACE;
  int s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::W4a16Args a{};
  a.x = x; a.ldx = ldx; a.wq = wq; a.tiled = tiled;
  a.sw = w_scale; a.sw_f16 = w_scale_dtype == W4A4_F16;
  a.M = M; a.N = N; a.K = static_cast<int>(K);
  a.groups = static_cast<int>(w_group ? K / w_group : 1);
  a.group_halves = w4a4::Divisor(static_cast<uint32_t>((w_group ? w_group : K) / 64));
  a.y = y; a.y_f16 = y_dtype == W4A4_F16; a.ldy = ldy;
  a.y_wide = aligned(y, 16) && ldy % 4 == 0;
  a.partial = need > 0 ? static_cast<float*>(workspace) : nullptr;
  return status(w4a4::launch_w4a16(a, x_dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

int w4a4_cache_write(const w4a4_cache* cache, const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype,
                     const int32_t* slots, int64_t T, void* stream) {
  int s = check_cache(cache, true);
  if (s != W4A4_OK) return s;
  const int64_t C = cache->heads * cache->head_dim;
  if (!dtype_ok(dtype) || T < 0 || ldk < C || ldv < C) return W4A4_ERR_INVALID_ARG;
  if (!rows_fit(cache, T)) return W4A4_ERR_UNSUPPORTED;
  if (T == 0) return W4A4_OK;
  if (!k || !v || !slots) return W4A4_ERR_INVALID_ARG;
  if (!aligned(k, esize(dtype)) || !aligned(v, esize(dtype)) || !aligned(slots, 4)) return W4A4_ERR_MISALIGNED;
  s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::CacheArgs a = cache_args(cache, slots, T);
  a.x[0] = const_cast<void*>(k); a.x[1] = const_cast<void*>(v);
  a.ld[0] = ldk; a.ld[1] = ldv;
  return status(w4a4::launch_cache_write(a, dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

int w4a4_cache_read(const w4a4_cache* cache, const int32_t* slots, int64_t T, void* k, int64_t ldk, void* v,
                    int64_t ldv, int dtype, void* stream) {
  int s = check_cache(cache, true);
  if (s != W4A4_OK) return s;
  const int64_t C = cache->heads * cache->head_dim;
  if (!dtype_ok(dtype) || T < 0 || (k && ldk < C) || (v && ldv < C)) return W4A4_ERR_INVALID_ARG;
  if (!rows_fit(cache, T)) return W4A4_ERR_UNSUPPORTED;
  if (T == 0) return W4A4_OK;
  if ((!k && !v) || !slots) return W4A4_ERR_INVALID_ARG;
  if (!aligned(k, esize(dtype)) || !aligned(v, esize(dtype)) || !aligned(slots, 4)) return W4A4_ERR_MISALIGNED;
  s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::CacheArgs a = cache_args(cache, slots, T);
  a.x[0] = k; a.x[1] = v;
  a.ld[0] = ldk; a.ld[1] = ldv;
  return status(w4a4::launch_cache_read(a, dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

size_t w4a4_cache_attention_workspace_size(const w4a4_cache* cache, int64_t tokens, int64_t q_heads, int64_t seqs,
                                           int64_t table_width, int64_t max_q, int64_t prefix_width) {
  w4a4::AttentionArgs a{};
  w4a4::AttentionPlan plan{};
  if (check_cache(cache, false) != W4A4_OK ||
      attention_sizes(cache, tokens, q_heads, seqs, table_width, max_q, prefix_width, &a, &plan) != W4A4_OK)
    return 0;
  return w4a4::attention_workspace(a, plan);
}

int w4a4_cache_attention(const w4a4_cache* cache, const void* q, int q_dtype, int64_t ldq, int64_t tokens,
                         int64_t q_heads, const int32_t* tables, int64_t seqs, int64_t table_width,
                         const int32_t* lengths, const int32_t* q_start, int64_t max_q, int causal,
                         const int32_t* prefix_table, int64_t prefix_width, const int32_t* prefix_length, float scale,
                         void* out, int out_dtype, int64_t ldo, void* workspace, size_t ws_bytes, void* stream) {
  int s = check_cache(cache, true);
  if (s != W4A4_OK) return s;
  w4a4::AttentionArgs a{};
  w4a4::AttentionPlan plan{};
  if (!dtype_ok(q_dtype) || !dtype_ok(out_dtype) || !std::isfinite(scale)) return W4A4_ERR_INVALID_ARG;
  s = attention_sizes(cache, tokens, q_heads, seqs, table_width, max_q, prefix_width, &a, &plan);
  if (s != W4A4_OK) return s;
  const int64_t C = q_heads * cache->head_dim;
  if (ldq < C || ldo < C) return W4A4_ERR_INVALID_ARG;
  if (!q_start && (max_q != 1 || tokens < seqs)) return W4A4_ERR_INVALID_ARG;
  if ((prefix_width > 0) != (prefix_table != nullptr) || (prefix_table != nullptr) != (prefix_length != nullptr))
    return W4A4_ERR_INVALID_ARG;
  if (tokens == 0 || seqs == 0) return W4A4_OK;
  const size_t need = w4a4::attention_workspace(a, plan);
  if (!q || !out || !lengths || (table_width > 0 && !tables) || (need > 0 && !workspace)) return W4A4_ERR_INVALID_ARG;
  if (!aligned(q, esize(q_dtype)) || !aligned(out, esize(out_dtype)) || !aligned(tables, 4) || !aligned(lengths, 4) ||
      !aligned(q_start, 4) || !aligned(prefix_table, 4) || !aligned(prefix_length, 4) || !aligned(workspace, 16))
    return W4A4_ERR_MISALIGNED;
  if (ws_bytes < need) return W4A4_ERR_WORKSPACE;
  s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  a.k = cache->k; a.v = cache->v; a.ks = cache->k_scale; a.vs = cache->v_scale;
  a.q = q; a.ldq = ldq;
  a.tables = tables; a.lengths = lengths; a.q_start = q_start; a.causal = causal != 0;
  a.prefix_table = prefix_table; a.prefix_length = prefix_length;
  a.scale = scale;
  a.out = out; a.out_f16 = out_dtype == W4A4_F16; a.ldo = ldo;
  a.partial = static_cast<float*>(workspace);
  return status(w4a4::launch_attention(a, plan, q_dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
