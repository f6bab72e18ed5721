// Internal launch interface of the operators of a decoding step: decode_api.cpp
// validates, w4a16.hip, cache.hip and attention*.hip run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

// ---- a projection with 4-bit weights and unquantized activations (w4a16.hip) ----
struct W4a16Args {
  const void* x;  // [M, K], row distance ldx
  int64_t ldx;
  const uint8_t* wq;
  int tiled;
  const void* sw;  // [N, K / group]
  int sw_f16;
  int64_t M, N;
  int K, group;  // group K: one scale per channel
  void* y;       // [M, N], row distance ldy
  int y_f16;
  int64_t ldy;
  float* partial;  // workspace: [parts][M][N], or null
};

// How a call is cut: 16 nb output channels and 16 mt rows to a workgroup, whose
// waves share the channels' K; parts of K over workgroups.
struct W4a16Plan {
  int nb, mt, waves, parts;
};
W4a16Plan w4a16_plan(int64_t M, int64_t N, int64_t K);
hipError_t launch_w4a16(const W4a16Args& a, bool x_f16, hipStream_t st);

// ---- quantized cache (cache.hip) -------------------------------------------------
struct CacheArgs {
  uint8_t* codes[2];  // keys, values: [pages, heads, page, D * bits / 8]
  float* scale[2];    // [pages, heads, page]
  void* x[2];         // [T, heads * D], or null; row distances ld
  int64_t ld[2];
  const int32_t* slots;
  int64_t T;
  int heads, page_log2, D, bits;
  int64_t slots_end;  // pages * page
};
hipError_t launch_cache_write(const CacheArgs& a, bool f16, hipStream_t st);
hipError_t launch_cache_read(const CacheArgs& a, bool f16, hipStream_t st);

// ---- attention over the cache (attention.hip) -------------------------------------
struct AttentionArgs {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  int pages, heads, page_log2, D, bits;
  const void* q;
  int64_t ldq;
  int tokens, q_heads, group;  // group: query heads to a cache head
  const int32_t* tables;
  int seqs;
  int64_t width;
  const int32_t* lengths;
  const int32_t* q_start;  // or null
  int max_q, causal;
  const int32_t* prefix_table;  // or null
  int64_t prefix_width;
  const int32_t* prefix_length;
  float scale;
  void* out;
  int out_f16;
  int64_t ldo;
  float* partial;  // workspace, or null
};

// How a call is cut.  `own`: the sequences' own tokens, in up to own_parts
// parts of at least own_least tokens each; `front`: the prefix, the same.
// A workgroup takes 16 * tiles rows (its waves sharing the tokens) or, with
// rowsplit, four times as many (a wave's rows its own).
struct AttentionCut {
  int tiles, rowsplit, parts, least;
  int64_t row_groups;  // workgroups' rows per sequence (own) or in all (front)
};
struct AttentionPlan {
  AttentionCut own, front;
  int64_t slots;  // partial results of a row, 0: results are stored at once
};
bool attention_plan(const AttentionArgs& a, AttentionPlan* plan);
size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& plan);
hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, bool q_f16, hipStream_t st);

}  // namespace w4a4
