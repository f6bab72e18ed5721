// Internal launch interface of the operators of a decoding step: decode_api.cpp
// validates, w4a16.hip, cache.hip and attention*.hip run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

// Division of numbers below 2^31 by one that the host knows: q = (hi(n m) + n) >> s
// with s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.
struct Divisor {
  uint32_t d = 1, m = 1, s = 0;
  Divisor() = default;
  explicit Divisor(uint32_t v) : d(v) {
    while ((uint64_t{1} << s) < d) ++s;
    m = static_cast<uint32_t>((uint64_t{1} << 32) * ((uint64_t{1} << s) - d) / d + 1);
  }
  __host__ __device__ uint32_t quotient(uint32_t n) const {
    return (static_cast<uint32_t>(static_cast<uint64_t>(n) * m >> 32) + n) >> s;
  }
};

// ---- a projection with 4-bit weights and unquantized activations (w4a16.hip) ----
struct W4a16Args {
  const void* x;  // [M, K], row distance ldx
  int64_t ldx;
  const uint8_t* wq;
  int tiled;
  const void* sw;  // [N, K / group]
  int sw_f16;
  int64_t M, N;
  int K, groups;         // groups of K a channel, each with its scale
  Divisor group_halves;  // 64s of K to a group
  void* y;       // [M, N], row distance ldy
  int y_f16;
  int y_wide;    // rows of y allow stores of four elements
  int64_t ldy;
  float* partial;  // workspace: [parts][M][N], or null
};

// How a call is cut: 16 nb output channels to a workgroup (up to 16 rows) or a
// wave, 16 mt rows, K in parts that another launch adds up.
struct W4a16Plan {
  int nb, mt, parts;
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
  int tokens, q_heads;
  Divisor group;  // query heads to a cache head
  Divisor by_heads;  // heads
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

// How the tokens of the sequences (own), or of the prefix (front), are cut.
// Few rows (rowsplit 0): a workgroup takes the rows of a cache head, its
// waves sharing the tokens.  Tokens come in pieces of 2^piece_log2, and each of
// `groups` workgroups of a head takes an equal run of the pieces of all
// sequences (`groups` ones of the prefix).
// Many rows: it takes 64, a wave's 16 its own; `groups` is the row groups that a
// sequence (or all queries) can have, and their tokens are cut into up to
// `parts` equal parts of 2^piece_log2 or more.  Where sequences have far fewer
// queries than the longest, `places` row groups are numbered through over the
// queries there are (attention_kernel.h), else it is 0.
struct AttentionCut {
  int rowsplit, piece_log2;
  int one_piece;  // few rows: a workgroup of a head for every piece there can be
  Divisor groups;
  Divisor parts;
  int places;
};
struct AttentionPlan {
  AttentionCut own, front;
  int join;                  // partial results are joined by another launch
  int join_queries;          // of so many queries: all of q, or
  int join_by_place;         // max_q of every sequence
  int64_t own_slots;         // [own_slots][rows of a slot]: few rows: the runs' sections, many: the parts
  int64_t front_slots;
};
bool attention_plan(const AttentionArgs& a, AttentionPlan* plan);
size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& plan);
hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, bool q_f16, hipStream_t st);

}  // namespace w4a4
