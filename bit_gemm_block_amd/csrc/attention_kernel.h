// attention_kernel.h — softmax(c q . k) v of 16-row tiles over the quantized
// cache, one pass over the tokens.
//
// A wave takes 16 rows (a row: a query of one head of the group that shares the
// cache head) through steps of 32 tokens:
//
//   S^T = K Q^T   16 tokens x 16 rows an instruction; lane (row r, g) gets
//                 tokens 4 g + i of both halves of the step;
//   p = 2^(t - ref), t = c s_k S;   w = p s_v;
//   O^T += V^T W^T with the 32 tokens as the inner dimension, in the order in
//                 which the lanes hold them: nothing moves between lanes.
//
// Codes meet the matrix instruction as exact fp16 numbers, widened in
// registers as they come from memory: K's words hold eight channels of one
// token, V's of two tokens are paired by halves first.  A query is brought under
// a power of two of its row; a float32 one is a pair hi + lo of fp16 there, and
// so is w, so that no more than 2^-23 of either is lost.  (A single fp16 w would
// save an eighth of the many-row kernel's instructions and lose 2^-11 of every
// weight.)  All other numbers are float32.
//
// ref stands in for the running maximum: any reference gives the same
// quotient, and this one moves only when a weight |w| leaves 2^14 (fp16 ends at
// 2^16) or a sum of p leaves 2^60.  It then becomes the maximum of t + log2 s_v
// (s_v no less than 2^-60), minus 8, over the tokens seen.  The usual step
// exchanges nothing between lanes and rescales nothing.
//
// What bounds it.  Few rows: the cache's bytes.  64 sequences of 300 to 16384
// tokens, 8 heads of 128 at 4 bits (527 MB, 101 us at a large copy's rate, 88 at
// the rate at which a kernel can only read them) take 119 to 124 us, their join 5.
// Many rows: instructions.  A step of a wave is 24 to 32 matrix instructions (384
// to 512 cycles), about 150 others (700) and 20 KB of LDS, and they overlap
// little: 3 prompts of up to 1021 queries take 84 to 93 us beside 16 of the join, 17
// of them in matrix instructions.
#pragma once

#include <type_traits>

#include "decode_internal.h"
#include "int4_operands.h"
#include "vec_io.h"

namespace w4a4 {
namespace {

constexpr int kStep = 32;       // tokens of a step
constexpr int kAttnWaves = 4;   // of a workgroup

__host__ __device__ inline int64_t least64(int64_t a, int64_t b) { return a < b ? a : b; }

// Pieces of a range of L tokens (at most 2^30), one at least.
__host__ __device__ inline int pieces_of(int64_t L, const AttentionCut& c) {
  const uint32_t p = (static_cast<uint32_t>(L) + (1u << c.piece_log2) - 1) >> c.piece_log2;
  return static_cast<int>(p < 1 ? 1 : p);
}

// What a sequence (own tokens) or the prefix is to its queries.
struct Span {
  int64_t length;  // tokens
  int first, n;    // rows of q: the first, how many
  int rows;        // (query, head of the group) pairs that are computed
};

__device__ __forceinline__ int64_t clamp_length(int32_t v, int64_t cap) {
  const int64_t n = v;
  return n < 0 ? 0 : n < cap ? n : cap;
}

__device__ __forceinline__ Span own_span(const AttentionArgs& a, int s) {
  Span p;
  p.length = clamp_length(a.lengths[s], a.width << a.page_log2);
  int q0 = s, q1 = s + 1;
  if (a.q_start) {
    q0 = a.q_start[s];
    q1 = a.q_start[s + 1];
    q0 = q0 < 0 ? 0 : q0 < a.tokens ? q0 : a.tokens;
    q1 = q1 < q0 ? q0 : q1 < a.tokens ? q1 : a.tokens;
  }
  p.first = q0;
  p.n = q1 - q0;
  p.rows = (p.n < a.max_q ? p.n : a.max_q) * static_cast<int>(a.group.d);
  return p;
}

__device__ __forceinline__ Span front_span(const AttentionArgs& a) {
  Span p;
  p.length = clamp_length(a.prefix_length[0], a.prefix_width << a.page_log2);
  int q1 = a.seqs;
  if (a.q_start) {
    q1 = a.q_start[a.seqs];
    q1 = q1 < 0 ? 0 : q1 < a.tokens ? q1 : a.tokens;
  }
  p.first = 0;
  p.n = q1;
  p.rows = q1 * static_cast<int>(a.group.d);
  return p;
}

// The first sequence s for which bound(s + 1, q_start[s + 1]), which ascends, is
// above `target`; the number of sequences where none is.  64 of them at a time, by
// all lanes of a wave.
template <typename F>
__device__ __forceinline__ int first_above(const AttentionArgs& a, int target, F bound) {
  const int lane = threadIdx.x & 63;
  int first = 0, n = a.seqs;
  for (;;) {
    const int stride = (n + 63) >> 6;
    const int reach = (lane + 1) * stride;
    const int k = first + (reach < n ? reach : n);
    int q = a.q_start[k];
    q = q < 0 ? 0 : q < a.tokens ? q : a.tokens;
    const int below = __builtin_popcountll(__ballot(reach - stride < n && bound(k, q) <= target)) * stride;
    if (stride <= 1 || below >= n) return first + (below < n ? below : n);
    first += below;
    n = n - below < stride ? n - below : stride;
  }
}
// Row groups numbered through: those of sequence s begin at 64ths(q_start[s] group)
// + s.  64ths of a sum are no fewer than those of its parts, so that its n group
// rows have the 64ths(n group) + 1 places that they may need.
__device__ __forceinline__ int place_of(const AttentionArgs& a, int s, int q) {
  return static_cast<int>(static_cast<uint32_t>(q) * a.group.d >> 6) + s;
}

// Bytes 0 and 1, or 2 and 3, of w (unsigned codes u = q + 128) as fp16, minus 128.
template <bool UPPER>
__device__ __forceinline__ h2 two_bytes(uint32_t w) {
  const h2 off = {1152.f16, 1152.f16};
  return __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, w, UPPER ? 0x04030402u : 0x04010400u)) - off;
}

// A step's codes as a lane holds them: of the keys, its share of token r of both
// halves; of the values, its channels of tokens 4 g + i of both.
template <int D, int BITS>
struct Row {
  static constexpr int kBytes = D * BITS / 8;
  static constexpr int kKeyWords = kBytes / 16;                        // of each half
  static constexpr int kValueWords = kBytes >= 64 ? kBytes / 64 : 1;   // of each token
  static constexpr int kWords = 8 * kValueWords;                       // of either, at most
};
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* d) {
  if constexpr (WORDS == 1) {
    d[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    d[0] = w.x;
    d[1] = w.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const u4 w = *reinterpret_cast<const u4*>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i + e] = w[e];
    }
  }
}
// Of one half, whose first token is cache row rb.
template <int D, int BITS>
__device__ __forceinline__ void load_half_keys(const AttentionArgs& a, int64_t rb, uint32_t r, uint32_t g, uint32_t* k) {
  using X = Row<D, BITS>;
  load_words<X::kKeyWords>(a.k + rb * X::kBytes + (r * X::kBytes + g * (X::kBytes / 4)), k);
}
template <int D, int BITS>
__device__ __forceinline__ void load_half_values(const AttentionArgs& a, int64_t rb, uint32_t r, uint32_t g,
                                                 uint32_t* v) {
  using X = Row<D, BITS>;
  const uint8_t* first = a.v + rb * X::kBytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = first + (g * (4 * X::kBytes) + r * (X::kBytes / 16)) + i * X::kBytes;
    if constexpr (X::kBytes == 32)
      v[i] = *reinterpret_cast<const uint16_t*>(p);
    else
      load_words<X::kValueWords>(p, v + i * X::kValueWords);
  }
}
// rb: the cache rows of the halves' first tokens.
template <int D, int BITS>
__device__ __forceinline__ void load_keys(const AttentionArgs& a, const int64_t* rb, uint32_t r, uint32_t g,
                                          uint32_t* k) {
#pragma unroll
  for (int h = 0; h < 2; ++h) load_half_keys<D, BITS>(a, rb[h], r, g, k + h * Row<D, BITS>::kKeyWords);
}
template <int D, int BITS>
__device__ __forceinline__ void load_values(const AttentionArgs& a, const int64_t* rb, uint32_t r, uint32_t g,
                                            uint32_t* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) load_half_values<D, BITS>(a, rb[h], r, g, v + h * 4 * Row<D, BITS>::kValueWords);
}
// The scales of tokens 4 g + i of both halves.
__device__ __forceinline__ void load_scales(const float* s, const int64_t* rb, uint32_t g, f4* d) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    d[h] = *reinterpret_cast<const f4*>(s + rb[h] + 4 * g);
}

// K's codes 8 j to 8 j + 7 of a lane as fp16 (4 bits in the order 0 4 1 5 2 6 3 7).
// WHOLE: the whole numbers that they are.
// Else, of 4 bits, unsigned, as subnormal numbers u 2^-20, two fewer instructions
// for two codes: the bits of a small whole number are that times 2^-24.  Their
// offset of 8 is taken out of the product by its starting value.  The instruction
// aligns products by the exponent that subnormals share, 2^-14, and cuts what falls
// behind: codes stand high in their ten bits (as u 2^-24 they cost five bits of the
// scores), and 8 bits have no room to.
template <int BITS, bool WHOLE>
__device__ __forceinline__ h8 key_operand(const uint32_t* k, int j, const Masks& m) {
  Operand o;
  if constexpr (BITS == 4 && WHOLE) {
    o = int4_to_f16(k[j], m);
  } else if constexpr (BITS == 4) {
    o.w[0] = ((k[j] << 4) & m.odd) ^ m.key;
    o.w[1] = (k[j] & m.odd) ^ m.key;
    o.w[2] = ((k[j] >> 4) & m.odd) ^ m.key;
    o.w[3] = ((k[j] >> 8) & m.odd) ^ m.key;
  } else {
    const uint32_t a = k[2 * j] ^ 0x80808080u, b = k[2 * j + 1] ^ 0x80808080u;
    o.p[0] = two_bytes<false>(a);
    o.p[1] = two_bytes<true>(a);
    o.p[2] = two_bytes<false>(b);
    o.p[3] = two_bytes<true>(b);
  }
  return o.h;
}
// The channel of the element e of such an operand.
template <int BITS>
__device__ constexpr int key_channel(int e) {
  return BITS == 4 ? (e & 1) * 4 + e / 2 : e;
}
// What makes scores (over log 2) of products with a query brought up by 2^up.
template <bool WHOLE>
__device__ __forceinline__ float score_factor(const AttentionArgs& a, int up) {
  return ldexpf(a.scale * 1.4426950408889634f, (WHOLE ? 0 : 20) - up);
}

// Four channels of a lane's tokens in pairs (four of a step, two of a half), as
// fp16: channels 4 q to 4 q + 3 of the lane's own.  (An offset of the values cannot
// wait like the keys': it would be 8 times the sum of the weights, which the result
// is a small part of.)
template <int D, int BITS, int PAIRS = 4>
__device__ __forceinline__ void value_operands(const uint32_t* v, int q, const Masks& m, Operand* o) {
  constexpr int VW = Row<D, BITS>::kValueWords;
#pragma unroll
  for (int p = 0; p < PAIRS; ++p) {
    const int word = BITS == 4 ? q / 2 : q;
    const uint32_t w0 = v[2 * p * VW + word], w1 = v[(2 * p + 1) * VW + word];
    if constexpr (BITS == 4) {
      const uint32_t t = __builtin_amdgcn_perm(w1, w0, q % 2 ? 0x07060302u : 0x05040100u);
      nibbles_to_f16(t, m, &o[0].p[p], &o[1].p[p], &o[2].p[p], &o[3].p[p]);
    } else {
      const uint32_t lo = __builtin_amdgcn_perm(w1, w0, 0x05010400u) ^ 0x80808080u;  // bytes 0, 0, 1, 1
      const uint32_t hi = __builtin_amdgcn_perm(w1, w0, 0x07030602u) ^ 0x80808080u;  // 2, 2, 3, 3
      o[0].p[p] = two_bytes<false>(lo);
      o[1].p[p] = two_bytes<true>(lo);
      o[2].p[p] = two_bytes<false>(hi);
      o[3].p[p] = two_bytes<true>(hi);
    }
  }
}

// Two values as fp16, to nearest, and what that leaves of them.
__device__ __forceinline__ h2 two_halves(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f2{a, b}), h2);
}
__device__ __forceinline__ h2 remainders(h2 hi, float a, float b) {
  return two_halves(fmaf(static_cast<float>(hi[0]), -1.f, a), fmaf(static_cast<float>(hi[1]), -1.f, b));
}

// log2 of a scale's size, down to the integer, between 2^-60 and 2^127.
__device__ __forceinline__ float exponent(float v) {
  const int e = __builtin_amdgcn_frexp_expf(v);
  return fabsf(v) > 8.6736174e-19f ? static_cast<float>(e) : -60.f;
}

constexpr float kUnset = -__FLT_MAX__;  // reference of a row that has seen nothing: below any score

// What brings a sum under a reference higher by `by`: 2^-by in two steps.  Where
// values' sizes differ by 2^126 and more that is no number of its own, but a sum
// of weights under the lower reference may stand as high.
struct Lower {
  float half;
  __device__ __forceinline__ explicit Lower(float by) : half(__builtin_amdgcn_exp2f(-0.5f * by)) {}
  __device__ __forceinline__ float sum(float l) const { return l * half * half; }
  __device__ __forceinline__ float factor() const { return half * half; }
};

// What a row of lane (r, g) has gathered: lanes of one r share ref, and hold
// their own tokens' part of l and their channels of O.
template <int NV>
struct RowState {
  f4 o[NV];
  float ref, l;
  __device__ __forceinline__ void clear() {
    ref = kUnset;
    l = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) o[j] = f4{0.f, 0.f, 0.f, 0.f};
  }
};

// The weights of a step from its products sc, the keys' scales times the row's
// factor, kc, and the values' scales: hi and lo.  With `partly` positions from limit
// on, and those of absent pages, are not seen.
template <int NV>
__device__ __forceinline__ void weigh_step(const f4* sc, const float* kc_, const f4* vs_, bool partly, int limit,
                                           int tok, bool bad0, bool bad1, RowState<NV>& s, Operand* w) {
  float x[8], kc[8], vs[8], wt[8], sum, top;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = sc[i / 4][i % 4];
    kc[i] = kc_[i];
    vs[i] = vs_[i / 4][i % 4];
  }
  if (partly) {
    asm volatile("");  // a branch, not forty selects in every step
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (tok + 16 * (i / 4) + i % 4 >= limit || (i < 4 ? bad0 : bad1)) {  // whatever the scales there are
        x[i] = -INFINITY;
        kc[i] = 1.f;
        vs[i] = 0.f;
      }
    }
  }
  auto weigh = [&]() {
    sum = 0.f;
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = __builtin_amdgcn_exp2f(fmaf(x[i], kc[i], -s.ref));
      wt[i] = p * vs[i];
      sum += p;
      top = fmaxf(top, fabsf(wt[i]));
    }
  };
  weigh();
  const uint64_t lanes = __ballot(top > 16384.f || sum > 1.15292150e18f);
  if (lanes) {
    // Of this row: others, which may be of other sequences, leave it as it is.
    const uint32_t pairs = static_cast<uint32_t>(lanes | lanes >> 32);
    const bool far = ((pairs | pairs >> 16) >> (threadIdx.x & 15) & 1) != 0;
    float u = kUnset;
#pragma unroll
    for (int i = 0; i < 8; ++i) u = fmaxf(u, fmaf(x[i], kc[i], exponent(vs[i])));
    u = fmaxf(u, __shfl_xor(u, 16));
    u = fmaxf(u, __shfl_xor(u, 32));
    const float moved = far ? fmaxf(s.ref, u - 8.f) : s.ref;
    const Lower lower(moved - s.ref);
    s.ref = moved;
    s.l = lower.sum(s.l);
#pragma unroll
    for (int j = 0; j < NV; ++j) s.o[j] *= lower.factor();
    weigh();
  }
  s.l += sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[0].p[i] = two_halves(wt[2 * i], wt[2 * i + 1]);
    w[1].p[i] = remainders(w[0].p[i], wt[2 * i], wt[2 * i + 1]);
  }
}

struct Sight {
  int length, n;
  bool all;
  __device__ __forceinline__ Sight(const AttentionArgs& a, const Span& span, int front)
      : length(static_cast<int>(span.length)), n(span.n), all(front || !a.causal) {}
  // Positions below this are what a query sees.
  __device__ __forceinline__ int limit(int query) const {
    const int l = length - n + query + 1;
    return all ? length : l < 0 ? 0 : l;
  }
};

// The pages of up to 32 steps, lane 2 i + half holding that of step first + i
// stride: no wait for the table stands between a step and its loads.  -1: no
// such page.
struct Pages {
  const int32_t* table;
  int end;  // tokens that it has pages for
  __device__ __forceinline__ Pages(const AttentionArgs& a, int s, int front)
      : table(front ? a.prefix_table : a.tables + s * a.width),
        end(static_cast<int>((front ? a.prefix_width : a.width) << a.page_log2)) {}
  __device__ __forceinline__ int32_t raw(const AttentionArgs& a, int first, int stride, int lane) const {
    int tok = (first + (lane >> 1) * stride) * kStep + 16 * (lane & 1);
    tok = tok < end && tok >= 0 ? tok : end - 16;
    return end > 0 ? table[tok >> a.page_log2] : -1;
  }
  static __device__ __forceinline__ int32_t checked(const AttentionArgs& a, int32_t p) {
    return p >= 0 && p < a.pages ? p : -1;
  }
};
// The cache row of a half step's first token, in page p.
__device__ __forceinline__ int64_t half_row(const AttentionArgs& a, int h, int step, int half, int32_t p) {
  const int off = (step * kStep + 16 * half) & ((1 << a.page_log2) - 1);
  return ((static_cast<int64_t>(p < 0 ? 0 : p) * a.heads + h) << a.page_log2) + off;
}
// The cache rows of the halves of a step in pages p0 and p1.
__device__ __forceinline__ void rows_of(const AttentionArgs& a, int h, int step, int32_t p0, int32_t p1, int64_t* rb) {
  rb[0] = half_row(a, h, step, 0, p0);
  rb[1] = half_row(a, h, step, 1, p1);
}

// A lane's channels [g D / 4, +D / 4) of a row of queries.
template <int D, typename Q>
__device__ __forceinline__ void load_query(const AttentionArgs& a, const Span& span, int h, int row, int g,
                                           Raw8<Q>* x) {
  row = row < span.rows ? row : 0;
  const int query = a.group.quotient(row);
  const int64_t at = static_cast<int64_t>(span.first + query) * a.ldq +
                     static_cast<int64_t>(h * a.group.d + row - query * a.group.d) * D + g * (D / 4);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) x[j].load(static_cast<const Q*>(a.q) + at + 8 * j);
}
// The power of two that brings the row's largest below 2^14.
template <int D, typename Q>
__device__ __forceinline__ int query_shift(const Raw8<Q>* x) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[j].get(e)));
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  return m > 0.f && m < INFINITY ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;
}
// Eight channels as operands in the codes' order.
template <int BITS, typename Q>
__device__ __forceinline__ void query_operands(const Raw8<Q>& x, int up, Operand* hi, Operand* lo) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float v0 = ldexpf(x.get(key_channel<BITS>(e)), up);
    const float v1 = ldexpf(x.get(key_channel<BITS>(e + 1)), up);
    hi->p[e / 2] = two_halves(v0, v1);
    lo->p[e / 2] = remainders(hi->p[e / 2], v0, v1);
  }
}
// The offset of 4-bit codes as an operand: a product with it is what it adds.
__device__ __forceinline__ h8 offset_operand() {
  Operand o;
#pragma unroll
  for (int p = 0; p < 4; ++p) o.w[p] = 0x00800080u;  // 16 times 8
  return o.h;
}

// Partial results: rows of D float32 (O), of the own tokens' slots and then of the
// prefix's, after them (ref, l) of each, after these, per sequence and for the
// prefix, its first slot and their number.
struct Partial {
  int64_t own_rows, rows;
  __device__ __forceinline__ Partial(const AttentionArgs& a, const AttentionPlan& p)
      : own_rows(p.own_slots * (p.own.rowsplit ? a.tokens : a.max_q) * a.q_heads),
        rows(own_rows + p.front_slots * a.tokens * a.q_heads) {}
  // The row of a slot: own tokens of few rows are kept by their place in the
  // sequence, others by their token.
  __device__ __forceinline__ int64_t row(const AttentionArgs& a, const AttentionPlan& p, bool front, int64_t slot,
                                         int64_t token, int query, int head) const {
    const bool by_place = !front && !p.own.rowsplit;
    const int64_t at = slot * (by_place ? a.max_q : a.tokens) + (by_place ? query : token);
    return (front ? own_rows : 0) + at * a.q_heads + head;
  }
  __device__ __forceinline__ float* o(const AttentionArgs& a, int64_t row) const { return a.partial + row * a.D; }
  __device__ __forceinline__ float* stat(const AttentionArgs& a, int64_t row) const {
    return a.partial + rows * a.D + row * 2;
  }
  __device__ __forceinline__ int32_t* slots(const AttentionArgs& a, int s) const {
    return reinterpret_cast<int32_t*>(a.partial + rows * (a.D + 2)) + 2 * s;
  }
};

// Few rows: the waves of a workgroup share its 16 rows and take every fourth
// step each.  The workgroups that fit the chip at once take equal runs of all
// sequences' tokens: with parts of one sequence each, as many as the longest
// needs, 64 sequences of 300 to 16384 tokens took 148 us for 117, since short
// ones leave and long ones start late.  The queries' operands stay in LDS: in
// registers they would leave two workgroups a compute unit for three.
template <int D, bool PAIR>
struct TokensLds {
  typedef u4 Queries[D / 32][PAIR ? 2 : 1][64];
  // Where two workgroups would not fit a compute unit's 160 KB, the queries lie
  // where the waves' shares come to lie.
  static constexpr bool kShare = D == 256 && PAIR;
  f4 o[kAttnWaves][D / 16][64];
  float stat[kAttnWaves][16][2];
  u4 apart[kShare ? 1 : sizeof(Queries) / 16];
  __device__ __forceinline__ Queries& queries() {
    return *reinterpret_cast<Queries*>(kShare ? static_cast<void*>(o) : static_cast<void*>(apart));
  }
};
// Inclusive sums along the lanes.
__device__ __forceinline__ int sum_to_lane(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row 0 to 1, 2 to 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2, 3
  return v;
}

// A workgroup's run of pieces, and the sequence in which it begins.
struct Run {
  int first, end;   // pieces of all sequences
  int s, start;     // the sequence, and its first piece
  int each;         // pieces to a workgroup
  __device__ __forceinline__ Run(const AttentionArgs& a, const AttentionCut& cut, int front, int w, int lane) {
    const int seqs = front ? 1 : a.seqs;
    const int64_t cap = (front ? a.prefix_width : a.width) << a.page_log2;
    const int32_t* lengths = front ? a.prefix_length : a.lengths;
    auto pieces = [&](int i) { return i < seqs ? pieces_of(clamp_length(lengths[i], cap), cut) : 0; };
    const int mine = pieces(lane);
    int all = mine;
    for (int i = 64 + lane; i < seqs; i += 64) all += pieces(i);
    all = __builtin_amdgcn_readlane(sum_to_lane(all), 63);
    each = cut.groups.quotient(all + cut.groups.d - 1);
    first = w * each;
    end = first + each < all ? first + each : all;
    s = start = 0;
    for (int base = 0; base < seqs && first < end; base += 64) {
      const int n = base == 0 ? mine : pieces(base + lane);
      const int to = start + sum_to_lane(n);
      const uint64_t here = __ballot(to > first);
      if (here) {
        const int i = __builtin_ctzll(here);
        s = base + i;
        start = __builtin_amdgcn_readlane(to - n, i);
        break;
      }
      start = __builtin_amdgcn_readlane(to, 63);
    }
  }
};

// A section of a run: pieces [from, to) of sequence s.  whole: 1 if these are all
// and there is no prefix, -1 if that is still to be found out.
template <int D, int BITS, bool PAIR>
__device__ __forceinline__ void tokens_section(const AttentionArgs& a, const AttentionPlan& plan, int front, int h,
                                               int s, int from, int to, int whole, int slot,
                                               TokensLds<D, PAIR>& lds) {
  constexpr int NK = D / 32;   // instructions along a head's channels
  constexpr int NV = D / 16;   // channels of O a lane's row block holds
  constexpr int HALVES = PAIR ? 2 : 1;
  const AttentionCut& cut = front ? plan.front : plan.own;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int begin = (from << (cut.piece_log2 - 5)) + wave;
  // Pages and queries are on their way together.
  const Pages table(a, s, front);
  int32_t pages = table.raw(a, begin, kAttnWaves, lane);
  const Span span = front ? front_span(a) : own_span(a, s);
  if (span.rows <= 0) return;
  using Q = std::conditional_t<PAIR, float, _Float16>;
  Raw8<Q> x[NK];
  load_query<D>(a, span, h, r, g, x);

  if (whole < 0) {
    const int n = pieces_of(span.length, cut);
    if (from >= n) return;
    whole = n == 1 && !front && !a.prefix_table;
    if (plan.join && from == 0 && h == 0 && threadIdx.x == 0) {
      int32_t* m = Partial(a, plan).slots(a, front ? a.seqs : 0);
      m[0] = 0;
      m[1] = n;
    }
  }
  const Sight sight(a, span, front);
  const int all_see = 16 <= span.rows ? sight.limit(0) : 0;  // what every row sees
  const int steps = (sight.limit(a.group.quotient(span.rows - 1)) + kStep - 1) / kStep;
  const int stop = to << (cut.piece_log2 - 5);
  const int end = stop < steps ? stop : steps;
  const int limit = r < span.rows ? sight.limit(a.group.quotient(r)) : 0;

  constexpr int KW = Row<D, BITS>::kKeyWords;
  uint32_t keys[2 * KW], values[Row<D, BITS>::kWords];
  f4 ks[2], vs[2];
  int64_t rb[2];
  int32_t p0 = 0, p1 = 0;  // of the step whose keys are loaded
  pages = Pages::checked(a, pages);
  if (begin < end) {
    p0 = __builtin_amdgcn_readlane(pages, 0);
    p1 = __builtin_amdgcn_readlane(pages, 1);
    rows_of(a, h, begin, p0, p1, rb);
    load_keys<D, BITS>(a, rb, r, g, keys);
    load_scales(a.ks, rb, g, ks);
    load_values<D, BITS>(a, rb, r, g, values);
    load_scales(a.vs, rb, g, vs);
  }

  // With codes as whole numbers a score is one sum over both parts of a query.  With
  // unsigned ones that sum would be rounded at the size of the offset's, three times
  // the score's: the two parts are summed apart, the first nearly exact and the
  // second too small for its roundings to count, and then added (64 sequences of 300
  // to 16384 tokens, 4 bits: outputs off by 1.2e-6 of themselves in one sum, 3.3e-7 in
  // two, for 0.8 us of 125).
  constexpr bool WHOLE = BITS == 8;
  constexpr int SUMS = WHOLE ? 1 : HALVES;
  // The queries go to LDS as operands, a wave's share of the channels each; c
  // makes scores (over log 2) of the products.
  const int up = query_shift<D>(x);
  const float c = score_factor<WHOLE>(a, up);
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    if (j % kAttnWaves != wave) continue;
    Operand hi, lo;
    query_operands<BITS>(x[j], up, &hi, &lo);
    lds.queries()[j][0][lane] = u4{hi.w[0], hi.w[1], hi.w[2], hi.w[3]};
    if constexpr (PAIR) lds.queries()[j][1][lane] = u4{lo.w[0], lo.w[1], lo.w[2], lo.w[3]};
  }
  __syncthreads();
  auto query_operand = [&](int j, int p) { return __builtin_bit_cast(h8, lds.queries()[j][p][lane]); };
  // The products start from what the codes' offset adds to them, taken off.
  f4 start[SUMS];
#pragma unroll
  for (int p = 0; p < SUMS; ++p) {
    start[p] = f4{0.f, 0.f, 0.f, 0.f};
    if constexpr (WHOLE) continue;
#pragma unroll
    for (int j = 0; j < NK; ++j)
      start[p] = __builtin_amdgcn_mfma_f32_16x16x32_f16(offset_operand(), query_operand(j, p), start[p], 0, 0, 0);
    start[p] = -start[p];
  }

  RowState<NV> state;
  state.clear();
  const Masks masks;

  int turn = 0;  // steps into the 32 whose pages are at hand
  // A step; all but the last bring the next one's keys in while the softmax and
  // the second product run, and its values at the end.  (A condition around the
  // loads would make every wait one for all of them.)
  auto take = [&](int step, auto last_step) {
    constexpr bool LAST = decltype(last_step)::value;
    const bool bad0 = p0 < 0, bad1 = p1 < 0;
    const bool partly = bad0 || bad1 || (step + 1) * kStep > all_see;  // some row does not see some token

    asm volatile("" ::: "memory");  // the queries are read again, not kept in registers
    f4 part[SUMS][2];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      h8 k[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) k[half] = key_operand<BITS, WHOLE>(keys + half * KW, j, masks);
#pragma unroll
      for (int p = HALVES - 1; p >= 0; --p) {
        const h8 q = query_operand(j, p);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool first = j == 0 && (SUMS == HALVES || p == HALVES - 1);
          f4& d = part[p % SUMS][half];
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[half], q, first ? start[p % SUMS] : d, 0, 0, 0);
        }
      }
    }
    f4 sc[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) sc[half] = SUMS == 2 ? part[0][half] + part[SUMS - 1][half] : part[0][half];
    float kc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) kc[i] = ks[i / 4][i % 4] * c;
    if constexpr (!LAST) {
      if (++turn == 32) {
        pages = Pages::checked(a, table.raw(a, step + kAttnWaves, kAttnWaves, lane));
        turn = 0;
      }
      p0 = __builtin_amdgcn_readlane(pages, 2 * turn);
      p1 = __builtin_amdgcn_readlane(pages, 2 * turn + 1);
      rows_of(a, h, step + kAttnWaves, p0, p1, rb);
      load_keys<D, BITS>(a, rb, r, g, keys);
      load_scales(a.ks, rb, g, ks);
    }

    Operand w[2];
    weigh_step<NV>(sc, kc, vs, partly, limit, step * kStep + 4 * g, bad0, bad1, state, w);

#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      Operand v[4];
      value_operands<D, BITS>(values, j, masks, v);
#pragma unroll
      for (int p = 1; p >= 0; --p)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          state.o[4 * j + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[e].h, w[p].h, state.o[4 * j + e], 0, 0, 0);
    }
    if constexpr (!LAST) {
      load_values<D, BITS>(a, rb, r, g, values);
      load_scales(a.vs, rb, g, vs);
    }
  };
  if (begin < end) {
    int step = begin;
    for (; step + kAttnWaves < end; step += kAttnWaves) take(step, std::false_type{});
    take(step, std::true_type{});
  }

  // The waves' shares are brought to one reference and added up, in the order of
  // the waves, each wave taking a quarter of the channels.
  if constexpr (TokensLds<D, PAIR>::kShare) __syncthreads();  // the queries are used up
  float own = state.l;
  own += __shfl_xor(own, 16);
  own += __shfl_xor(own, 32);
  if (g == 0) {
    lds.stat[wave][r][0] = state.ref;
    lds.stat[wave][r][1] = own;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) lds.o[wave][j][lane] = state.o[j];
  __syncthreads();
  float top = kUnset, f[kAttnWaves], l = 0.f;
#pragma unroll
  for (int k = 0; k < kAttnWaves; ++k) top = fmaxf(top, lds.stat[k][r][0]);
#pragma unroll
  for (int k = 0; k < kAttnWaves; ++k) {
    const Lower lower(top - lds.stat[k][r][0]);
    f[k] = lower.factor();
    l += lower.sum(lds.stat[k][r][1]);
  }
  // Channels of this wave: its quarter of each lane's NV (i, 0 .. NV - 1).
  constexpr int Q4 = NV / 4;
  f4 sum[Q4];
#pragma unroll
  for (int j = 0; j < Q4; ++j) {
    sum[j] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kAttnWaves; ++k) sum[j] += f[k] * lds.o[k][wave * Q4 + j][lane];
  }
  if (r >= span.rows) return;
  const int query = a.group.quotient(r);
  const int64_t token = span.first + query;
  const int head = h * a.group.d + r - query * a.group.d;
  const int channel = g * (D / 4) + wave * Q4;  // + NV i + j
  if (whole) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t to = token * a.ldo + static_cast<int64_t>(head) * D + channel;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < Q4; ++j) {
        if (a.out_f16)
          static_cast<_Float16*>(a.out)[to + NV * i + j] = static_cast<_Float16>(sum[j][i] * inv);
        else
          static_cast<float*>(a.out)[to + NV * i + j] = sum[j][i] * inv;
      }
  } else {
    const Partial partial(a, plan);
    const int64_t at = partial.row(a, plan, front, slot, token, query, head);
    float* po = partial.o(a, at) + channel;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < Q4; ++j) po[NV * i + j] = sum[j][i];
    if (g == 0 && wave == 0) {
      float* st = partial.stat(a, at);
      st[0] = top;
      st[1] = l;
    }
  }
}
template <int D, int BITS, bool PAIR>
__device__ __forceinline__ void tokens_body(const AttentionArgs& a, const AttentionPlan& plan, int front,
                                            uint32_t block, TokensLds<D, PAIR>& lds) {
  const AttentionCut& cut = front ? plan.front : plan.own;
  const int lane = threadIdx.x & 63;
  const int w = a.by_heads.quotient(block), h = block - w * a.heads;
  const bool single = (front || a.seqs == 1) && cut.one_piece;  // its table need not wait for its length
  int s = 0, start = 0, from = w, end = w + 1, each = 1;
  if (!single) {
    const Run run(a, cut, front, w, lane);
    s = run.s;
    start = run.start;
    from = run.first;
    end = run.end;
    each = run.each;
  }
  const int first = from;
  for (; from < end; ++s) {
    int to = end, whole = -1, n = 0;
    if (!single) {
      const int64_t cap = (front ? a.prefix_width : a.width) << a.page_log2;
      n = pieces_of(clamp_length((front ? a.prefix_length : a.lengths)[s], cap), cut);
      to = end < start + n ? end : start + n;
      const bool all = from == start && to == start + n;
      whole = all && !front && !a.prefix_table;
      // Slots of a sequence follow one another: its runs, counted from its number.
      if (plan.join && from == start && h == 0 && threadIdx.x == 0) {
        int32_t* m = Partial(a, plan).slots(a, front ? a.seqs : s);
        m[0] = front ? 0 : w + s;
        m[1] = all ? 1 : static_cast<int>(static_cast<uint32_t>(start + n - 1) / static_cast<uint32_t>(each)) - w + 1;
      }
      if (from > first) __syncthreads();  // the section before has left LDS
    }
    tokens_section<D, BITS, PAIR>(a, plan, front, h, s, from - start, to - start, whole, front ? w : w + s, lds);
    from = to;
    start += n;
  }
}
template <int D, int BITS, bool PAIR>
__global__ void __launch_bounds__(kAttnWaves * 64, D == 256 ? 2 : 3)
    attention_tokens_kernel(AttentionArgs a, AttentionPlan plan, int front) {
  __shared__ TokensLds<D, PAIR> lds;
  tokens_body<D, BITS, PAIR>(a, plan, front, blockIdx.x, lds);
}

// Many rows: a wave's 16 rows are its own, and the waves share the widening.
// Two steps at a time (a block) go through LDS as operands, each wave bringing
// the keys and values of half a step, and all waves multiply all.  The codes of
// two more blocks are on their way meanwhile.  (Keys to two waves and values to
// the others, one block ahead: 102 us for 98 at 3 prompts of up to 1021 queries.
// Two row tiles a wave, which read LDS half as often but leave two waves to a
// SIMD for three: 188.  Four waves at the price of one block ahead: 111.)
template <int D>
struct RowsLds {
  static constexpr int kBlock = 2;
  u4 k[kBlock][2][D / 32][64];
  u4 v[kBlock][D / 16][64];
  f4 ks[kBlock][8], vs[kBlock][8];
};
constexpr int kGroupRows = 16 * kAttnWaves;

// Parts of a range of L tokens.
__device__ __forceinline__ int parts_of(int64_t L, const AttentionCut& c) {
  const uint32_t p = static_cast<uint32_t>(L) >> c.piece_log2;
  return static_cast<int>(p < 1 ? 1 : p < c.parts.d ? p : c.parts.d);
}

template <int D, int BITS, bool PAIR>
__device__ __forceinline__ void rows_body(const AttentionArgs& a, const AttentionPlan& plan, int front,
                                          uint32_t place, RowsLds<D>& lds) {
  constexpr int NK = D / 32, NV = D / 16;
  constexpr int BLOCK = RowsLds<D>::kBlock;
  constexpr int HALVES = PAIR ? 2 : 1;
  const AttentionCut& cut = front ? plan.front : plan.own;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroup (part, s, rg, h), h fastest, so that those of one length lie
  // together; late row groups, which see most, first.  (s, rg) counts the row groups
  // that the longest sequence has for each, or those there are.
  uint32_t id = a.by_heads.quotient(place);
  const int h = place - id * a.heads;
  int part, s, rg;
  const bool through = !front && cut.places;
  if (through) {
    part = id / static_cast<uint32_t>(cut.places);
    const int at = id - part * cut.places;
    s = __builtin_amdgcn_readfirstlane(first_above(a, at, [&](int k, int q) { return place_of(a, k, q); }));
    if (s >= a.seqs) return;
    rg = at;  // from its sequence's first on, below
  } else {
    const uint32_t rest = cut.groups.quotient(id);
    rg = cut.groups.d - 1 - (id - rest * cut.groups.d);
    const uint32_t seqs = front ? 1 : a.seqs;
    part = rest / seqs;
    s = rest - part * seqs;
  }
  const Pages table(a, s, front);
  const Span span = front ? front_span(a) : own_span(a, s);
  if (through) rg = (span.rows + kGroupRows - 1) / kGroupRows - 1 - (rg - place_of(a, s, span.first));
  if (rg < 0 || rg * kGroupRows >= span.rows) return;
  const int parts = parts_of(span.length, cut);
  if (part >= parts) return;
  if (plan.join && part == 0 && rg == 0 && h == 0 && threadIdx.x == 0) {
    int32_t* m = Partial(a, plan).slots(a, front ? a.seqs : s);
    m[0] = 0;
    m[1] = parts;
  }
  const int row = rg * kGroupRows + wave * 16 + r;  // of this lane

  const Sight sight(a, span, front);
  const int first = row - r;  // of this wave
  const int last = (first + 16 < span.rows ? first + 16 : span.rows) - 1;
  const int group_last = ((rg + 1) * kGroupRows < span.rows ? (rg + 1) * kGroupRows : span.rows) - 1;
  const int wave_steps = last >= first ? (sight.limit(a.group.quotient(last)) + kStep - 1) / kStep : 0;
  const int all_see = first + 16 <= span.rows ? sight.limit(a.group.quotient(first)) : 0;
  const int limit = row < span.rows ? sight.limit(a.group.quotient(row)) : 0;
  const int steps = (sight.limit(a.group.quotient(group_last)) + kStep - 1) / kStep;
  const int share =
      parts == 1 ? steps : static_cast<int>(static_cast<uint32_t>(steps + parts - 1) / static_cast<uint32_t>(parts));
  const int begin = part * share;
  const int end = begin + share < steps ? begin + share : steps;

  int32_t pages = table.raw(a, begin, 1, lane), ahead = 0;  // of the 32 steps at hand and of the next
  using Q = std::conditional_t<PAIR, float, _Float16>;
  Raw8<Q> x[NK];
  load_query<D>(a, span, h, row, g, x);

  // This wave brings half `half` of step `mine` of each block; DEPTH blocks at a
  // time are on their way (one where two would not fit the registers).  Without
  // conditions: a wait for one set's loads must not become one for all.
  constexpr int DEPTH = BITS == 8 && (PAIR || D == 256) ? 1 : 2;
  const int mine = wave & 1, half = wave >> 1;
  constexpr int KW = Row<D, BITS>::kKeyWords, VW = 4 * Row<D, BITS>::kValueWords;
  uint32_t keys[DEPTH][KW], values[DEPTH][VW];
  float scale[DEPTH];  // of token lane % 16: lanes 0 to 15 the keys', 16 to 31 the values'
  const float* const scales = lane & 16 ? a.vs : a.ks;
  auto bring = [&](int set, int step, int32_t from, int turn) {
    const int64_t rb = half_row(a, h, step, half, __builtin_amdgcn_readlane(from, 2 * turn + half));
    load_half_keys<D, BITS>(a, rb, r, g, keys[set]);
    load_half_values<D, BITS>(a, rb, r, g, values[set]);
    scale[set] = scales[rb + r];
  };
  const int last_step = end - 1;
  pages = Pages::checked(a, pages);
  if (begin < end) {
#pragma unroll
    for (int set = 0; set < DEPTH; ++set) {
      const int step = begin + set * BLOCK + mine < last_step ? begin + set * BLOCK + mine : last_step;
      bring(set, step, pages, step - begin);
    }
  }

  constexpr bool WHOLE = BITS == 8 || PAIR;  // as above; the widening is shared, and there are no registers for two sums
  Operand q[NK][HALVES];
  const int up = query_shift<D>(x);
  const float c = score_factor<WHOLE>(a, up);
  f4 start = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NK; ++j) {
    Operand lo;
    query_operands<BITS>(x[j], up, &q[j][0], &lo);
    if constexpr (PAIR) q[j][1] = lo;
    if constexpr (!WHOLE) start = __builtin_amdgcn_mfma_f32_16x16x32_f16(offset_operand(), q[j][0].h, start, 0, 0, 0);
  }
  start = -start;
  RowState<NV> state;
  state.clear();
  const Masks masks;

  auto take = [&](int block, int set) {
    const int turn = (block - begin) & 31;
    if (turn == 0 && block > begin) pages = ahead;
    __syncthreads();  // the block before is used up
#pragma unroll
    for (int j = 0; j < NK; ++j)
      lds.k[mine][half][j][lane] = __builtin_bit_cast(u4, key_operand<BITS, WHOLE>(keys[set], j, masks));
#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      Operand v[4];
      value_operands<D, BITS, 2>(values[set], j, masks, v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<uint2*>(&lds.v[mine][4 * j + e][lane])[half] = uint2{v[e].w[0], v[e].w[1]};
    }
    if (lane < 32) reinterpret_cast<float*>(lane & 16 ? lds.vs[mine] : lds.ks[mine])[16 * half + r] = scale[set];
    const int next = block + DEPTH * BLOCK - begin;  // to be brought, from begin
    if ((next & 31) == 0 && next + begin < end) ahead = Pages::checked(a, table.raw(a, next + begin, 1, lane));
    const int step = next + begin + mine < last_step ? next + begin + mine : last_step;
    bring(set, step, (step - begin) >> 5 == (block - begin) >> 5 ? pages : ahead, (step - begin) & 31);
    __syncthreads();

#pragma unroll
    for (int b = 0; b < BLOCK; ++b) {
      const int step = block + b;
      if (step >= end || step >= wave_steps) break;
      const bool bad0 = __builtin_amdgcn_readlane(pages, 2 * (turn + b)) < 0;
      const bool bad1 = __builtin_amdgcn_readlane(pages, 2 * (turn + b) + 1) < 0;
      const bool partly = bad0 || bad1 || (step + 1) * kStep > all_see;
      f4 sc[2];
#pragma unroll
      for (int j = 0; j < NK; ++j) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const h8 k = __builtin_bit_cast(h8, lds.k[b][half][j][lane]);
#pragma unroll
          for (int p = HALVES - 1; p >= 0; --p)
            sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[j][p].h, j == 0 && p == HALVES - 1 ? start : sc[half],
                                                              0, 0, 0);
        }
      }
      const f4 ks[2] = {lds.ks[b][g], lds.ks[b][4 + g]}, vs[2] = {lds.vs[b][g], lds.vs[b][4 + g]};
      float kc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) kc[i] = ks[i / 4][i % 4] * c;
      Operand w[2];
      weigh_step<NV>(sc, kc, vs, partly, limit, step * kStep + 4 * g, bad0, bad1, state, w);
#pragma unroll
      for (int j0 = 0; j0 < NV; j0 += 4) {
        h8 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(h8, lds.v[b][j0 + j][lane]);
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            state.o[j0 + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[j], w[p].h, state.o[j0 + j], 0, 0, 0);
      }
    }
  };
  for (int block = begin; block < end; block += DEPTH * BLOCK) {
    take(block, 0);
    if (DEPTH == 1 || block + BLOCK >= end) continue;
    take(block + BLOCK, DEPTH - 1);
  }

  state.l += __shfl_xor(state.l, 16);
  state.l += __shfl_xor(state.l, 32);
  if (row >= span.rows) return;
  const int query = a.group.quotient(row);
  const int64_t token = span.first + query;
  const int head = h * a.group.d + row - query * a.group.d;
  // Lane (r, g) holds channels [g D / 4, +D / 4): NV i + j is o[j][i].
  if (parts == 1 && !front && !a.prefix_table) {
    const float f = state.l == 0.f ? 0.f : 1.f / state.l;
    const int64_t at = token * a.ldo + static_cast<int64_t>(head) * D + g * (D / 4);
#pragma unroll
    for (int e = 0; e < D / 4; e += 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = state.o[(e + k) % NV][(e + k) / NV] * f;
      if (a.out_f16)
        store_whole8(static_cast<_Float16*>(a.out) + at + e, v);
      else
        store_whole8(static_cast<float*>(a.out) + at + e, v);
    }
  } else {
    const Partial partial(a, plan);
    const int64_t at = partial.row(a, plan, front, part, token, query, head);
    float* po = partial.o(a, at) + g * (D / 4);
#pragma unroll
    for (int e = 0; e < D / 4; e += 4)
      *reinterpret_cast<f4*>(po + e) = f4{state.o[e % NV][e / NV], state.o[(e + 1) % NV][(e + 1) / NV],
                                          state.o[(e + 2) % NV][(e + 2) / NV], state.o[(e + 3) % NV][(e + 3) / NV]};
    if (g == 0) {
      float* f = partial.stat(a, at);
      f[0] = state.ref;
      f[1] = state.l;
    }
  }
}
// Workgroups to a compute unit; the widest variant would keep registers in memory
// with two.
constexpr int rows_resident(int D, int bits, bool pair) { return D < 256 ? 3 : pair && bits == 8 ? 1 : 2; }
template <int D, int BITS, bool PAIR>
__global__ void __launch_bounds__(kAttnWaves * 64, rows_resident(D, BITS, PAIR))
    attention_rows_kernel(AttentionArgs a, AttentionPlan plan, int front) {
  __shared__ RowsLds<D> lds;
  rows_body<D, BITS, PAIR>(a, plan, front, blockIdx.x, lds);
}

// A prefix with many rows and own tokens with few, as in decoding: both in one
// launch, the prefix's workgroups first.
template <int D, int BITS, bool PAIR>
__global__ void __launch_bounds__(kAttnWaves * 64, rows_resident(D, BITS, PAIR))
    attention_both_kernel(AttentionArgs a, AttentionPlan plan, uint32_t front_blocks) {
  __shared__ union Lds {
    RowsLds<D> rows;
    TokensLds<D, PAIR> tokens;
    __device__ Lds() {}
  } lds;
  if (blockIdx.x < front_blocks)
    rows_body<D, BITS, PAIR>(a, plan, 1, blockIdx.x, lds.rows);
  else
    tokens_body<D, BITS, PAIR>(a, plan, 0, blockIdx.x - front_blocks, lds.tokens);
}

// Workgroups of a cut.
inline int64_t cut_blocks(const AttentionArgs& a, const AttentionCut& c, int64_t seqs) {
  if (!c.rowsplit) return a.heads * static_cast<int64_t>(c.groups.d);
  return a.heads * (c.places ? c.places : seqs * c.groups.d) * c.parts.d;
}

template <int D, int BITS, bool PAIR>
void launch_cut(const AttentionArgs& a, const AttentionPlan& plan, int front, hipStream_t st) {
  const AttentionCut& c = front ? plan.front : plan.own;
  const dim3 block(kAttnWaves * 64), grid(static_cast<unsigned>(cut_blocks(a, c, front ? 1 : a.seqs)));
  if (c.rowsplit) {
    hipLaunchKernelGGL((attention_rows_kernel<D, BITS, PAIR>), grid, block, 0, st, a, plan, front);
    return;
  }
  hipLaunchKernelGGL((attention_tokens_kernel<D, BITS, PAIR>), grid, block, 0, st, a, plan, front);
}

template <int D, int BITS, bool PAIR>
void launch_parts(const AttentionArgs& a, const AttentionPlan& plan, hipStream_t st) {
  if (a.prefix_table && plan.front.rowsplit && !plan.own.rowsplit) {
    const int64_t front = cut_blocks(a, plan.front, 1);
    const dim3 grid(static_cast<unsigned>(front + cut_blocks(a, plan.own, a.seqs)));
    hipLaunchKernelGGL((attention_both_kernel<D, BITS, PAIR>), grid, dim3(kAttnWaves * 64), 0, st, a, plan,
                       static_cast<uint32_t>(front));
    return;
  }
  if (a.prefix_table) launch_cut<D, BITS, PAIR>(a, plan, 1, st);
  launch_cut<D, BITS, PAIR>(a, plan, 0, st);
}

template <int D>
void launch_head_dim(const AttentionArgs& a, const AttentionPlan& plan, bool pair, hipStream_t st) {
  if (a.bits == 4)
    pair ? launch_parts<D, 4, true>(a, plan, st) : launch_parts<D, 4, false>(a, plan, st);
  else
    pair ? launch_parts<D, 8, true>(a, plan, st) : launch_parts<D, 8, false>(a, plan, st);
}

}  // namespace

void launch_attention_64(const AttentionArgs& a, const AttentionPlan& plan, bool pair, hipStream_t st);
void launch_attention_128(const AttentionArgs& a, const AttentionPlan& plan, bool pair, hipStream_t st);
void launch_attention_256(const AttentionArgs& a, const AttentionPlan& plan, bool pair, hipStream_t st);

}  // namespace w4a4
