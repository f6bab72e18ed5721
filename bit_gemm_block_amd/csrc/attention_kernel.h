// attention_kernel.h — softmax(c q . k) v of 16-row tiles over the quantized
// cache, one pass over the tokens.
//
// A wave takes 16 R rows (a row: a query of one head of the group that shares
// the cache head) through steps of 32 tokens:
//
//   S^T = K Q^T   16 tokens x 16 rows an instruction; lane (row r, g) gets
//                 tokens 4 g + i of both halves of the step;
//   p = 2^(t - ref), t = c s_k S;   w = p s_v;
//   O^T += V^T W^T with the 32 tokens as the inner dimension, in the order in
//                 which the lanes hold them: nothing moves between lanes.
//
// Codes meet the matrix instruction as exact fp16 numbers, widened in
// registers as they come from memory: K's words hold eight channels of one
// token, V's of two tokens are paired by halves first.  A float32 query is a
// pair hi + lo of fp16 under a power of two of its row, and w is such a pair,
// so that only the queries' and the probabilities' low 2^-20 are lost.
//
// ref stands in for the running maximum: any reference gives the same
// quotient, and this one moves only when a weight w leaves 2^14 (fp16 ends at
// 2^16) or a sum of p leaves 2^60.  It then becomes the maximum of t + log2 s_v
// (s_v no less than 2^-60), minus 8, over the tokens seen.  The usual step
// exchanges nothing between lanes and rescales nothing.
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

// Parts in use of a range of L tokens.
__host__ __device__ inline int parts_of(int64_t L, int parts, int least) {
  const uint32_t p = (static_cast<uint32_t>(L) + least - 1) / static_cast<uint32_t>(least);  // L below 2^30 + 1
  return static_cast<int>(p < 1 ? 1 : p < static_cast<uint32_t>(parts) ? p : parts);
}

// What a sequence (own tokens) or the prefix is to its queries.
struct Span {
  const int32_t* table;
  int64_t width;
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
  p.table = a.tables + s * a.width;
  p.width = a.width;
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
  p.rows = (p.n < a.max_q ? p.n : a.max_q) * a.group;
  return p;
}

__device__ __forceinline__ Span front_span(const AttentionArgs& a) {
  Span p;
  p.table = a.prefix_table;
  p.width = a.prefix_width;
  p.length = clamp_length(a.prefix_length[0], a.prefix_width << a.page_log2);
  int q1 = a.seqs;
  if (a.q_start) {
    q1 = a.q_start[a.seqs];
    q1 = q1 < 0 ? 0 : q1 < a.tokens ? q1 : a.tokens;
  }
  p.first = 0;
  p.n = q1;
  p.rows = q1 * a.group;
  return p;
}

// Bytes E and F of w (unsigned codes u = q + 128) as fp16, minus 128.
template <int SEL>
__device__ __forceinline__ h2 two_bytes(uint32_t w1, uint32_t w0) {
  union {
    uint32_t u;
    h2 h;
  } v;
  v.u = __builtin_amdgcn_perm(w1, w0, SEL) | 0x64006400u;
  return v.h - h2{1152.f16, 1152.f16};
}

// Constants that stay in registers: with two literals the mask and the sign's
// flip below would be two instructions.
struct Masks {
  uint32_t even = 0x000f000fu, odd = 0x00f000f0u;
  uint32_t key_even = 0x00080008u, key_odd = 0x00800080u;
  uint32_t value_even = 0x64086408u, value_odd = 0x64806480u;
  __device__ __forceinline__ Masks() {
    asm("" : "+s"(even), "+s"(odd), "+v"(key_even), "+v"(key_odd), "+v"(value_even), "+v"(value_odd));
  }
};

// The codes and scales of a step's keys or values, tokens 4 g + i of both halves
// for the scales and the values, token r for the keys.
template <int D, int BITS>
struct StepKeys {
  static constexpr int RB = D * BITS / 8;  // bytes of a row
  static constexpr int KW = RB / 16;       // words of its token's row a lane holds
  uint32_t k[2][KW];
  f4 s[2];
  __device__ __forceinline__ void load(const AttentionArgs& a, const int64_t* rb, uint32_t r, uint32_t g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* p = a.k + rb[h] * RB + (r * RB + g * (RB / 4));
      if constexpr (KW == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        k[h][0] = w.x;
        k[h][1] = w.y;
      } else {
#pragma unroll
        for (int i = 0; i < KW; i += 4) {
          const u4 w = *reinterpret_cast<const u4*>(p + 4 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) k[h][i + e] = w[e];
        }
      }
      s[h] = *reinterpret_cast<const f4*>(a.ks + rb[h] + 4 * g);
    }
  }
};

template <int D, int BITS>
struct StepValues {
  static constexpr int RB = D * BITS / 8;
  static constexpr int VW = RB >= 64 ? RB / 64 : 1;  // words of each of its tokens a lane holds
  uint32_t v[8][VW];
  f4 s[2];
  __device__ __forceinline__ void load(const AttentionArgs& a, const int64_t* rb, uint32_t r, uint32_t g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h] = *reinterpret_cast<const f4*>(a.vs + rb[h] + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = a.v + rb[h] * RB + (g * (4 * RB) + r * (RB / 16)) + i * RB;
        uint32_t* d = v[4 * h + i];
        if constexpr (RB == 32) {
          d[0] = *reinterpret_cast<const uint16_t*>(p);
        } else if constexpr (VW == 1) {
          d[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (VW == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(p);
          d[0] = w.x;
          d[1] = w.y;
        } else {
          const u4 w = *reinterpret_cast<const u4*>(p);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = w[e];
        }
      }
    }
  }
};

// K's codes 8 j to 8 j + 7 of a lane, unsigned, as fp16 subnormal numbers u 2^-24
// (the bits of a small whole number are that times 2^-24): in the order
// 0 4 1 5 2 6 3 7, the third, fourth, seventh and eighth times 16 (4 bits), or
// in their own (8 bits).  Their offset, 8 or 128, is taken out of the product
// by its starting value.
template <int BITS>
__device__ __forceinline__ h8 key_operand(const uint32_t* k, int j, const Masks& m) {
  Operand o;
  if constexpr (BITS == 4) {
    const uint32_t s = k[j] >> 8;
    o.w[0] = (k[j] & m.even) ^ m.key_even;
    o.w[1] = (k[j] & m.odd) ^ m.key_odd;
    o.w[2] = (s & m.even) ^ m.key_even;
    o.w[3] = (s & m.odd) ^ m.key_odd;
  } else {
    const uint32_t a = k[2 * j] ^ 0x80808080u, b = k[2 * j + 1] ^ 0x80808080u;
    o.w[0] = __builtin_amdgcn_perm(a, a, 0x0c010c00);
    o.w[1] = __builtin_amdgcn_perm(a, a, 0x0c030c02);
    o.w[2] = __builtin_amdgcn_perm(b, b, 0x0c010c00);
    o.w[3] = __builtin_amdgcn_perm(b, b, 0x0c030c02);
  }
  return o.h;
}
// The channel of the element e of such an operand, and log2 of its factor.
template <int BITS>
__device__ constexpr int key_channel(int e) {
  return BITS == 4 ? (e & 1) * 4 + e / 2 : e;
}
template <int BITS>
__device__ constexpr int key_factor(int e) {
  return BITS == 4 && (e & 2) ? 4 : 0;
}

// Four channels of the eight tokens of a lane, as fp16: channels 4 q to 4 q + 3
// of the lane's own.  (An offset of the values cannot wait like the keys': it
// would be 8 times the sum of the weights, which the result is a small part of.)
template <int D, int BITS>
__device__ __forceinline__ void value_operands(const StepValues<D, BITS>& s, int q, const Masks& m, Operand* o) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (BITS == 4) {
      const uint32_t t =
          __builtin_amdgcn_perm(s.v[2 * p + 1][q / 2], s.v[2 * p][q / 2], q % 2 ? 0x07060302u : 0x05040100u);
      const uint32_t u = t >> 8;
      o[0].w[p] = (t & m.even) ^ m.value_even;
      o[1].w[p] = (t & m.odd) ^ m.value_odd;
      o[2].w[p] = (u & m.even) ^ m.value_even;
      o[3].w[p] = (u & m.odd) ^ m.value_odd;
      const h2 off = {1032.f16, 1032.f16}, sixteenth = {0.0625f16, 0.0625f16}, off16 = {-72.f16, -72.f16};
      o[0].p[p] -= off;
      o[1].p[p] = __builtin_elementwise_fma(o[1].p[p], sixteenth, off16);
      o[2].p[p] -= off;
      o[3].p[p] = __builtin_elementwise_fma(o[3].p[p], sixteenth, off16);
    } else {
      const uint32_t w0 = s.v[2 * p][q] ^ 0x80808080u, w1 = s.v[2 * p + 1][q] ^ 0x80808080u;
      o[0].p[p] = two_bytes<0x0c040c00>(w1, w0);
      o[1].p[p] = two_bytes<0x0c050c01>(w1, w0);
      o[2].p[p] = two_bytes<0x0c060c02>(w1, w0);
      o[3].p[p] = two_bytes<0x0c070c03>(w1, w0);
    }
  }
}

// log2 of a scale, down to the integer, between 2^-60 and 2^127.
__device__ __forceinline__ float exponent(float v) {
  const int e = __builtin_amdgcn_frexp_expf(v);
  return v > 8.6736174e-19f ? static_cast<float>(e) : -60.f;
}

template <int D, int BITS, bool PAIR, int R, bool ROWS>
__global__ void __launch_bounds__(kAttnWaves * 64, D == 256 || R > 1 ? 2 : 3)
    attention_kernel(AttentionArgs a, AttentionCut cut, int front, int slot0, int slots) {
  constexpr int NK = D / 32;   // instructions along a head's channels
  constexpr int NV = D / 16;   // channels of O a lane's row block holds
  constexpr int HALVES = PAIR ? 2 : 1;
  constexpr float kUnset = -1e30f;  // of a row that has seen nothing
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  uint32_t id = blockIdx.x;
  const int h = id % a.heads;
  id /= a.heads;
  const int part = id % cut.parts;
  id /= cut.parts;
  const int rg = static_cast<int>(cut.row_groups) - 1 - static_cast<int>(id % static_cast<uint32_t>(cut.row_groups));
  const int s = static_cast<int>(id / static_cast<uint32_t>(cut.row_groups));

  const Span span = front ? front_span(a) : own_span(a, s);
  constexpr int kRows = 16 * R;
  const int group_rows = ROWS ? kRows * kAttnWaves : kRows;
  if (static_cast<int64_t>(rg) * group_rows >= span.rows) return;
  const int eff = parts_of(span.length, cut.parts, cut.least);
  if (part >= eff) return;
  const int row0 = rg * group_rows + (ROWS ? wave * kRows : 0);

  // What the queries see: positions below the limit.
  const int length = static_cast<int>(span.length);
  auto limit_of = [&](int query) -> int {
    if (front || !a.causal) return length;
    const int l = length - span.n + query + 1;
    return l < 0 ? 0 : l;
  };
  auto query_of = [&](int row) { return static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(a.group)); };
  int limit[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int row = row0 + 16 * t + r;
    limit[t] = row < span.rows ? limit_of(query_of(row)) : 0;
  }
  const int last = (row0 + kRows < span.rows ? row0 + kRows : span.rows) - 1;  // of this wave
  const int group_last = static_cast<int>(least64(static_cast<int64_t>(rg + 1) * group_rows, span.rows)) - 1;
  const int wave_end = last >= row0 ? limit_of(last / a.group) : 0;
  const int all_see = row0 + kRows <= span.rows ? limit_of(row0 / a.group) : 0;  // positions every row sees
  const int share = static_cast<int>((static_cast<uint32_t>(limit_of(group_last / a.group) + kStep - 1) / kStep + eff - 1) /
                                     static_cast<uint32_t>(eff));  // steps to a part
  const int wave_steps = (wave_end + kStep - 1) / kStep;
  const int begin = part * share + (ROWS ? 0 : wave);
  const int end = (part + 1) * share < wave_steps ? (part + 1) * share : wave_steps;
  constexpr int kStride = ROWS ? 1 : kAttnWaves;

  // Pages come 64 at a time, lane 2 i + half holding that of the half of the
  // wave's step i (of 32): a step reads its two from the lanes, and no wait
  // for the table stands between a step and its loads.  -1: no such page.
  const int tile_end = static_cast<int>(span.width << a.page_log2);
  auto pages_from = [&](int step) -> int32_t {
    int tok = (step + (lane >> 1) * kStride) * kStep + 16 * (lane & 1);
    tok = tok < tile_end && tok >= 0 ? tok : tile_end - 16;
    const int32_t p = span.table[tok >> a.page_log2];
    return p >= 0 && p < a.pages ? p : -1;
  };
  int64_t rb[2];  // cache rows of a step's halves
  auto rows_of = [&](int step, int32_t p0, int32_t p1) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int off = (step * kStep + 16 * half) & ((1 << a.page_log2) - 1);
      const int32_t p = half ? p1 : p0;
      rb[half] = ((static_cast<int64_t>(p < 0 ? 0 : p) * a.heads + h) << a.page_log2) + off;
    }
  };
  StepKeys<D, BITS> keys;
  StepValues<D, BITS> values;
  int32_t pages = 0;
  int32_t p0 = 0, p1 = 0;  // of the step whose keys are loaded
  if (begin < end) {
    pages = pages_from(begin);
    p0 = __builtin_amdgcn_readlane(pages, 0);
    p1 = __builtin_amdgcn_readlane(pages, 1);
    rows_of(begin, p0, p1);
    keys.load(a, rb, r, g);
    values.load(a, rb, r, g);
  }

  // The queries in the codes' order, under a power of two of the row, go to LDS
  // as operands, and what makes scores (over log 2) of the products to c.  Waves
  // that share their rows share the work.
  constexpr int kOwners = ROWS ? kAttnWaves : 1;
  __shared__ u4 queries[kOwners][R][NK][HALVES][64];
  auto& mine = queries[ROWS ? wave : 0];
  float c[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const bool have = row0 + 16 * t + r < span.rows;
    const int row = have ? row0 + 16 * t + r : 0;
    const int64_t at = static_cast<int64_t>(span.first + query_of(row)) * a.ldq +
                       static_cast<int64_t>(h * a.group + row - query_of(row) * a.group) * D + g * (D / 4);
    using Q = std::conditional_t<PAIR, float, _Float16>;
    Raw8<Q> x[NK];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      x[j].load(static_cast<const Q*>(a.q) + at + 8 * j);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[j].get(e)));
    }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const int up = m > 0.f && m < INFINITY ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;  // the row's largest below 2^14
    c[t] = ldexpf(a.scale * 1.4426950408889634f, 24 - up);
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      if (!ROWS && j % kAttnWaves != wave) continue;
      Operand hi, lo;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float v0 = ldexpf(x[j].get(key_channel<BITS>(e)), up - key_factor<BITS>(e));
        const float v1 = ldexpf(x[j].get(key_channel<BITS>(e + 1)), up - key_factor<BITS>(e + 1));
        hi.p[e / 2] = h2{static_cast<_Float16>(v0), static_cast<_Float16>(v1)};
        lo.p[e / 2] = h2{static_cast<_Float16>(fmaf(static_cast<float>(hi.p[e / 2][0]), -1.f, v0)),
                         static_cast<_Float16>(fmaf(static_cast<float>(hi.p[e / 2][1]), -1.f, v1))};
      }
      mine[t][j][0][lane] = u4{hi.w[0], hi.w[1], hi.w[2], hi.w[3]};
      if constexpr (PAIR) mine[t][j][1][lane] = u4{lo.w[0], lo.w[1], lo.w[2], lo.w[3]};
    }
  }
  if constexpr (!ROWS) __syncthreads();
  auto query_operand = [&](int t, int j, int p) { return __builtin_bit_cast(h8, mine[t][j][p][lane]); };
  // The products start from what the codes' offset adds to them, taken off.
  f4 start[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    f4 sum = {0.f, 0.f, 0.f, 0.f};
    Operand offset;
#pragma unroll
    for (int p = 0; p < 4; ++p) offset.w[p] = BITS == 8 || p % 2 ? 0x00800080u : 0x00080008u;
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
      for (int p = HALVES - 1; p >= 0; --p)
        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(offset.h, query_operand(t, j, p), sum, 0, 0, 0);
    start[t] = -sum;
  }

  f4 o[R][NV];
  float ref[R], l[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    ref[t] = kUnset;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) o[t][j] = f4{0.f, 0.f, 0.f, 0.f};
  }
  const Masks masks;

  int turn = 0;  // steps into the 32 whose pages are at hand
  // A step; all but the last bring the next one's keys in while the softmax and
  // the second product run, and its values at the end.  (A condition around the
  // loads would make every wait one for all of them.)
  auto take = [&](int step, auto last_step) {
    constexpr bool LAST = decltype(last_step)::value;
    const int tok0 = step * kStep;
    const bool bad0 = p0 < 0, bad1 = p1 < 0;
    const bool partly = bad0 || bad1 || tok0 + kStep > all_see;  // some row does not see some token

    asm volatile("" ::: "memory");  // the queries are read again, not kept in registers
    f4 sc[R][2];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      h8 k[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) k[half] = key_operand<BITS>(keys.k[half], j, masks);
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int p = HALVES - 1; p >= 0; --p) {
          const h8 q = query_operand(t, j, p);
#pragma unroll
          for (int half = 0; half < 2; ++half)
            sc[t][half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                k[half], q, j == 0 && p == HALVES - 1 ? start[t] : sc[t][half], 0, 0, 0);
        }
    }
    float kc[R][8];
#pragma unroll
    for (int t = 0; t < R; ++t)
#pragma unroll
      for (int i = 0; i < 8; ++i) kc[t][i] = keys.s[i / 4][i % 4] * c[t];
    if constexpr (!LAST) {
      if (++turn == 32) {
        pages = pages_from(step + kStride);
        turn = 0;
      }
      p0 = __builtin_amdgcn_readlane(pages, 2 * turn);
      p1 = __builtin_amdgcn_readlane(pages, 2 * turn + 1);
      rows_of(step + kStride, p0, p1);
      keys.load(a, rb, r, g);
    }

    Operand w[R][2];  // hi, lo
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float x[8], vs[8], wt[8], sum, top;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = sc[t][i / 4][i % 4];
        vs[i] = values.s[i / 4][i % 4];
      }
      if (partly) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = tok0 + 16 * (i / 4) + 4 * g + i % 4;
          if (tok >= limit[t] || (i < 4 ? bad0 : bad1)) {  // whatever the scales there are
            x[i] = -INFINITY;
            kc[t][i] = 1.f;
            vs[i] = 0.f;
          }
        }
      }
      auto weigh = [&]() {
        sum = 0.f;
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __builtin_amdgcn_exp2f(fmaf(x[i], kc[t][i], -ref[t]));
          wt[i] = p * vs[i];
          sum += p;
          top = fmaxf(top, wt[i]);
        }
      };
      weigh();
      if (__any(top > 16384.f || sum > 1.15292150e18f)) {
        float u = kUnset;
#pragma unroll
        for (int i = 0; i < 8; ++i) u = fmaxf(u, fmaf(x[i], kc[t][i], exponent(vs[i])));
        u = fmaxf(u, __shfl_xor(u, 16));
        u = fmaxf(u, __shfl_xor(u, 32));
        const float moved = fmaxf(ref[t], u - 8.f);
        const float f = __builtin_amdgcn_exp2f(ref[t] - moved);
        ref[t] = moved;
        l[t] *= f;
#pragma unroll
        for (int j = 0; j < NV; ++j) o[t][j] *= f;
        weigh();
      }
      l[t] += sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto hi = __builtin_amdgcn_cvt_pkrtz(wt[2 * i], wt[2 * i + 1]);
        const auto lo = __builtin_amdgcn_cvt_pkrtz(fmaf(static_cast<float>(hi[0]), -1.f, wt[2 * i]),
                                                   fmaf(static_cast<float>(hi[1]), -1.f, wt[2 * i + 1]));
        w[t][0].w[i] = __builtin_bit_cast(uint32_t, hi);
        w[t][1].w[i] = __builtin_bit_cast(uint32_t, lo);
      }
    }

#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      Operand v[4];
      value_operands<D, BITS>(values, j, masks, v);
#pragma unroll
      for (int p = 1; p >= 0; --p)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int t = 0; t < R; ++t)
            o[t][4 * j + e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[e].h, w[t][p].h, o[t][4 * j + e], 0, 0, 0);
    }
    if constexpr (!LAST) values.load(a, rb, r, g);
  };
  if (begin < end) {
    int step = begin;
    for (; step + kStride < end; step += kStride) take(step, std::false_type{});
    take(step, std::true_type{});
  }

#pragma unroll
  for (int t = 0; t < R; ++t) {
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
  }

  // The waves' shares of the same rows: brought to one reference, added up in
  // wave 0, in the order (0 + 2) + (1 + 3).
  if constexpr (!ROWS) {
    __shared__ float stat[kAttnWaves][R][16][2];
    __shared__ f4 lds[2][R * NV][64];
    if (g == 0) {
#pragma unroll
      for (int t = 0; t < R; ++t) {
        stat[wave][t][r][0] = ref[t];
        stat[wave][t][r][1] = l[t];
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float top = kUnset;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) top = fmaxf(top, stat[k][t][r][0]);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) {
        sum += __builtin_amdgcn_exp2f(stat[k][t][r][0] - top) * stat[k][t][r][1];
      }
      const float f = __builtin_amdgcn_exp2f(ref[t] - top);
#pragma unroll
      for (int j = 0; j < NV; ++j) o[t][j] *= f;
      ref[t] = top;
      l[t] = sum;
    }
#pragma unroll
    for (int far = 2; far >= 1; far >>= 1) {
      if (wave >= far && wave < 2 * far) {
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int j = 0; j < NV; ++j) lds[wave - far][t * NV + j][lane] = o[t][j];
      }
      __syncthreads();
      if (wave < far) {
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int j = 0; j < NV; ++j) o[t][j] += lds[wave][t * NV + j][lane];
      }
      __syncthreads();
    }
    if (wave != 0) return;
  }

  // Lane (r, g) holds channels [g D / 4, +D / 4) of its row: NV i + j is o[j][i].
  const bool whole = eff == 1 && !front && !a.prefix_table;
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int row = row0 + 16 * t + r;
    if (row >= span.rows) continue;
    const int64_t token = span.first + query_of(row);
    const int head = h * a.group + row - query_of(row) * a.group;
    if (whole) {
      const float f = l[t] == 0.f ? 0.f : 1.f / l[t];
      const int64_t at = token * a.ldo + static_cast<int64_t>(head) * D + g * (D / 4);
#pragma unroll
      for (int e = 0; e < D / 4; e += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = o[t][(e + k) % NV][(e + k) / NV] * f;
        if (a.out_f16)
          store_whole8(static_cast<_Float16*>(a.out) + at + e, v);
        else
          store_whole8(static_cast<float*>(a.out) + at + e, v);
      }
    } else {
      const int64_t at = (static_cast<int64_t>(slot0 + part) * a.tokens + token) * a.q_heads + head;
      float* po = a.partial + at * D + g * (D / 4);
#pragma unroll
      for (int e = 0; e < D / 4; e += 4)
        *reinterpret_cast<f4*>(po + e) = f4{o[t][e % NV][e / NV], o[t][(e + 1) % NV][(e + 1) / NV],
                                            o[t][(e + 2) % NV][(e + 2) / NV], o[t][(e + 3) % NV][(e + 3) / NV]};
      if (g == 0) {
        float* st = a.partial + static_cast<int64_t>(slots) * a.tokens * a.q_heads * D + at * 2;
        st[0] = ref[t];
        st[1] = l[t];
      }
    }
  }
}

template <int D, int BITS, bool PAIR>
void launch_cut(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, hipStream_t st) {
  const int64_t seqs = front ? 1 : a.seqs;
  const dim3 grid(static_cast<unsigned>(seqs * c.row_groups * c.parts * a.heads)), block(kAttnWaves * 64);
  if (c.rowsplit) {
    if constexpr (D < 256) {
      if (c.tiles == 2) {
        hipLaunchKernelGGL((attention_kernel<D, BITS, PAIR, 2, true>), grid, block, 0, st, a, c, front, slot0, slots);
        return;
      }
    }
    hipLaunchKernelGGL((attention_kernel<D, BITS, PAIR, 1, true>), grid, block, 0, st, a, c, front, slot0, slots);
  } else {
    if constexpr (D < 256) {
      if (c.tiles == 2) {
        hipLaunchKernelGGL((attention_kernel<D, BITS, PAIR, 2, false>), grid, block, 0, st, a, c, front, slot0, slots);
        return;
      }
    }
    hipLaunchKernelGGL((attention_kernel<D, BITS, PAIR, 1, false>), grid, block, 0, st, a, c, front, slot0, slots);
  }
}

template <int D>
void launch_head_dim(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                     hipStream_t st) {
  if (a.bits == 4)
    pair ? launch_cut<D, 4, true>(a, c, front, slot0, slots, st) : launch_cut<D, 4, false>(a, c, front, slot0, slots, st);
  else
    pair ? launch_cut<D, 8, true>(a, c, front, slot0, slots, st) : launch_cut<D, 8, false>(a, c, front, slot0, slots, st);
}

}  // namespace

void launch_attention_64(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                         hipStream_t st);
void launch_attention_128(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                          hipStream_t st);
void launch_attention_256(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                          hipStream_t st);

}  // namespace w4a4
