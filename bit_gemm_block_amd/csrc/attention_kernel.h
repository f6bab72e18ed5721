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
  const int64_t p = (L + least - 1) / least;
  return static_cast<int>(p < 1 ? 1 : p < parts ? p : parts);
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

// Codes and scales of a step: tokens 4 g + i of halves a and b.
template <int D, int BITS>
struct StepData {
  static constexpr int RB = D * BITS / 8;  // bytes of a row
  static constexpr int KW = RB / 16;       // words of K a lane holds of its token
  static constexpr int VW = RB >= 64 ? RB / 64 : 1;
  uint32_t k[2][KW];
  uint32_t v[8][VW];
  f4 ks[2], vs[2];

  // rb: the cache rows of the two halves' first tokens.
  __device__ __forceinline__ void load(const AttentionArgs& a, const int64_t* rb, int r, int g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* kp = a.k + (rb[h] + r) * RB + g * (RB / 4);
      if constexpr (KW == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(kp);
        k[h][0] = w.x;
        k[h][1] = w.y;
      } else {
#pragma unroll
        for (int i = 0; i < KW; i += 4) {
          const u4 w = *reinterpret_cast<const u4*>(kp + 4 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) k[h][i + e] = w[e];
        }
      }
      ks[h] = *reinterpret_cast<const f4*>(a.ks + rb[h] + 4 * g);
      vs[h] = *reinterpret_cast<const f4*>(a.vs + rb[h] + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* vp = a.v + (rb[h] + 4 * g + i) * RB + r * (RB / 16);
        uint32_t* d = v[4 * h + i];
        if constexpr (RB == 32) {
          d[0] = *reinterpret_cast<const uint16_t*>(vp);
        } else if constexpr (VW == 1) {
          d[0] = *reinterpret_cast<const uint32_t*>(vp);
        } else if constexpr (VW == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(vp);
          d[0] = w.x;
          d[1] = w.y;
        } else {
          const u4 w = *reinterpret_cast<const u4*>(vp);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = w[e];
        }
      }
    }
  }
};

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

// K's codes 8 j to 8 j + 7 of a lane: in the order 0 4 1 5 2 6 3 7 (4 bits) or
// their own (8 bits).
template <int BITS>
__device__ __forceinline__ h8 key_operand(const uint32_t* k, int j) {
  if constexpr (BITS == 4) {
    return int4_to_f16(k[j]).h;
  } else {
    const uint32_t a = k[2 * j] ^ 0x80808080u, b = k[2 * j + 1] ^ 0x80808080u;
    Operand o;
    o.p[0] = two_bytes<0x0c010c00>(a, a);
    o.p[1] = two_bytes<0x0c030c02>(a, a);
    o.p[2] = two_bytes<0x0c010c00>(b, b);
    o.p[3] = two_bytes<0x0c030c02>(b, b);
    return o.h;
  }
}

// Four channels of the eight tokens of a lane: channels 4 q to 4 q + 3 of the
// lane's own.
template <int D, int BITS>
__device__ __forceinline__ void value_operands(const StepData<D, BITS>& s, int q, Operand* o) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (BITS == 4) {
      const uint32_t w0 = s.v[2 * p][q / 2] ^ 0x88888888u, w1 = s.v[2 * p + 1][q / 2] ^ 0x88888888u;
      const uint32_t t = __builtin_amdgcn_perm(w1, w0, q % 2 ? 0x07060302u : 0x05040100u);
      o[0].p[p] = nibbles<false>(t);
      o[1].p[p] = nibbles<true>(t);
      o[2].p[p] = nibbles<false>(t >> 8);
      o[3].p[p] = nibbles<true>(t >> 8);
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
__global__ void __launch_bounds__(kAttnWaves * 64, 2)
    attention_kernel(AttentionArgs a, AttentionCut cut, int front, int slot0, int slots) {
  constexpr int NK = D / 32;   // instructions along a head's channels
  constexpr int NV = D / 16;   // channels of O a lane's row block holds
  constexpr int HALVES = PAIR ? 2 : 1;
  constexpr float kNone = -INFINITY;
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

  // What each row sees: positions below limit.
  auto limit_of = [&](int row) -> int64_t {
    if (front || !a.causal) return span.length;
    const int64_t l = span.length - span.n + row / a.group + 1;
    return l < 0 ? 0 : l;
  };
  int limit[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int row = row0 + 16 * t + r;
    limit[t] = row < span.rows ? static_cast<int>(limit_of(row)) : 0;
  }
  const int last = static_cast<int>(least64(row0 + kRows, span.rows)) - 1;       // of this wave
  const int group_last = static_cast<int>(least64(static_cast<int64_t>(rg + 1) * group_rows, span.rows)) - 1;
  const int wave_end = last >= row0 ? static_cast<int>(limit_of(last)) : 0;
  const int all_see = row0 + kRows <= span.rows ? static_cast<int>(limit_of(row0)) : 0;  // positions every row sees
  const int64_t steps = (limit_of(group_last) + kStep - 1) / kStep;
  const int begin = static_cast<int>(steps * part / eff) + (ROWS ? 0 : wave);
  const int end = static_cast<int>(least64(steps * (part + 1) / eff, (wave_end + kStep - 1) / kStep));
  constexpr int kStride = ROWS ? 1 : kAttnWaves;

  // The queries, in the codes' order, and each row's factor of the scores.
  Operand q[R][NK][HALVES];
  float c[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    const int row = row0 + 16 * t + r;
    const bool have = row < span.rows;
    const int64_t token = span.first + (have ? row / a.group : 0);
    const int64_t at = token * a.ldq + static_cast<int64_t>(h * a.group + (have ? row % a.group : 0)) * D + g * (D / 4);
    c[t] = a.scale * 1.4426950408889634f;
    if constexpr (PAIR) {
      Raw8<float> x[NK];
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        if (have) x[j].load(static_cast<const float*>(a.q) + at + 8 * j);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!have) x[j].set(e, 0.f);
          m = fmaxf(m, fabsf(x[j].get(e)));
        }
      }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const int up = m > 0.f && m < INFINITY ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;  // the row's largest below 2^14
      c[t] = ldexpf(c[t], -up);
#pragma unroll
      for (int j = 0; j < NK; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int from = BITS == 4 ? (e & 1) * 4 + e / 2 : e;
          const float v = ldexpf(x[j].get(from), up);
          const _Float16 hi = static_cast<_Float16>(v);
          q[t][j][0].h[e] = hi;
          q[t][j][1].h[e] = static_cast<_Float16>(v - static_cast<float>(hi));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        Raw8<_Float16> x;
        if (have) x.load(static_cast<const _Float16*>(a.q) + at + 8 * j);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          q[t][j][0].h[e] = have ? x.a[BITS == 4 ? (e & 1) * 4 + e / 2 : e] : static_cast<_Float16>(0.f);
      }
    }
  }

  f4 o[R][NV];
  float ref[R], l[R];
#pragma unroll
  for (int t = 0; t < R; ++t) {
    ref[t] = kNone;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) o[t][j] = f4{0.f, 0.f, 0.f, 0.f};
  }

  // Cache rows of a step's halves, and whether their pages exist.
  const int64_t tile_end = span.width << a.page_log2;
  auto page_of = [&](int step, int half) -> int32_t {
    int64_t tok = static_cast<int64_t>(step) * kStep + 16 * half;
    tok = tok < tile_end ? tok : tile_end - 16;
    return span.table[tok >> a.page_log2];
  };
  auto rows_of = [&](int step, const int32_t* page, int64_t* rb) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int off = (step * kStep + 16 * half) & ((1 << a.page_log2) - 1);
      const int32_t p = page[half] >= 0 && page[half] < a.pages ? page[half] : 0;
      rb[half] = ((static_cast<int64_t>(p) * a.heads + h) << a.page_log2) + off;
    }
  };

  StepData<D, BITS> next;
  int32_t page[2] = {0, 0};
  int64_t rb[2];
  if (begin < end) {
    page[0] = page_of(begin, 0);
    page[1] = page_of(begin, 1);
    rows_of(begin, page, rb);
    next.load(a, rb, r, g);
  }
  for (int step = begin; step < end; step += kStride) {
    const StepData<D, BITS> cur = next;
    const bool bad0 = page[0] < 0 || page[0] >= a.pages, bad1 = page[1] < 0 || page[1] >= a.pages;
    if (step + kStride < end) {
      page[0] = page_of(step + kStride, 0);
      page[1] = page_of(step + kStride, 1);
      rows_of(step + kStride, page, rb);
      next.load(a, rb, r, g);
    }
    const int tok0 = step * kStep;
    const bool partly = bad0 || bad1 || tok0 + kStep > all_see;  // some row does not see some token

    f4 sc[R][2];
#pragma unroll
    for (int t = 0; t < R; ++t) sc[t][0] = sc[t][1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NK; ++j) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const h8 k = key_operand<BITS>(cur.k[half], j);
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
          for (int p = HALVES - 1; p >= 0; --p)
            sc[t][half] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[t][j][p].h, sc[t][half], 0, 0, 0);
      }
    }

    Operand w[R][2];  // hi, lo
#pragma unroll
    for (int t = 0; t < R; ++t) {
      float x[8], p[8], wt[8], sum, top;
      uint32_t hidden = 0;
      auto weigh = [&]() {
        sum = 0.f;
        top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = __builtin_amdgcn_exp2f(x[i] - ref[t]);
          wt[i] = p[i] * cur.vs[i / 4][i % 4];
        }
        if (partly) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (hidden >> i & 1) p[i] = wt[i] = 0.f;  // whatever the scales there are
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum += p[i];
          top = fmaxf(top, wt[i]);
        }
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = sc[t][i / 4][i % 4] * (cur.ks[i / 4][i % 4] * c[t]);
      if (partly) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tok = tok0 + 16 * (i / 4) + 4 * g + i % 4;
          if (tok >= limit[t] || (i < 4 ? bad0 : bad1)) {
            x[i] = kNone;
            hidden |= 1u << i;
          }
        }
      }
      weigh();
      if (__any(top > 16384.f || sum > 1.15292150e18f)) {
        float u = kNone;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = x[i] + exponent(cur.vs[i / 4][i % 4]);
          u = fmaxf(u, x[i] == kNone ? kNone : y);
        }
        u = fmaxf(u, __shfl_xor(u, 16));
        u = fmaxf(u, __shfl_xor(u, 32));
        const float moved = fmaxf(ref[t], u - 8.f);
        const float f = moved == kNone ? 1.f : __builtin_amdgcn_exp2f(ref[t] - moved);
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
        const auto lo = __builtin_amdgcn_cvt_pkrtz(wt[2 * i] - static_cast<float>(hi[0]),
                                                   wt[2 * i + 1] - static_cast<float>(hi[1]));
        w[t][0].w[i] = __builtin_bit_cast(uint32_t, hi);
        w[t][1].w[i] = __builtin_bit_cast(uint32_t, lo);
      }
    }

#pragma unroll
    for (int j = 0; j < NV / 4; ++j) {
      Operand v[4];
      value_operands<D, BITS>(cur, j, v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int t = 0; t < R; ++t) {
          f4& d = o[t][4 * j + e];
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[e].h, w[t][1].h, d, 0, 0, 0);
          d = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[e].h, w[t][0].h, d, 0, 0, 0);
        }
    }
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
      float top = kNone;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) top = fmaxf(top, stat[k][t][r][0]);
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) {
        const float f = stat[k][t][r][0] == kNone ? 0.f : __builtin_amdgcn_exp2f(stat[k][t][r][0] - top);
        sum += f * stat[k][t][r][1];
      }
      const float f = ref[t] == kNone ? 0.f : __builtin_amdgcn_exp2f(ref[t] - top);
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
    const int64_t token = span.first + row / a.group;
    const int head = h * a.group + row % a.group;
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
