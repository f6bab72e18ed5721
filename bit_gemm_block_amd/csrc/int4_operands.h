// int4_operands.h — packed codes widened to matrix operands in registers.
//
// fp16: the bits of 1024 + u are 0x6400 | u, so a nibble (or byte) lands in the
// mantissa by a mask and an OR and one exact packed operation removes the
// offset.  Two's-complement codes are first made unsigned (u = q + 8 or + 128).
// bfloat16: the instruction that makes q / 16 of a nibble as float32, whose
// upper half holds it exactly.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

union Operand {
  uint32_t w[4];
  h2 p[4];
  h8 h;
  b8 b;
};

// Constants that stay in registers: with two literals the mask and what follows
// it would be two instructions.
struct Masks {
  uint32_t even = 0x000f000fu, odd = 0x00f000f0u;
  uint32_t key = 0x00800080u;
  uint32_t value_even = 0x64086408u, value_odd = 0x64806480u;
  __device__ __forceinline__ Masks() {
    asm("" : "+s"(even), "+s"(odd), "+v"(key), "+v"(value_even), "+v"(value_odd));
  }
};

// Nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word of codes as fp16: flipping
// the sign bit in the same instruction makes u = q + 8 of the code (a nibble
// higher up counts 16 times).
__device__ __forceinline__ void nibbles_to_f16(uint32_t w, const Masks& m, h2* even0, h2* odd0, h2* even1, h2* odd1) {
  const uint32_t s = w >> 8;
  const h2 off = {1032.f16, 1032.f16}, sixteenth = {0.0625f16, 0.0625f16}, off16 = {-72.f16, -72.f16};
  *even0 = __builtin_bit_cast(h2, (w & m.even) ^ m.value_even) - off;
  *odd0 = __builtin_elementwise_fma(__builtin_bit_cast(h2, (w & m.odd) ^ m.value_odd), sixteenth, off16);
  *even1 = __builtin_bit_cast(h2, (s & m.even) ^ m.value_even) - off;
  *odd1 = __builtin_elementwise_fma(__builtin_bit_cast(h2, (s & m.odd) ^ m.value_odd), sixteenth, off16);
}

// The eight codes of a word as fp16, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ Operand int4_to_f16(uint32_t w, const Masks& m) {
  Operand o;
  nibbles_to_f16(w, m, &o.p[0], &o.p[1], &o.p[2], &o.p[3]);
  return o;
}
// Eight fp16 values to that order.
__device__ __forceinline__ Operand order_04152637(u4 x) {
  Operand o;
  o.w[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
  o.w[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
  o.w[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
  o.w[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
  return o;
}

// The upper halves of two words.
__device__ __forceinline__ uint32_t upper(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}
__device__ __forceinline__ uint32_t bits_of(float v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ float float_of(uint32_t v) { return __builtin_bit_cast(float, v); }

// The eight codes of a word over 16 as bfloat16, in their order.
__device__ __forceinline__ Operand int4_to_bf16_over16(uint32_t w) {
  Operand o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.w[i] = upper(bits_of(__builtin_amdgcn_cvt_off_f32_i4(static_cast<int>(w >> (8 * i)))),
                   bits_of(__builtin_amdgcn_cvt_off_f32_i4(static_cast<int>(w >> (8 * i + 4)))));
  return o;
}

// Eight float32 values as three bfloat16 parts that add up to them: eight bits
// of the significand each, cut off, so that every difference is exact.
__device__ __forceinline__ void split_bf16(const float* x, Operand* o) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int part = 0; part < 3; ++part) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[part].w[i] = upper(bits_of(r[2 * i]), bits_of(r[2 * i + 1]));
    if (part < 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] -= float_of(bits_of(r[i]) & 0xffff0000u);
    }
  }
}

}  // namespace
}  // namespace w4a4
