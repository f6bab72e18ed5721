// vec_io.h — eight consecutive (or strided) elements of a row as float32, for
// the streaming kernels beside the layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {
namespace {

typedef float vf4 __attribute__((ext_vector_type(4)));
typedef _Float16 vh8 __attribute__((ext_vector_type(8)));

// Eight raw elements of a row at p: 32 bytes of float32 or 16 of fp16.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  vf4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const vf4*>(p)[0];
    b = reinterpret_cast<const vf4*>(p)[1];
  }
  __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
};
template <>
struct Raw8<_Float16> {
  vh8 a;
  __device__ __forceinline__ void load(const _Float16* p) { a = *reinterpret_cast<const vh8*>(p); }
  __device__ __forceinline__ float get(int e) const { return static_cast<float>(a[e]); }
};

__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<vf4*>(p)[0] = vf4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<vf4*>(p)[1] = vf4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(_Float16* p, const float* v) {
  vh8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = static_cast<_Float16>(v[e]);  // nearest, ties to even
  *reinterpret_cast<vh8*>(p) = h;
}

}  // namespace

// Whether rows at p, ld elements of esize bytes apart, all start on 16 bytes.
inline bool rows_aligned16(const void* p, int64_t ld, int64_t esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && static_cast<uint64_t>(ld * esize) % 16 == 0;
}

}  // namespace w4a4
