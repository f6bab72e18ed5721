// vec_io.h — eight consecutive elements of a row as float32, for the streaming
// kernels beside the layer.
//
// Rows need only their element's alignment: the vector types below claim no
// more, and the hardware takes 16-byte accesses at any element's address (a
// wave's run of 1 KB then touches one more cache line).
//
// Activations pass once: they are stored (and, where nothing else reads them,
// loaded) past the caches' retention, which keeps what is shared in them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {
namespace {

typedef float vf4 __attribute__((ext_vector_type(4)));
typedef vf4 vf4u __attribute__((aligned(4)));
typedef _Float16 vh8 __attribute__((ext_vector_type(8)));
typedef vh8 vh8u __attribute__((aligned(2)));

// Eight raw elements: 32 bytes of float32 or 16 of fp16.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  vf4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const vf4u*>(p)[0];
    b = reinterpret_cast<const vf4u*>(p)[1];
  }
  __device__ __forceinline__ void load_once(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const vf4u*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const vf4u*>(p) + 1);
  }
  __device__ __forceinline__ void set(int e, float v) {
    if (e < 4) a[e & 3] = v;
    else b[e & 3] = v;
  }
  __device__ __forceinline__ float get(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
};
template <>
struct Raw8<_Float16> {
  vh8 a;
  __device__ __forceinline__ void load(const _Float16* p) { a = *reinterpret_cast<const vh8u*>(p); }
  __device__ __forceinline__ void load_once(const _Float16* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const vh8u*>(p));
  }
  __device__ __forceinline__ void set(int e, _Float16 v) { a[e] = v; }
  __device__ __forceinline__ float get(int e) const { return static_cast<float>(a[e]); }
};

// Elements [c, c + 8) of a row of C that is read once; those past its end are
// zero.
template <typename T, typename I>
__device__ __forceinline__ Raw8<T> load8_once(const T* row, I c, I C) {
  Raw8<T> r;
  if (c + 8 <= C) {
    r.load_once(row + c);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.set(e, c + e < C ? row[c + e] : static_cast<T>(0.f));
  }
  return r;
}

__device__ __forceinline__ void store_whole8(float* p, const float* v) {
  __builtin_nontemporal_store(vf4u{v[0], v[1], v[2], v[3]}, reinterpret_cast<vf4u*>(p));
  __builtin_nontemporal_store(vf4u{v[4], v[5], v[6], v[7]}, reinterpret_cast<vf4u*>(p) + 1);
}
__device__ __forceinline__ void store_whole8(_Float16* p, const float* v) {
  vh8 h;
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = static_cast<_Float16>(v[e]);  // nearest, ties to even
  __builtin_nontemporal_store(static_cast<vh8u>(h), reinterpret_cast<vh8u*>(p));
}

// The same elements of a row, those past its end left alone.
template <typename T, typename I>
__device__ __forceinline__ void store8(T* row, I c, I C, const float* v) {
  if (c + 8 <= C) {
    store_whole8(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) row[c + e] = static_cast<T>(v[e]);
  }
}

}  // namespace
}  // namespace w4a4
