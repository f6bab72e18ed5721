// cache.hip — keys and values quantized as they are written into a paged cache,
// and read back.
//
//   write: s = max|x| / qmax, q = clamp(rint(x / s), -qmax, qmax) per token and
//   head (IEEE float32 division, ties to even);  read: x = q s.
//
// A token's head is a row of D elements, eight to a lane: 8, 16 or 32 lanes
// meet for the maximum and write the row's codes in one run.  Keys and values
// are the two halves of one grid.
#include "decode_internal.h"
#include "vec_io.h"

namespace w4a4 {
namespace {

// The 64-bit index of the row of (slot, head): page-major, then heads, then
// the page's tokens.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& a, int32_t slot, int head) {
  const int64_t page = slot >> a.page_log2;
  const int off = slot & ((1 << a.page_log2) - 1);
  return ((page * a.heads + head) << a.page_log2) + off;
}

template <int LANES, int BITS, typename T>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheArgs a) {
  const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / LANES;  // the grid has fewer than 2^32 threads
  const int lane = threadIdx.x % LANES;
  const int64_t t = row / static_cast<uint32_t>(a.heads);
  if (t >= a.T) return;  // whole rows: lanes that meet below leave together
  const int head = static_cast<int>(row - static_cast<uint32_t>(t) * a.heads);
  const int32_t slot = a.slots[t];
  if (slot < 0 || slot >= a.slots_end) return;
  const int side = blockIdx.y;
  Raw8<T> r;
  r.load_once(static_cast<const T*>(a.x[side]) + t * a.ld[side] + static_cast<int64_t>(head) * (LANES * 8) +
              lane * 8);
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(r.get(e)));
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  constexpr float kMax = BITS == 4 ? 7.f : 127.f;
  const float s = m / kMax;
  uint32_t w[2] = {0, 0};
  if (s > 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = fminf(fmaxf(rintf(r.get(e) / s), -kMax), kMax);
      const uint32_t c = static_cast<uint32_t>(static_cast<int>(q));
      if constexpr (BITS == 4)
        w[0] |= (c & 15u) << (4 * e);
      else
        w[e / 4] |= (c & 255u) << (8 * (e % 4));
    }
  }
  const int64_t at = cache_row(a, slot, head);
  uint8_t* dst = a.codes[side] + at * (LANES * BITS) + lane * BITS;
  if constexpr (BITS == 4)
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  if (lane == 0) a.scale[side][at] = s;
}

template <int LANES, int BITS, typename T>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheArgs a) {
  const uint32_t row = (blockIdx.x * 256u + threadIdx.x) / LANES;  // the grid has fewer than 2^32 threads
  const int lane = threadIdx.x % LANES;
  const int64_t t = row / static_cast<uint32_t>(a.heads);
  const int side = blockIdx.y;
  if (t >= a.T || !a.x[side]) return;
  const int head = static_cast<int>(row - static_cast<uint32_t>(t) * a.heads);
  const int32_t slot = a.slots[t];
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && slot < a.slots_end) {
    const int64_t at = cache_row(a, slot, head);
    const uint8_t* src = a.codes[side] + at * (LANES * BITS) + lane * BITS;
    const float s = a.scale[side][at];
    if constexpr (BITS == 4) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(static_cast<int32_t>(w << (28 - 4 * e)) >> 28) * s;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(src);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = static_cast<float>(static_cast<int32_t>((e < 4 ? w.x : w.y) << (24 - 8 * (e % 4))) >> 24) * s;
    }
  }
  store_whole8(static_cast<T*>(a.x[side]) + t * a.ld[side] + static_cast<int64_t>(head) * (LANES * 8) + lane * 8,
               v);
}

template <bool WRITE, int LANES, int BITS, typename T>
void launch_rows(const CacheArgs& a, hipStream_t st) {
  const int64_t groups = (a.T * a.heads * LANES + 255) / 256;
  const dim3 grid(static_cast<unsigned>(groups), 2);
  if constexpr (WRITE)
    hipLaunchKernelGGL((cache_write_kernel<LANES, BITS, T>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((cache_read_kernel<LANES, BITS, T>), grid, dim3(256), 0, st, a);
}

template <bool WRITE, typename T>
hipError_t launch_cache(const CacheArgs& a, hipStream_t st) {
  if (a.bits == 4)
    a.D == 64 ? launch_rows<WRITE, 8, 4, T>(a, st)
              : a.D == 128 ? launch_rows<WRITE, 16, 4, T>(a, st) : launch_rows<WRITE, 32, 4, T>(a, st);
  else
    a.D == 64 ? launch_rows<WRITE, 8, 8, T>(a, st)
              : a.D == 128 ? launch_rows<WRITE, 16, 8, T>(a, st) : launch_rows<WRITE, 32, 8, T>(a, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs& a, bool f16, hipStream_t st) {
  return f16 ? launch_cache<true, _Float16>(a, st) : launch_cache<true, float>(a, st);
}
hipError_t launch_cache_read(const CacheArgs& a, bool f16, hipStream_t st) {
  return f16 ? launch_cache<false, _Float16>(a, st) : launch_cache<false, float>(a, st);
}

}  // namespace w4a4
