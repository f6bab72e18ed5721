// gated.hip — out = act(gate) * up, elementwise between two projections.
//
//   silu       g / (1 + e^-g)
//   gelu       g Phi(g) = g / 2 erfc(-g / sqrt 2), which keeps the relative
//              precision of the left tail
//   gelu_tanh  g / 2 (1 + tanh u) = g / (1 + e^-2u),
//              u = sqrt(2/pi) (g + 0.044715 g^3)
//   relu       max(g, 0)
//
// In the left tails of the two gelus a rounding of the argument z is 2 z^2 (or
// |2u|) roundings of the result, so what the argument's rounding loses is
// carried to first order: erfc(z + d) = erfc(z) (1 - 2 z d) for z > 0 to
// within d / z, e^-(p + d) = e^-p (1 - d).
// Everything is float32 between one read and one rounding of the result (fp64 for
// the cubic argument of gelu_tanh alone).
//
// What bounds it: memory.  Every element is read and written once, eight to a
// thread, past the caches (4096 x 14336 silu, fp32 to fp16: 587 MB in 96 us, 6.1
// TB/s; 102.7 us with cached loads, 105 with cached stores as well).  Short calls
// are one launch (8 x 14336: 2.5 us).
#include "block_internal.h"
#include "vec_io.h"

#include "w4a4_block.h"

namespace w4a4 {
namespace {

// g / (1 + e^-(p + d)) for a small d, by the exponential that cannot overflow:
// the left tail runs down through the subnormal numbers.
__device__ __forceinline__ float times_sigmoid(float g, float p, float d) {
  const float e = expf(-fabsf(p)) * (1.f - (p < 0.f ? -d : d));
  return (p < 0.f ? g * e : g) / (1.f + e);
}

template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if constexpr (ACT == W4A4_ACT_SILU) {
    return times_sigmoid(g, g, 0.f);
  } else if constexpr (ACT == W4A4_ACT_GELU) {
    constexpr float kHi = 0.70710678118654752f;  // 1 / sqrt 2 as a float
    constexpr float kLo = static_cast<float>(0.70710678118654752440 - static_cast<double>(kHi));
    const float z = -kHi * g;
    float e = erfcf(z);
    if (z > 0.f && z < 16.f) e *= 1.f - 2.f * z * (fmaf(-kHi, g, -z) - kLo * g);
    return 0.5f * g * e;
  } else if constexpr (ACT == W4A4_ACT_GELU_TANH) {
    const double gd = static_cast<double>(g);
    const double p = 1.5957691216057308 * gd * (1.0 + 0.044715 * gd * gd);
    const float ph = static_cast<float>(p);
    const float pl = fabsf(ph) < 1000.f ? static_cast<float>(p - static_cast<double>(ph)) : 0.f;
    return times_sigmoid(g, ph, pl);
  } else {
    return g < 0.f ? 0.f : g;
  }
}

// act(g) u as a float32: the product is rounded before the conversion to fp16
// in every kernel below (not contracted with it in some of them), so that the
// result does not depend on the rows' alignment.
template <int ACT, bool UP>
__device__ __forceinline__ float gated(float g, float u) {
  float v = act_of<ACT>(g);
  if (UP) v *= u;
  asm volatile("" : "+v"(v));
  return v;
}

// One row (or the whole matrix as one row) per grid.y step, 8 * 256
// consecutive elements per workgroup.
template <typename I, typename O, int ACT, bool UP>
__global__ void __launch_bounds__(256) gated_kernel(GatedArgs a) {
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const I* gr = static_cast<const I*>(a.gate) + m * a.ldg;
    const I* ur = UP ? static_cast<const I*>(a.up) + m * a.ldu : nullptr;
    O* orow = static_cast<O*>(a.out) + m * a.ldo;
    for (int64_t c = blockIdx.x; c * 2048 < a.F; c += gridDim.x) {
      const int64_t f = c * 2048 + 8 * threadIdx.x;
      if (f >= a.F) continue;
      const Raw8<I> g = load8_once(gr, f, a.F);
      Raw8<I> u{};
      if (UP) u = load8_once(ur, f, a.F);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = gated<ACT, UP>(g.get(e), UP ? u.get(e) : 1.f);
      store8(orow, f, a.F, v);
    }
  }
}

template <typename I, typename O, int ACT>
void launch_act(const GatedArgs& a, hipStream_t st) {
  const int64_t chunks = (a.F + 2047) / 2048;
  const dim3 grid(static_cast<unsigned>(chunks < (1 << 20) ? chunks : (1 << 20)),
                  static_cast<unsigned>(a.M < 32768 ? a.M : 32768));
  if (a.up)
    hipLaunchKernelGGL((gated_kernel<I, O, ACT, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((gated_kernel<I, O, ACT, false>), grid, dim3(256), 0, st, a);
}

template <typename I, typename O>
void launch_types(const GatedArgs& a, int act, hipStream_t st) {
  switch (act) {
    case W4A4_ACT_SILU: return launch_act<I, O, W4A4_ACT_SILU>(a, st);
    case W4A4_ACT_GELU: return launch_act<I, O, W4A4_ACT_GELU>(a, st);
    case W4A4_ACT_GELU_TANH: return launch_act<I, O, W4A4_ACT_GELU_TANH>(a, st);
    default: return launch_act<I, O, W4A4_ACT_RELU>(a, st);
  }
}

}  // namespace

hipError_t launch_gated_activation(const GatedArgs& args, bool in_f16, bool out_f16, int act,
                                   hipStream_t st) {
  GatedArgs a = args;
  // Matrices without gaps between their rows are one long row.
  if (a.ldg == a.F && a.ldo == a.F && (!a.up || a.ldu == a.F)) {
    a.F *= a.M;
    a.M = 1;
  }
  if (in_f16) {
    if (out_f16) launch_types<_Float16, _Float16>(a, act, st);
    else launch_types<_Float16, float>(a, act, st);
  } else {
    if (out_f16) launch_types<float, _Float16>(a, act, st);
    else launch_types<float, float>(a, act, st);
  }
  return hipGetLastError();
}

}  // namespace w4a4
