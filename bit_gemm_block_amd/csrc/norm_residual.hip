// norm_residual.hip — the seam between two blocks in one pass over a row:
//   v = norm_post(y) * gate;  h' = h + rs v;  x = norm_pre(h').
//
// A row stays in the registers of one workgroup (T threads, 8 NC channels
// each), so y and h are read once and h' and x written once; the statistics
// are float32 sums over the row, the variance of a layer norm over the
// centred values (a second sum over registers, not a second read).
//
// What bounds it: long calls by memory (4096 x 4096, fp32 rows, fp16 x: 235 MB in
// 45 us, 5.2 TB/s), up to 4096 x 16384, fp16 rows, fp32 y, a gate: 671 MB in 139 to 146
// us, 4.6 to 4.8 TB/s, where the loads of a 16-wave workgroup, one to a compute unit,
// pause at its sums.  Short ones by latency (8 x 4096: 3.8 to 4.0 us, of which an empty
// launch is 1.6): a load, two or four sums over the workgroup, each of six exchanges
// between lanes that go through LDS and a barrier, and the parameters' loads follow one
// another.  The parameters are not loaded before the sums: kept in registers
// they spill at 1024 threads (4096 x 16384: 150 -> 269 us), and brought early into
// the caches they gain nothing (8 x 4096: 4.16 -> 4.25 us).
#include "block_internal.h"
#include "vec_io.h"

#include "w4a4_block.h"

namespace w4a4 {
namespace {

// Sum over the WAVES * 64 threads of a workgroup.  Two slots in turn: a wave
// reaches the write of slot s again only after the barrier of the other
// slot's sum, which every wave passes after it has read slot s.
template <int WAVES>
struct RowSum {
  float* lds;  // [2][WAVES]
  int slot = 0;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if constexpr (WAVES > 1) {
      float* s = lds + slot * WAVES;
      slot ^= 1;
      if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
      __syncthreads();
      v = s[0];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += s[w];
    }
    return v;
  }
};

// How a thread's chunk of eight channels from c = 8 (i T + t) meets the row's
// end.  EVEN (C % 8 == 0): a chunk is in the row or past it.  SHIFTED (C >= 8):
// the chunk that crosses the end moves back to the row's last eight channels
// and does not own those that its neighbour has as well, so that every load is
// one whole, unconditional one (a branch around the last elements' own loads
// cost more than the kernel's whole work: 777 x 5003, 29.7 -> 19 us).  SHORT
// (C < 8): elements one by one.
enum Ends { EVEN = 0, SHIFTED = 1, SHORT = 2 };

// One row per workgroup (WAVES > 1) or per wave (WAVES == 1, four rows per
// workgroup), NC chunks per thread.
template <int WAVES, int NC, int ENDS, typename H, typename Y, typename P>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) norm_residual_kernel(NormArgs a) {
  constexpr int T = WAVES * 64;
  constexpr int E = 8 * NC;
  __shared__ float lds[2 * WAVES];
  RowSum<WAVES> row_sum{lds};
  const int C = a.C;
  const int t = WAVES == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const float inv_c = 1.f / static_cast<float>(C);
  const int64_t row0 = WAVES == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (WAVES == 1 ? 4 : 1);

  // Chunk i starts at col[i] and owns its elements from skip[i] on.
  int col[NC], skip[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * T + t) * 8;
    if constexpr (ENDS == EVEN) {
      col[i] = c < C ? c : 0;
      skip[i] = c < C ? 0 : 8;
    } else if constexpr (ENDS == SHIFTED) {
      col[i] = c + 8 <= C ? c : C - 8;
      skip[i] = c - col[i];
    } else {
      col[i] = c;
      skip[i] = 0;
    }
  }
  auto owned = [&](int j) {
    const int i = j / 8, e = j % 8;
    return ENDS == EVEN ? skip[i] == 0 : ENDS == SHIFTED ? e >= skip[i] : col[i] + e < C;
  };
  // Elements of a row; those that the thread does not own may be anything.
  auto load_row = [&](auto* p, float* out) {
    using Q = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
    Raw8<Q> r[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if constexpr (ENDS == SHORT)
        r[i] = load8_once(p, col[i], C);
      else
        r[i].load(p + col[i]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) out[j] = r[j / 8].get(j % 8);
  };
  auto store_row = [&](auto* p, const float* v) {
    using Q = std::remove_reference_t<decltype(*p)>;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if constexpr (ENDS == SHORT) {
        store8(p, col[i], C, v + 8 * i);
      } else {
        if (skip[i] == 0) {
          store_whole8(p + col[i], v + 8 * i);
        } else if (ENDS == SHIFTED && skip[i] < 8) {
#pragma unroll
          for (int e = 1; e < 8; ++e)
            if (e >= skip[i]) p[col[i] + e] = static_cast<Q>(v[8 * i + e]);
        }
      }
    }
  };
  auto norm = [&](float* v, int kind, const void* w, const void* b) {
    if (kind == W4A4_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) s += v[j];
      const float mean = row_sum(s) * inv_c;
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = owned(j) ? v[j] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) q = fmaf(v[j], v[j], q);
    const float r = 1.f / sqrtf(row_sum(q) * inv_c + a.eps);
    if (w) {
      float p[E];
      load_row(static_cast<const P*>(w), p);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= r * (a.offset + p[j]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= r;
    }
    if (b) {
      float p[E];
      load_row(static_cast<const P*>(b), p);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] += p[j];
    }
  };

  for (int64_t m = row0; m < a.M; m += step) {
    float v[E], h[E];
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = h[j] = 0.f;
    if (a.y) load_row(static_cast<const Y*>(a.y) + m * a.ldy, v);
    if (a.h) load_row(static_cast<const H*>(a.h) + m * a.ldh, h);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = owned(j) ? v[j] : 0.f;
    if (a.post != W4A4_NORM_NONE) norm(v, a.post, a.post_w, a.post_b);
    if (a.gate) {
      float g[E];
      const int64_t gr = m / a.gate_rows * a.ldg;
      if (a.gate_f16)
        load_row(static_cast<const _Float16*>(a.gate) + gr, g);
      else
        load_row(static_cast<const float*>(a.gate) + gr, g);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] *= g[j];
    }
    if (a.y) {
#pragma unroll
      for (int j = 0; j < E; ++j) h[j] = fmaf(a.rs, v[j], h[j]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) h[j] = owned(j) ? h[j] : 0.f;
    if (a.h_out) store_row(static_cast<H*>(a.h_out) + m * a.ldho, h);
    if (a.x_out) {
      if (a.pre != W4A4_NORM_NONE) norm(h, a.pre, a.pre_w, a.pre_b);
      if (a.x_f16)
        store_row(static_cast<_Float16*>(a.x_out) + m * a.ldx, h);
      else
        store_row(static_cast<float*>(a.x_out) + m * a.ldx, h);
    }
  }
}

template <int WAVES, int NC, typename H, typename Y, typename P>
void launch_shape(const NormArgs& a, hipStream_t st) {
  const int64_t groups = WAVES == 1 ? (a.M + 3) / 4 : a.M;
  const dim3 grid(static_cast<unsigned>(groups < (1 << 20) ? groups : (1 << 20)));
  const dim3 block(WAVES == 1 ? 256 : WAVES * 64);
  if constexpr (WAVES == 1) {
    if (a.C < 8) {
      hipLaunchKernelGGL((norm_residual_kernel<WAVES, NC, SHORT, H, Y, P>), grid, block, 0, st, a);
      return;
    }
  }
  if (a.C % 8)
    hipLaunchKernelGGL((norm_residual_kernel<WAVES, NC, SHIFTED, H, Y, P>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_residual_kernel<WAVES, NC, EVEN, H, Y, P>), grid, block, 0, st, a);
}

// The waves that a row needs with one chunk each, two from C = 4096 on.  Both sides, three
// sets of inputs in turn: four waves for C <= 512 cost 11.8 us instead of 7.5 (4096 x
// 512); for C = 4096 four with two chunks 4.15 instead of 3.97 (8 rows), 4.95 instead of
// 4.74 (256) and the same 45.2 (4096); for C = 8192 sixteen with one chunk 5.07 instead
// of 4.69 (8) and 105 instead of 86.5 (4096); for C = 16384 eight with four 6.2 instead
// of 6.0 (8) and 146 instead of 139 (4096).
template <typename H, typename Y, typename P>
void launch_types(const NormArgs& a, hipStream_t st) {
  if (a.C <= 512) return launch_shape<1, 1, H, Y, P>(a, st);
  if (a.C <= 2048) return launch_shape<4, 1, H, Y, P>(a, st);
  if (a.C <= 4096) return launch_shape<8, 1, H, Y, P>(a, st);
  if (a.C <= 8192) return launch_shape<8, 2, H, Y, P>(a, st);
  return launch_shape<16, 2, H, Y, P>(a, st);
}

}  // namespace

hipError_t launch_norm_residual(const NormArgs& a, bool h_f16, bool y_f16, bool p_f16,
                                hipStream_t st) {
  typedef _Float16 F;
  if (h_f16) {
    if (y_f16)
      p_f16 ? launch_types<F, F, F>(a, st) : launch_types<F, F, float>(a, st);
    else
      p_f16 ? launch_types<F, float, F>(a, st) : launch_types<F, float, float>(a, st);
  } else {
    if (y_f16)
      p_f16 ? launch_types<float, F, F>(a, st) : launch_types<float, F, float>(a, st);
    else
      p_f16 ? launch_types<float, float, F>(a, st) : launch_types<float, float, float>(a, st);
  }
  return hipGetLastError();
}

}  // namespace w4a4
