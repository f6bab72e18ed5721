// w4a16.hip — y = x . W^T for few rows, W in 4-bit codes with group scales, the
// activations as they are.
//
//   y[m, n] = sum_j s[n, j] sum_{k in group j} x[m, k] q[n, k]
//
// A wave takes 16 NB output channels and 16 MT rows (rows past M repeat the
// last one and are not stored) over some of K's tiles of 128: lane 16 g + r
// loads the 16 bytes that hold codes [32 g, +32) of channel r, which in tiled
// weights makes one run of 1 KB, and widens each word to an operand of the
// 16 x 16 x 32 matrix instruction.  The order of K inside an instruction is
// free, so x is brought to the codes' order: 32 of its elements to a lane.
// The waves of a workgroup share the channels' tiles, next to each other, and
// add up through LDS in a fixed order.
//
// fp16 x meets fp16 codes.  float32 x enters as three bfloat16 parts.  Products
// are exact in both, sums float32.  A tile whose halves have different scales
// (groups of an odd multiple of 64) is multiplied once per half, with the
// other half of x zero.
#include "decode_internal.h"
#include "gemm_common.h"
#include "int4_operands.h"

namespace w4a4 {
namespace {

constexpr int kWaves = 8;

enum Groups { WHOLE = 0, TILES = 1, HALVES = 2 };  // scales: one per channel, per tiles, per half tiles

template <bool XF16, int NB, int MT, int GROUPS>
__global__ void __launch_bounds__(kWaves * 64) w4a16_kernel(W4a16Args a, int parts, int ntiles) {
  constexpr int PARTS = XF16 ? 1 : 3;
  __shared__ f4 lds[kWaves][NB * MT][64];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = blockIdx.x % parts;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / parts) * (16 * NB);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
  const int t0 = static_cast<int>(static_cast<int64_t>(ntiles) * part / parts);
  const int t1 = static_cast<int>(static_cast<int64_t>(ntiles) * (part + 1) / parts);
  const int ngroups = a.K / a.group;
  const bool half_tile = (a.K & 127) != 0;  // the last tile's upper half is past K (row-major only)

  const uint8_t* w[NB];
  int64_t n[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    n[b] = n0 + 16 * b + r;
    n[b] = n[b] < a.N ? n[b] : a.N - 1;
    // Tiled: a block past the last one repeats it.
    const int64_t blk = n0 / 16 + b < (a.N + 15) / 16 ? n0 / 16 + b : (a.N - 1) / 16;
    w[b] = a.tiled ? a.wq + blk * (8 * static_cast<int64_t>(a.K)) + lane * 16
                   : a.wq + n[b] * (a.K / 2) + g * 16;
  }
  const int64_t wstep = a.tiled ? 1024 : 64;
  const char* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t m = m0 + 16 * i + r;
    m = m < a.M ? m : a.M - 1;
    x[i] = static_cast<const char*>(a.x) + (m * a.ldx + 32 * g) * (XF16 ? 2 : 4);
  }

  f4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[b][i] = f4{0.f, 0.f, 0.f, 0.f};

  for (int t = t0 + wave; t < t1; t += kWaves) {
    const bool past = half_tile && t == ntiles - 1 && g >= 2;  // this lane's codes are past K
    u4 c[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint8_t* p = w[b] + t * wstep - (past ? 32 : 0);
      c[b] = __builtin_nontemporal_load(reinterpret_cast<const u4*>(p));
    }
    float s[NB][GROUPS == HALVES ? 2 : 1];
    if constexpr (GROUPS != WHOLE) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        s[b][0] = load_scale(a.sw, n[b] * ngroups + t * 128 / a.group, a.sw_f16);
        if constexpr (GROUPS == HALVES) {
          const int up = t * 128 + 64 < a.K ? (t * 128 + 64) / a.group : ngroups - 1;
          s[b][1] = load_scale(a.sw, n[b] * ngroups + up, a.sw_f16);
        }
      }
    }
    f4 sum[NB][MT][GROUPS == HALVES ? 2 : 1];
    if constexpr (GROUPS != WHOLE) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < (GROUPS == HALVES ? 2 : 1); ++h) sum[b][i][h] = f4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // eight codes of every lane at a time
      Operand q[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) q[b] = XF16 ? int4_to_f16(c[b][j]) : int4_to_bf16_over16(c[b][j]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        Operand xo[PARTS];
        if constexpr (XF16) {
          u4 v = *reinterpret_cast<const u4*>(x[i] + t * 256 + 16 * j - (past ? 128 : 0));
          if (past) v = u4{0, 0, 0, 0};
          xo[0] = order_04152637(v);
        } else {
          union {
            f4 v[2];
            float f[8];
          } u;
          const f4* p = reinterpret_cast<const f4*>(x[i] + t * 512 + 32 * j - (past ? 256 : 0));
          u.v[0] = p[0];
          u.v[1] = p[1];
          if (past) u.v[0] = u.v[1] = f4{0.f, 0.f, 0.f, 0.f};
          split_bf16(u.f, xo);
        }
#pragma unroll
        for (int h = 0; h < (GROUPS == HALVES ? 2 : 1); ++h) {
#pragma unroll
          for (int p = PARTS - 1; p >= 0; --p) {  // the small parts first
            Operand xh = xo[p];
            if constexpr (GROUPS == HALVES) {
#pragma unroll
              for (int e = 0; e < 4; ++e) xh.w[e] = (g >= 2) == (h == 1) ? xh.w[e] : 0u;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              f4& d = GROUPS == WHOLE ? acc[b][i] : sum[b][i][h];
              if constexpr (XF16)
                d = __builtin_amdgcn_mfma_f32_16x16x32_f16(xh.h, q[b].h, d, 0, 0, 0);
              else
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xh.b, q[b].b, d, 0, 0, 0);
            }
          }
        }
      }
    }
    if constexpr (GROUPS != WHOLE) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < (GROUPS == HALVES ? 2 : 1); ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][i][e] = fmaf(s[b][h], sum[b][i][h][e], acc[b][i][e]);
    }
  }

#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) lds[wave][b * MT + i][lane] = acc[b][i];
  __syncthreads();
  for (int o = wave; o < NB * MT; o += kWaves) {
    f4 v = lds[0][o][lane];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += lds[k][o][lane];
    const int64_t col = n0 + 16 * (o / MT) + r;
    const int64_t row = m0 + 16 * (o % MT) + 4 * g;
    if (col >= a.N) continue;
    float f = XF16 ? 1.f : 16.f;
    if constexpr (GROUPS == WHOLE) f *= load_scale(a.sw, col, a.sw_f16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (row + e >= a.M) break;
      const float y = v[e] * f;
      if (parts > 1)
        a.partial[(part * a.M + row + e) * a.N + col] = y;
      else if (a.y_f16)
        static_cast<_Float16*>(a.y)[(row + e) * a.ldy + col] = static_cast<_Float16>(y);
      else
        static_cast<float*>(a.y)[(row + e) * a.ldy + col] = y;
    }
  }
}

// The sum over the parts of K, in their order.
__global__ void __launch_bounds__(256) w4a16_join_kernel(W4a16Args a, int parts) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = blockIdx.y;
  if (col >= a.N) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v += a.partial[(p * a.M + row) * a.N + col];
  if (a.y_f16)
    static_cast<_Float16*>(a.y)[row * a.ldy + col] = static_cast<_Float16>(v);
  else
    static_cast<float*>(a.y)[row * a.ldy + col] = v;
}

template <bool XF16, int NB, int MT>
void launch_groups(const W4a16Args& a, const W4a16Plan& p, hipStream_t st) {
  const int ntiles = (a.K + 127) / 128;
  const dim3 grid(static_cast<unsigned>((a.N + 16 * NB - 1) / (16 * NB) * p.parts),
                  static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT)));
  const dim3 block(kWaves * 64);
  if (a.group == a.K)
    hipLaunchKernelGGL((w4a16_kernel<XF16, NB, MT, WHOLE>), grid, block, 0, st, a, p.parts, ntiles);
  else if (a.group % 128 == 0)
    hipLaunchKernelGGL((w4a16_kernel<XF16, NB, MT, TILES>), grid, block, 0, st, a, p.parts, ntiles);
  else
    hipLaunchKernelGGL((w4a16_kernel<XF16, NB, MT, HALVES>), grid, block, 0, st, a, p.parts, ntiles);
}

template <bool XF16>
void launch_x(const W4a16Args& a, const W4a16Plan& p, hipStream_t st) {
  if (p.mt == 1)
    launch_groups<XF16, 1, 1>(a, p, st);
  else
    launch_groups<XF16, 1, 4>(a, p, st);
}

}  // namespace

W4a16Plan w4a16_plan(int64_t M, int64_t N, int64_t K) {
  W4a16Plan p{1, M <= 16 ? 1 : 4, kWaves, 1};
  return p;
}

hipError_t launch_w4a16(const W4a16Args& a, bool x_f16, hipStream_t st) {
  const W4a16Plan p = w4a16_plan(a.M, a.N, a.K);
  x_f16 ? launch_x<true>(a, p, st) : launch_x<false>(a, p, st);
  if (p.parts > 1)
    hipLaunchKernelGGL(w4a16_join_kernel, dim3(static_cast<unsigned>((a.N + 255) / 256), static_cast<unsigned>(a.M)),
                       dim3(256), 0, st, a, p.parts);
  return hipGetLastError();
}

}  // namespace w4a4
