// w4a16.hip — y = x . W^T for few rows, W in 4-bit codes with group scales, the
// activations as they are.
//
//   y[m, n] = sum_j s[n, j] sum_{k in group j} x[m, k] q[n, k]
//
// Weights come in tiles of 16 channels and 128 of K: lane 16 g + r loads the 16
// bytes that hold codes [32 g, +32) of channel r, which in tiled weights makes
// one run of 1 KB, and widens each word to an operand of the 16 x 16 x 32
// matrix instruction.  The order of K inside an instruction is free, so x is
// brought to the codes' order.
//
// fp16 x meets fp16 codes.  float32 x enters as three bfloat16 parts, which hold
// all its 24 bits.  Products are exact in both, sums float32; only the result is
// rounded to fewer bits, where fp16 is asked for.  A tile whose halves have
// different scales (groups of an odd multiple of 64) is multiplied once per half,
// with the other half of x zero.
//
// What bounds it: the codes' bytes, at 5.2 TB/s of a large copy.  8 x 4096 ->
// 28672 (61 MB) takes 15.4 us, 4.0 TB/s, against 11.7; one token 4096 -> 6144 (13
// MB, 2.5 us) 5.7, which is the launch and one way to memory and back; 64 x 14336
// -> 4096 (31.7 MB, 6.1 us) 18.2: 15 in the product, whose tiles of x, 16 KB
// beside 8 KB of codes, each wait for a barrier, and 3 in the parts' sum.  float32
// x, with three matrix instructions for one and its parts to be made, takes 24.8
// and 37.8 us at the two larger sizes, with one scale a channel.
#include "decode_internal.h"
#include "gemm_common.h"
#include "int4_operands.h"

namespace w4a4 {
namespace {

constexpr int kWaves = 8;      // of a workgroup, few rows
constexpr int kManyWaves = 4;  // many rows: that share a tile of x
constexpr int kManySides = 2;  // and how many such tiles at a time

enum Groups { WHOLE = 0, TILES = 1, HALVES = 2 };  // scales: one per channel, per tiles, per half tiles

// Where a lane's codes and scales of 16 channels lie: uniform bases and 32-bit
// offsets, two registers instead of six.
struct Channels {
  const uint8_t* base;
  int64_t n0, scale;        // the first channel, its first scale
  uint32_t off, scale_off;  // the lane's
  int in;                   // its channel is n0 + in (the last one past N)
  __device__ __forceinline__ void set(const W4a16Args& a, int64_t block, int lane) {
    const int64_t last = (a.N - 1) / 16;
    block = block < last ? block : last;  // a block past the last one repeats it
    n0 = block * 16;
    const int left = a.N - n0 < 16 ? static_cast<int>(a.N - n0) : 16;
    in = (lane & 15) < left ? lane & 15 : left - 1;
    base = a.wq + (a.tiled ? block * (8 * static_cast<int64_t>(a.K)) : n0 * (a.K / 2));
    off = a.tiled ? lane * 16 : in * (a.K / 2) + (lane >> 4) * 16;
    scale = n0 * a.groups;
    scale_off = in * a.groups;
  }
  __device__ __forceinline__ u4 codes(int64_t at, bool past) const {
    return *reinterpret_cast<const u4*>(base + at + (off - (past ? 32u : 0u)));
  }
};

// Scales of 16 channels, four half tiles or tiles to a load: lane (r, i) holds that
// of the i-th from `first` on (in halves or tiles of K, not past `end`), and
// element i of channel r is that lane's.
template <int GROUPS>
__device__ __forceinline__ uint32_t load_scales(const W4a16Args& a, const Channels& ch, int first, int end, int i) {
  int at = first + i;
  if constexpr (GROUPS == HALVES) end = end < a.K / 64 ? end : a.K / 64;  // K may end in the middle of the last tile
  at = at < end ? at : end - 1;
  const uint32_t s = ch.scale_off + a.group_halves.quotient(GROUPS == HALVES ? at : 2 * at);
  return a.sw_f16 ? (static_cast<const uint16_t*>(a.sw) + ch.scale)[s]
                  : (static_cast<const uint32_t*>(a.sw) + ch.scale)[s];
}
__device__ __forceinline__ float scale_of(const W4a16Args& a, uint32_t s) {
  return a.sw_f16 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(s))) : float_of(s);
}
__device__ __forceinline__ float spread_scale(float s, int i, int r) { return __shfl(s, 16 * i + r); }

// x's operands for the word j of a tile's codes.
// `past` lanes hold what lies behind K: zeros.
// (Here, where the values are used: a change right behind the load would wait for
// it, and with it for every other load on its way.)
template <bool XF16>
__device__ __forceinline__ void widen_x(u4* v, bool last, bool past, Operand* o) {
  if (last) {
#pragma unroll
    for (int i = 0; i < (XF16 ? 1 : 2); ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = past ? 0u : v[i][e];
  }
  if constexpr (XF16)
    o[0] = order_04152637(v[0]);
  else
    split_bf16(reinterpret_cast<const float*>(v), o);
}
template <bool XF16>
__device__ __forceinline__ Operand widen_codes(uint32_t w, const Masks& m) {
  return XF16 ? int4_to_f16(w, m) : int4_to_bf16_over16(w);
}
template <bool XF16>
__device__ __forceinline__ f4 multiply(const Operand& x, const Operand& q, f4 d) {
  if constexpr (XF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x.h, q.h, d, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.b, q.b, d, 0, 0, 0);
}
// The operand with the other half of the tile's K zero: lanes of g / 2 == h stay.
__device__ __forceinline__ Operand half_of(const Operand& x, bool keep) {
  Operand o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o.w[e] = keep ? x.w[e] : 0u;
  return o;
}

__device__ __forceinline__ void store_y(const W4a16Args& a, int parts, int part, int64_t row, int64_t col, float y) {
  if (parts > 1)
    a.partial[(part * a.M + row) * a.N + col] = y;
  else if (a.y_f16)
    static_cast<_Float16*>(a.y)[row * a.ldy + col] = static_cast<_Float16>(y);
  else
    static_cast<float*>(a.y)[row * a.ldy + col] = y;
}

// Up to 16 rows: a workgroup takes 16 NB channels, its waves runs of their tiles,
// and adds the waves' sums up through LDS, in their order.  Each wave brings x
// from the caches itself (rows past M repeat the last one and are not stored).
// All loads of U tiles are issued before the first is used; at 8 x 4096 -> 28672 a
// ring of single tiles instead took 23 us for 17.5, loads that bypass the caches 23,
// and registers for one workgroup a compute unit only 17.4 for 15.7.  (With 16 or 32
// channels a workgroup has a compute unit to itself, and four tiles at a time take
// the registers of two: 8 x 4096 -> 8192 8.2 us with two, 7.8 with four.)
template <bool XF16, int NB, int GROUPS>
__global__ void __launch_bounds__(kWaves * 64, NB == 4 && XF16 && GROUPS != HALVES ? 4 : 2)
    w4a16_few_kernel(W4a16Args a, int ntiles) {
  constexpr int PARTS = XF16 ? 1 : 3, HALF = GROUPS == HALVES ? 2 : 1;
  constexpr int XV = XF16 ? 1 : 2;                   // 16 bytes of x to eight elements
  constexpr int U = NB <= 2 && XF16 ? 4 : 2;         // tiles of each block of channels on their way together
  constexpr int SL = GROUPS == WHOLE ? 1 : U * HALF / 4 < 1 ? 1 : U * HALF / 4;  // loads of their scales
  __shared__ f4 lds[kWaves][NB][64];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block0 = static_cast<int64_t>(blockIdx.x) * NB;
  const int share = (ntiles + kWaves - 1) / kWaves;
  const int t0 = wave * share, t1 = t0 + share < ntiles ? t0 + share : ntiles;
  const int64_t wstep = a.tiled ? 1024 : 64;
  const bool half_tile = (a.K & 127) != 0;  // the last tile's upper half is past K (row-major only)
  const int64_t m = r < a.M ? r : a.M - 1;
  const char* x = static_cast<const char*>(a.x) + (m * a.ldx + 32 * g) * (XF16 ? 2 : 4);
  f4 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f4{0.f, 0.f, 0.f, 0.f};
  Channels ch[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) ch[b].set(a, block0 + b, lane);
  const Masks masks;

  for (int t = t0; t < t1; t += U) {
    u4 c[U][NB], xr[U][4][XV];
    uint32_t sr[NB][SL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tt = t + u < t1 ? t + u : t1 - 1;
      const bool past = half_tile && tt == ntiles - 1 && g >= 2;  // this lane's codes are past K
#pragma unroll
      for (int b = 0; b < NB; ++b)
        c[u][b] = ch[b].codes(tt * wstep, past);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < XV; ++e) {
          const char* p = x + tt * (256 * XV) + j * (16 * XV) - (past ? 128 * XV : 0);
          xr[u][j][e] = reinterpret_cast<const u4*>(p)[e];
        }
    }
    if constexpr (GROUPS != WHOLE) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int l = 0; l < SL; ++l) sr[b][l] = load_scales<GROUPS>(a, ch[b], t * HALF + 4 * l, t1 * HALF, g);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u >= t1) break;
      f4 sum[NB][HALF];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < HALF; ++h) sum[b][h] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // eight codes of every lane at a time
        Operand xo[PARTS];
        widen_x<XF16>(xr[u][j], half_tile && t + u == ntiles - 1, g >= 2, xo);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const Operand q = widen_codes<XF16>(c[u][b][j], masks);
#pragma unroll
          for (int h = 0; h < HALF; ++h)
#pragma unroll
            for (int i = PARTS - 1; i >= 0; --i) {  // the small parts first
              f4& d = GROUPS == WHOLE ? acc[b] : sum[b][h];
              d = multiply<XF16>(HALF == 1 ? xo[i] : half_of(xo[i], (g >= 2) == (h == 1)), q, d);
            }
        }
      }
      if constexpr (GROUPS != WHOLE) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < HALF; ++h) {
            const int i = u * HALF + h;
            const float s = spread_scale(scale_of(a, sr[b][i / 4]), i % 4, r);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][e] = fmaf(s, sum[b][h][e], acc[b][e]);
          }
      }
    }
  }

#pragma unroll
  for (int b = 0; b < NB; ++b) lds[wave][b][lane] = acc[b];
  __syncthreads();
  for (int b = wave; b < NB; b += kWaves) {
    f4 v = lds[0][b][lane];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v += lds[k][b][lane];
    const int64_t col = (block0 + b) * 16 + r;
    if (col >= a.N) continue;
    float f = XF16 ? 1.f : 16.f;
    if constexpr (GROUPS == WHOLE) f *= load_scale(a.sw, col, a.sw_f16);
    asm volatile("" : "+v"(f));  // waits for it here, once, and not in each branch of a store
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (4 * g + e < a.M) store_y(a, 1, 0, 4 * g + e, col, v[e] * f);
  }
}

// More rows: a wave takes 16 NB channels, a workgroup those of its waves, 16 MT
// rows and a part of K.  Its two sides of four waves take every second tile each
// and add up through LDS (parts over workgroups instead would be written and read
// again).  x goes through LDS as operands, a tile ahead, each thread bringing its
// share; the waves' codes come from memory to registers a tile ahead too.
template <bool XF16, int NB, int MT, int GROUPS>
__global__ void __launch_bounds__(kManySides * kManyWaves * 64, 2)
    w4a16_many_kernel(W4a16Args a, Divisor parts, int share, int longer, int ntiles) {
  constexpr int PARTS = XF16 ? 1 : 3, HALF = GROUPS == HALVES ? 2 : 1;
  constexpr int BUFFERS = XF16 ? 2 : 1;
  // A thread brings the operands (i, j) of MT * 4, lane its own, of its wave.
  constexpr int OWN = MT * 4 / kManyWaves;
  constexpr int SIDE = BUFFERS * PARTS * MT * 4 * 64;                // of LDS, in u4
  constexpr int COLS = 16 * NB * kManyWaves;                         // of the workgroup
  static_assert(kManySides * 16 * MT * COLS <= kManySides * SIDE * 4, "the sides' sums fit LDS");
  __shared__ u4 shared[kManySides * SIDE];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int side = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / kManyWaves;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % kManyWaves;
  u4(*lds)[PARTS][MT * 4][64] = reinterpret_cast<u4(*)[PARTS][MT * 4][64]>(shared + side * SIDE);
  const int group = parts.quotient(blockIdx.x), part = blockIdx.x - group * parts.d;
  const int64_t block0 = (static_cast<int64_t>(group) * kManyWaves + wave) * NB;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
  const int t0 = part * share + (part < longer ? part : longer);  // the first parts have a tile more
  const int t1 = t0 + share + (part < longer ? 1 : 0);
  const int64_t wstep = a.tiled ? 1024 : 64;
  const bool half_tile = (a.K & 127) != 0;
  Channels ch[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) ch[b].set(a, block0 + b, lane);
  const char* x[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    const int o = wave * OWN + i;  // operand o: row block o / 4, word o % 4
    int64_t m = m0 + 16 * (o / 4) + r;
    m = m < a.M ? m : a.M - 1;
    x[i] = static_cast<const char*>(a.x) + (m * a.ldx + 32 * g + 8 * (o % 4)) * (XF16 ? 2 : 4);
  }
  const Masks masks;
  f4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[b][i] = f4{0.f, 0.f, 0.f, 0.f};

  u4 c[NB];
  uint32_t s[NB];
  u4 raw[OWN][XF16 ? 1 : 2];
  auto bring = [&](int t) {
    const bool past = half_tile && t == ntiles - 1 && g >= 2;
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
      for (int e = 0; e < (XF16 ? 1 : 2); ++e) {
        raw[i][e] = reinterpret_cast<const u4*>(x[i] + t * (XF16 ? 256 : 512) - (past ? (XF16 ? 128 : 256) : 0))[e];
      }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      c[b] = ch[b].codes(t * wstep, past);
      if constexpr (GROUPS != WHOLE) s[b] = load_scales<GROUPS>(a, ch[b], t * HALF, ntiles * HALF, g);
    }
  };
  auto put = [&](int t, int buffer) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      Operand o[PARTS];
      widen_x<XF16>(raw[i], half_tile && t == ntiles - 1, g >= 2, o);
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        lds[buffer][p][wave * OWN + i][lane] = u4{o[p].w[0], o[p].w[1], o[p].w[2], o[p].w[3]};
    }
  };
  // A side past the last tile goes through the motions with it, for the barriers.
  bring(t0 + side < t1 ? t0 + side : t0);
  for (int at = t0; at < t1; at += kManySides) {
    const int t = at + side < t1 ? at + side : t0;
    const int buffer = BUFFERS == 2 ? (at - t0) / kManySides & 1 : 0;
    if (BUFFERS == 1 && at > t0) __syncthreads();  // the tile before is used up
    put(t, buffer);
    u4 now[NB];
    uint32_t sn[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      now[b] = c[b];
      if constexpr (GROUPS != WHOLE) sn[b] = s[b];
    }
    bring(t + kManySides < t1 ? t + kManySides : t0);
    __syncthreads();
    if (at + side >= t1) continue;
    f4 sum[NB][MT][HALF];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < HALF; ++h) sum[b][i][h] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Operand q[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) q[b] = widen_codes<XF16>(now[b][j], masks);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int p = PARTS - 1; p >= 0; --p) {
          Operand xo;
          const u4 v = lds[buffer][p][4 * i + j][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) xo.w[e] = v[e];
#pragma unroll
          for (int h = 0; h < HALF; ++h) {
            const Operand xh = HALF == 1 ? xo : half_of(xo, (g >= 2) == (h == 1));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              f4& d = GROUPS == WHOLE ? acc[b][i] : sum[b][i][h];
              d = multiply<XF16>(xh, q[b], d);
            }
          }
        }
    }
    if constexpr (GROUPS != WHOLE) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < HALF; ++h) {
          const float f = spread_scale(scale_of(a, sn[b]), h, r);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][i][e] = fmaf(f, sum[b][i][h][e], acc[b][i][e]);
        }
    }
  }

  // The sides' sums as rows of COLS columns, their groups of 16 exchanged by row so
  // that a wave's writes meet different banks; then whole rows go out.
  float* const sums = reinterpret_cast<float*>(shared);
  __syncthreads();
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    float f = XF16 ? 1.f : 16.f;
    if constexpr (GROUPS == WHOLE) f *= load_scale(a.sw, ch[b].n0 + ch[b].in, a.sw_f16);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 16 * i + 4 * g + e, col = (wave * NB + b) * 16 + r;
        sums[(side * 16 * MT + row) * COLS + (col ^ (16 * g))] = acc[b][i][e] * f;
      }
  }
  __syncthreads();
  const int64_t col0 = static_cast<int64_t>(group) * COLS;
  const bool wide = a.N % 4 == 0 && (parts.d > 1 || a.y_wide);
#pragma unroll
  for (int k = 0; k < 16 * MT * COLS / 4; k += kManySides * kManyWaves * 64) {
    const int at = k + threadIdx.x, row = at / (COLS / 4), c = at % (COLS / 4) * 4;
    const int from = row * COLS + (c ^ (16 * (row / 4 % 4)));
    f4 v = *reinterpret_cast<const f4*>(sums + from);
#pragma unroll
    for (int s = 1; s < kManySides; ++s) v += *reinterpret_cast<const f4*>(sums + s * (16 * MT * COLS) + from);
    const int64_t m = m0 + row, n = col0 + c;
    if (m >= a.M || n >= a.N) continue;
    if (wide && (parts.d > 1 || !a.y_f16)) {
      float* to = parts.d > 1 ? a.partial + (part * a.M + m) * a.N + n : static_cast<float*>(a.y) + m * a.ldy + n;
      *reinterpret_cast<f4*>(to) = v;
    } else if (wide) {
      typedef _Float16 h4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<h4*>(static_cast<_Float16*>(a.y) + m * a.ldy + n) = __builtin_convertvector(v, h4);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) store_y(a, parts.d, part, m, n + e, v[e]);
    }
  }
}

// The sum over the parts of K, in their order; V columns to a thread.
template <int V>
__global__ void __launch_bounds__(256) w4a16_join_kernel(W4a16Args a, int parts) {
  typedef float fv __attribute__((ext_vector_type(V)));
  const int64_t col = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  const int64_t row = blockIdx.y;
  if (col >= a.N) return;
  fv v = 0.f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) v += *reinterpret_cast<const fv*>(a.partial + (p * a.M + row) * a.N + col);
#pragma unroll
  for (int e = 0; e < V; ++e) store_y(a, 1, 0, row, col + e, v[e]);
}

template <bool XF16, int NB, int MT, int GROUPS>
void launch_kernel(const W4a16Args& a, const W4a16Plan& p, hipStream_t st) {
  const int ntiles = (a.K + 127) / 128;
  const int64_t blocks = (a.N + 15) / 16;
  if constexpr (MT == 1) {
    hipLaunchKernelGGL((w4a16_few_kernel<XF16, NB, GROUPS>), dim3(static_cast<unsigned>((blocks + NB - 1) / NB)),
                       dim3(kWaves * 64), 0, st, a, ntiles);
  } else {
    constexpr int kBlocks = NB * kManyWaves;
    const dim3 grid(static_cast<unsigned>((blocks + kBlocks - 1) / kBlocks * p.parts),
                    static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((w4a16_many_kernel<XF16, NB, MT, GROUPS>), grid, dim3(kManySides * kManyWaves * 64), 0, st, a,
                       Divisor(static_cast<uint32_t>(p.parts)), ntiles / p.parts, ntiles % p.parts, ntiles);
  }
}

template <bool XF16, int NB, int MT>
void launch_groups(const W4a16Args& a, const W4a16Plan& p, hipStream_t st) {
  if (a.groups == 1)
    launch_kernel<XF16, NB, MT, WHOLE>(a, p, st);
  else if (a.group_halves.d % 2 == 0)
    launch_kernel<XF16, NB, MT, TILES>(a, p, st);
  else
    launch_kernel<XF16, NB, MT, HALVES>(a, p, st);
}

template <bool XF16>
void launch_x(const W4a16Args& a, const W4a16Plan& p, hipStream_t st) {
  if (p.mt == 1) {
    if (p.nb == 1)
      launch_groups<XF16, 1, 1>(a, p, st);
    else if (p.nb == 2)
      launch_groups<XF16, 2, 1>(a, p, st);
    else
      launch_groups<XF16, 4, 1>(a, p, st);
  } else if (p.mt == 2) {
    launch_groups<XF16, 2, 2>(a, p, st);
  } else {
    launch_groups<XF16, 2, 4>(a, p, st);
  }
}

}  // namespace

// Up to 16 rows: as few channels to a workgroup as leave one for each compute unit;
// fewer make a second round of them, more leave compute units empty.  Measured
// with 16 / 32 / 64 channels, 8 x 4096 ->: 4096 6.3 / 7.3 / 9.0 us, 8192 8.9 / 8.3
// / 9.6, 12288 12.3 / 11.7 / 9.8, 28672 25.4 / 20.2 / 18.5; float32 5 x 1024 ->
// 5008 6.4 / 5.5 / 6.3.
// More rows: parts of K until 256 workgroups share the work, one on each compute
// unit, each a tile to a side at least.  64 x 14336 -> 4096 takes 18.5 us with 256
// workgroups, 22.0 with 512 and 25.9 with 128 (of more parts the sums are written
// and read again); 58 x 1472 -> 855 12.1 us, with four tiles to a side 19.8.
W4a16Plan w4a16_plan(int64_t M, int64_t N, int64_t K) {
  const int64_t blocks = (N + 15) / 16, tiles = (K + 127) / 128;
  W4a16Plan p{1, 1, 1};
  if (M <= 16) {
    p.nb = blocks <= 256 ? 1 : blocks <= 512 ? 2 : 4;
    return p;
  }
  p.nb = 2;
  p.mt = M <= 32 ? 2 : 4;
  const int64_t groups = (blocks + 2 * kManyWaves - 1) / (2 * kManyWaves) * ((M + 16 * p.mt - 1) / (16 * p.mt));
  int64_t parts = 256 / groups;
  const int64_t most = tiles / kManySides;
  parts = parts < most ? parts : most;
  p.parts = static_cast<int>(parts < 1 ? 1 : parts);
  return p;
}

hipError_t launch_w4a16(const W4a16Args& a, bool x_f16, hipStream_t st) {
  const W4a16Plan p = w4a16_plan(a.M, a.N, a.K);
  x_f16 ? launch_x<true>(a, p, st) : launch_x<false>(a, p, st);
  if (p.parts > 1) {
    if (a.N % 4 == 0)
      hipLaunchKernelGGL(w4a16_join_kernel<4>,
                         dim3(static_cast<unsigned>((a.N + 1023) / 1024), static_cast<unsigned>(a.M)), dim3(256), 0, st,
                         a, p.parts);
    else
      hipLaunchKernelGGL(w4a16_join_kernel<1>, dim3(static_cast<unsigned>((a.N + 255) / 256), static_cast<unsigned>(a.M)),
                         dim3(256), 0, st, a, p.parts);
  }
  return hipGetLastError();
}

}  // namespace w4a4
