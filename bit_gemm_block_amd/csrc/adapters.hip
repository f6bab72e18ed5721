// adapters.hip — low-rank adapters of many requests beside one projection:
//   out[m] = y[m] + s_a (x[m] At[a]^T) Bt[a]^T,  a = index[m].
//
// Two launches: the first writes t = x At^T in S parts of K (float32, one
// partial sum per part), the second joins the parts in order and adds
// s_a t Bt^T to y.  No atomics: a row's result is the same from call to call.
//
// Rows are taken in tiles of 16, the row count of the matrix instruction.  A
// tile may hold rows of several adapters: every adapter in it is one pass, led
// by its first row, over operands in which only the adapter's own rows
// are kept (rows of a matrix product do not mix, so the other rows of the
// result are simply not stored).
#include "block_internal.h"

namespace w4a4 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

// A lane's 16-byte piece of a matrix operand: lane 16 g + r holds row r,
// channels [FL g, FL g + FL) of a chunk of KC = 4 FL channels.
template <typename T>
struct Frag;
template <>
struct Frag<_Float16> {
  static constexpr int FL = 8, KC = 32;
  typedef half8 V;
  static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  static constexpr int FL = 4, KC = 16;
  typedef f32x4 V;
  // The instruction takes one channel per lane: element i of every lane makes
  // one product over channels {i, 4 + i, 8 + i, 12 + i} of the chunk.
  static __device__ __forceinline__ f32x4 mma(V a, V b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The adapter of row m0 + (lane & 15), -1 where there is none.
__device__ __forceinline__ int row_adapter(const AdapterArgs& a, int64_t m0, int lane) {
  const int64_t m = m0 + (lane & 15);
  if (m >= a.M) return -1;
  const int v = a.index[m];
  return v >= 0 && v < a.L ? v : -1;
}
__device__ __forceinline__ int rank_of(const AdapterArgs& a, int ad) {
  if (!a.ranks) return a.R;
  const int r = uniform(a.ranks[ad]);
  return r < 0 ? 0 : r > a.R ? a.R : r;
}

// ---- t = x . At^T -----------------------------------------------------------
// One workgroup of four waves per (tile, part of K, slots): slot s (or every
// slot in turn, where grid.z is 1) runs the adapter led by row s of the tile.
// The waves share the part; their sums are joined in LDS in order.
constexpr int kShrinkWaves = 4;

template <typename T, int NT>
__device__ void shrink_pass(const AdapterArgs& a, int64_t m0, int ad, bool mine, int k0, int k1,
                            int split, f32x4 (*red)[NT][64]) {
  using F = Frag<T>;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rank = rank_of(a, ad);
  const int64_t m = m0 + r;
  f32x4 acc[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int chunks = (k1 - k0) / F::KC;
  const int c0 = chunks * wave / kShrinkWaves, c1 = chunks * (wave + 1) / kShrinkWaves;
  const T* xr = static_cast<const T*>(a.x) + (mine ? m : 0) * a.ldx;
  const T* ar = static_cast<const T*>(a.At) + static_cast<int64_t>(ad) * a.R * a.K;
  for (int ch = c0; ch < c1; ++ch) {
    const int k = k0 + ch * F::KC + g * F::FL;
    typename F::V xv = {};
    if (mine) xv = *reinterpret_cast<const typename F::V*>(xr + k);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      if (16 * c >= rank) break;
      const int j = 16 * c + r;
      typename F::V av = {};
      if (j < rank) av = *reinterpret_cast<const typename F::V*>(ar + static_cast<int64_t>(j) * a.K + k);
      acc[c] = F::mma(av, xv, acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < NT; ++c) red[wave][c][lane] = acc[c];
  __syncthreads();
  // Result lane 16 g + r: columns 16 c + 4 g + i of t, row r.
  float* tp = a.t + (static_cast<int64_t>(split) * a.M + m) * adapter_tstride(a.R);
  for (int c = wave; c < NT; c += kShrinkWaves) {
    if (16 * c >= rank) break;
    f32x4 s = red[0][c][lane];
#pragma unroll
    for (int w = 1; w < kShrinkWaves; ++w) s += red[w][c][lane];
    if (mine) *reinterpret_cast<f32x4*>(tp + 16 * c + 4 * g) = s;
  }
  __syncthreads();
}

template <typename T, int NT>
__global__ void __launch_bounds__(64 * kShrinkWaves) shrink_kernel(AdapterArgs a) {
  __shared__ f32x4 red[kShrinkWaves][NT][64];
  const int lane = threadIdx.x & 63;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int split = blockIdx.y;
  const int k0 = a.K / 64 * split / a.S * 64, k1 = a.K / 64 * (split + 1) / a.S * 64;
  const int my = row_adapter(a, m0, lane);
  for (int s = blockIdx.z; s < 16; s += gridDim.z) {
    const int ad = __builtin_amdgcn_readlane(my, s);
    if (ad < 0) continue;
    const bool mine = my == ad;
    if (static_cast<int>(__builtin_ctzll(__ballot(mine))) != s) continue;  // led by another row
    shrink_pass<T, NT>(a, m0, ad, mine, k0, k1, split, red);
  }
}

// ---- out = y + s t . Bt^T ---------------------------------------------------
// One workgroup of four waves per (tile, 256 columns, slots); a wave has 64
// columns.  The product is formed transposed (rows: columns of out), so that a
// lane holds four consecutive columns of one row.
constexpr int kExpandCols = 256;

// Chunk c of row m's t (scaled), channels [FL g, FL g + FL), zero past the rank.
template <typename T>
__device__ __forceinline__ void load_t(const AdapterArgs& a, int64_t m, int j0, int rank, float s,
                                       float* v) {
  constexpr int FL = Frag<T>::FL;
  const int64_t ts = adapter_tstride(a.R);
#pragma unroll
  for (int e = 0; e < FL; ++e) v[e] = 0.f;
  const float* p = a.t + m * ts + j0;
  for (int q = 0; q < a.S; ++q, p += a.M * ts) {
#pragma unroll
    for (int e = 0; e < FL; e += 4) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(p + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[e + i] += w[i];
    }
  }
#pragma unroll
  for (int e = 0; e < FL; ++e) v[e] = j0 + e < rank ? v[e] * s : 0.f;
}

template <typename T, int NC>
__device__ void expand_pass(const AdapterArgs& a, int64_t m0, int ad, bool mine, int64_t n0) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr bool F16 = F::FL == 8;
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int64_t m = m0 + r;
  const int rank = ad < 0 ? 0 : rank_of(a, ad);
  f32x4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
  float unscale = 1.f;
  if (rank > 0) {
    const float s = a.scales ? a.scales[ad] : 1.f;
    V hi[NC], lo[NC];
    if constexpr (F16) {
      // The row's largest finite |t| is moved to [2^13, 2^14): t fits an fp16 pair
      // whatever its magnitude.
      float v[NC][8];
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (mine && c * 32 < rank) {
          load_t<T>(a, m, c * 32 + 8 * g, rank, s, v[c]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(v[c][e]) < INFINITY) big = fmaxf(big, fabsf(v[c][e]));
      }
      big = fmaxf(big, __shfl_xor(big, 16));
      big = fmaxf(big, __shfl_xor(big, 32));
      float scale = 1.f;
      if (big > 0.f) {
        int e;
        (void)frexpf(big, &e);  // big = f 2^e, f in [1/2, 1)
        e = 14 - e;
        e = e > 120 ? 120 : e;
        scale = ldexpf(1.f, e);
        unscale = ldexpf(1.f, -e);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = v[c][e] * scale;
          const _Float16 h = static_cast<_Float16>(u);
          const float d = u - static_cast<float>(h);
          hi[c][e] = h;
          lo[c][e] = fabsf(u) < INFINITY ? static_cast<_Float16>(d) : static_cast<_Float16>(0.f);
        }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (mine && c * 16 < rank) load_t<T>(a, m, c * 16 + 4 * g, rank, s, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) hi[c][e] = v[e];
      }
    }
    const T* bb = static_cast<const T*>(a.Bt) + static_cast<int64_t>(ad) * a.N * a.R;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (c * F::KC >= rank) break;
      const int j = c * F::KC + g * F::FL;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t n = n0 + 16 * q + r < a.N ? n0 + 16 * q + r : a.N - 1;
        const T* p = bb + n * a.R + j;
        V b = {};
        if (a.R % F::FL == 0) {
          if (j < a.R) b = *reinterpret_cast<const V*>(p);
        } else {
#pragma unroll
          for (int e = 0; e < F::FL; ++e)
            if (j + e < a.R) b[e] = p[e];
        }
        if (c * F::KC + F::KC > rank) {
#pragma unroll
          for (int e = 0; e < F::FL; ++e) b[e] = j + e < rank ? b[e] : static_cast<T>(0.f);
        }
        acc[q] = F::mma(b, hi[c], acc[q]);
        if constexpr (F16) acc[q] = F::mma(b, lo[c], acc[q]);
      }
    }
  }
  // Result lane 16 g + r: columns n0 + 16 q + 4 g + i, row r.
  if (!mine) return;
  const float* yr = a.y ? a.y + m * a.ldy : nullptr;
  float* orow = a.out + m * a.ldo;
  const bool vec = a.N % 4 == 0 && a.ldo % 4 == 0 && a.ldy % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 16 * q + 4 * g;
    if (vec) {
      if (n < a.N) {
        f32x4 v = acc[q] * unscale;
        if (yr) v += *reinterpret_cast<const f32x4*>(yr + n);
        *reinterpret_cast<f32x4*>(orow + n) = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) orow[n + i] = (yr ? yr[n + i] : 0.f) + acc[q][i] * unscale;
    }
  }
}

template <typename T, int NC>
__global__ void __launch_bounds__(256) expand_kernel(AdapterArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kExpandCols + 64 * wave;
  if (n0 >= a.N) return;
  const int my = row_adapter(a, m0, lane);
  const bool row = m0 + (lane & 15) < a.M;
  for (int s = blockIdx.z; s < 16; s += gridDim.z) {
    if (m0 + s >= a.M) break;
    const int ad = __builtin_amdgcn_readlane(my, s);
    const bool mine = row && my == ad;
    if (static_cast<int>(__builtin_ctzll(__ballot(mine))) != s) continue;  // led by another row
    if (ad < 0 && a.y == a.out) continue;  // in place, nothing to add
    expand_pass<T, NC>(a, m0, ad, mine, n0);
  }
}

template <typename T, int NT>
void launch_rank(const AdapterArgs& a, hipStream_t st) {
  const int64_t tiles = (a.M + 15) / 16;
  const unsigned slots = tiles >= 64 ? 1 : static_cast<unsigned>(a.M < 16 ? a.M : 16);
  hipLaunchKernelGGL((shrink_kernel<T, NT>), dim3(static_cast<unsigned>(tiles), a.S, slots),
                     dim3(64 * kShrinkWaves), 0, st, a);
  constexpr int NC = (16 * NT + Frag<T>::KC - 1) / Frag<T>::KC;
  const unsigned cols = static_cast<unsigned>((a.N + kExpandCols - 1) / kExpandCols);
  hipLaunchKernelGGL((expand_kernel<T, NC>), dim3(static_cast<unsigned>(tiles), cols, slots),
                     dim3(256), 0, st, a);
}

template <typename T>
hipError_t launch_typed(const AdapterArgs& a, hipStream_t st) {
  if (a.R <= 16) launch_rank<T, 1>(a, st);
  else if (a.R <= 32) launch_rank<T, 2>(a, st);
  else if (a.R <= 64) launch_rank<T, 4>(a, st);
  else if (a.R <= 128) launch_rank<T, 8>(a, st);
  else launch_rank<T, 16>(a, st);
  return hipGetLastError();
}

}  // namespace

// Enough parts that a few rows still fill the chip, at least 256 channels each.
int adapter_splits(int64_t M, int64_t K) {
  const int64_t want = (512 + M - 1) / M;
  const int64_t most = (K + 255) / 256;
  const int64_t s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s);
}

hipError_t launch_adapter_add(const AdapterArgs& a, bool f16, hipStream_t st) {
  return f16 ? launch_typed<_Float16>(a, st) : launch_typed<float>(a, st);
}

}  // namespace w4a4
