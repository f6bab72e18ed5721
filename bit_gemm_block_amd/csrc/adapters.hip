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
#include "gemm_common.h"
#include "vec_io.h"

namespace w4a4 {
namespace {

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

// Row tiles from which the staged kernel takes over.
constexpr int64_t kStageTiles = 64;

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

// ---- t = x . At^T: one 16 x 16 block per workgroup -----------------------------
// Workgroup (tile, part of K and block of 16 ranks, slot): slot s (or every
// slot in turn, where grid.z is 1) runs the adapter led by row s of the tile.
// The waves share the part of K; their sums are joined in LDS in order.  All
// loads are whole and unconditional, PF chunks of them in flight: ranks past
// the adapter's read its last one, rows of other adapters the leading row
// (both fall on lines that are read anyway; neither's result is stored).
constexpr int kBlockWaves = 8;

template <typename T>
__global__ void __launch_bounds__(64 * kBlockWaves) shrink_block_kernel(AdapterArgs a) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr int PF = 4;
  __shared__ f32x4 red[kBlockWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int split = blockIdx.y % a.S, rb = blockIdx.y / a.S;
  const int k0 = a.K / 64 * split / a.S * 64, k1 = a.K / 64 * (split + 1) / a.S * 64;
  const int chunks = (k1 - k0) / F::KC;
  const int c0 = chunks * wave / kBlockWaves, c1 = chunks * (wave + 1) / kBlockWaves;
  const int my = row_adapter(a, m0, lane);
  for (int s = blockIdx.z; s < 16; s += gridDim.z) {
    const int ad = __builtin_amdgcn_readlane(my, s);
    if (ad < 0) continue;
    const bool mine = my == ad;
    if (static_cast<int>(__builtin_ctzll(__ballot(mine))) != s) continue;  // led by another row
    const int rank = rank_of(a, ad);
    if (16 * rb >= rank) continue;
    const int j = 16 * rb + r < rank ? 16 * rb + r : rank - 1;
    const int64_t m = m0 + (mine ? r : s);
    const T* xr = static_cast<const T*>(a.x) + m * a.ldx + k0 + g * F::FL;
    const T* ar = static_cast<const T*>(a.At) + (static_cast<int64_t>(ad) * a.R + j) * a.K + k0 + g * F::FL;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    int ch = c0;
    for (; ch + PF <= c1; ch += PF) {
      V xv[PF], av[PF];
#pragma unroll
      for (int u = 0; u < PF; ++u) {
        av[u] = *reinterpret_cast<const V*>(ar + (ch + u) * F::KC);
        xv[u] = *reinterpret_cast<const V*>(xr + (ch + u) * F::KC);
      }
#pragma unroll
      for (int u = 0; u < PF; ++u) acc = F::mma(av[u], xv[u], acc);
    }
    for (; ch < c1; ++ch)
      acc = F::mma(*reinterpret_cast<const V*>(ar + ch * F::KC),
                   *reinterpret_cast<const V*>(xr + ch * F::KC), acc);
    red[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4 sum = red[0][lane];
#pragma unroll
      for (int w = 1; w < kBlockWaves; ++w) sum += red[w][lane];
      // Result lane 16 g + r: ranks 16 rb + 4 g + i of row r.
      if (mine)
        *reinterpret_cast<f32x4*>(a.t + (static_cast<int64_t>(split) * a.M + m) * adapter_tstride(a.R) +
                                  16 * rb + 4 * g) = sum;
    }
    __syncthreads();
  }
}

// ---- t = x . At^T: many rows, one adapter for most tiles ------------------------
// A workgroup owns 16 rows and all (up to 16 NT) ranks of an adapter in them,
// and streams a part of K through LDS: stage s holds RUN bytes of each of the
// 16 rows of x and the 16 NT rows of At, every row one contiguous run that
// direct-to-LDS copies bring in (register loads of the matrix operands read 16
// rows x 64 bytes per instruction, which the caches serve at a fraction of the
// rate).  Three stages are in flight.  A row's 16-byte units are stored in the
// order u ^ (row & 15), chosen by the copies' addresses, so that the reads of
// one unit of 16 rows fall in distinct banks.
template <typename T, int NT, int RUN, int NW>
__global__ void __launch_bounds__(64 * NW) shrink_stage_kernel(AdapterArgs a) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr int ROWS = 16 + 16 * NT;
  constexpr int UNITS = RUN / 16;          // 16-byte units of a row in a stage
  constexpr int SW = UNITS < 16 ? UNITS - 1 : 15;
  constexpr int RPC = 1024 / RUN;          // rows of one copy
  constexpr int CPW = ROWS / RPC / NW;     // copies per wave and stage
  constexpr int CHUNKS = RUN / 64;         // matrix operands of a stage
  static_assert(ROWS % (RPC * NW) == 0, "whole copies per wave");
  static_assert(CPW < 32, "copies in flight");
  __shared__ __attribute__((aligned(16))) uint8_t st0[ROWS * RUN];
  __shared__ __attribute__((aligned(16))) uint8_t st1[ROWS * RUN];
  __shared__ __attribute__((aligned(16))) uint8_t st2[ROWS * RUN];
  auto stage = [&](int i) -> uint8_t* { return i == 0 ? st0 : i == 1 ? st1 : st2; };
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int split = blockIdx.y;
  const int k0 = a.K / 64 * split / a.S * 64, k1 = a.K / 64 * (split + 1) / a.S * 64;
  const int bytes = (k1 - k0) * static_cast<int>(sizeof(T));
  const int nst = (bytes + RUN - 1) / RUN;
  const int my = row_adapter(a, m0, lane);
  unsigned rest = static_cast<unsigned>(__ballot(my >= 0)) & 0xffffu;
  // Pass p of the tile's adapters runs in workgroup p mod grid.z.
  for (unsigned pass = 0; rest != 0; ++pass) {
    const int ad = __builtin_amdgcn_readlane(my, __builtin_ctz(rest));
    const bool mine = my == ad;
    rest &= ~static_cast<unsigned>(__ballot(mine));
    if (pass % gridDim.z != blockIdx.z) continue;
    const int rank = rank_of(a, ad);
    if (rank == 0) continue;

    // Copy q of this wave: rows RPC (wave + NW q) to + RPC - 1 of the stage.
    const uint8_t* src[CPW];
    int off[CPW];
#pragma unroll
    for (int q = 0; q < CPW; ++q) {
      const int row = RPC * (wave + NW * q) + lane / UNITS;
      off[q] = 16 * ((lane % UNITS) ^ (row & SW));
      const T* p;
      if (row < 16) {
        const int64_t m = m0 + row < a.M ? m0 + row : a.M - 1;
        p = static_cast<const T*>(a.x) + m * a.ldx;
      } else {
        const int j = row - 16 < rank ? row - 16 : rank - 1;
        p = static_cast<const T*>(a.At) + (static_cast<int64_t>(ad) * a.R + j) * a.K;
      }
      src[q] = reinterpret_cast<const uint8_t*>(p + k0);
    }
    auto issue = [&](int s, uint8_t* buf) {
      const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(buf));
      const int left = bytes - s * RUN;  // past the part's end: the stage's first unit again
#pragma unroll
      for (int q = 0; q < CPW; ++q)
        dma16(src[q] + s * RUN + (off[q] < left ? off[q] : 0), b + 1024 * (wave + NW * q));
    };
    f32x4 acc[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const uint8_t* buf, int s) {
      const int valid = (bytes - s * RUN) / 64;
#pragma unroll
      for (int u = 0; u < (CHUNKS + NW - 1) / NW; ++u) {
        const int ch = u * NW + wave;
        if (ch >= CHUNKS || ch >= valid) break;
        const int at = r * RUN + 16 * ((4 * ch + g) ^ (r & SW));  // row & SW is r & SW for every block of 16
        const V xv = *reinterpret_cast<const V*>(buf + at);
        V av[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) av[c] = *reinterpret_cast<const V*>(buf + (16 + 16 * c) * RUN + at);
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[c] = F::mma(av[c], xv, acc[c]);
      }
    };
    // Stage s: once it has landed and the barrier has retired every wave's
    // reads of stage s - 1, that buffer takes stage s + 2.
    auto iterate = [&](int s, int i) {
      if (s + 2 <= nst)
        wait_vmcnt<CPW>();
      else
        wait_vmcnt<0>();
      stage_barrier();
      if (s + 2 < nst) issue(s + 2, stage((i + 2) % 3));
      compute(stage(i), s);
    };
    wait_vmcnt<0>();  // from here on the wave's only vector accesses are the copies
    issue(0, st0);
    if (nst > 1) issue(1, st1);
    for (int s0 = 0; s0 < nst; s0 += 3) {
      iterate(s0, 0);
      if (s0 + 1 < nst) iterate(s0 + 1, 1);
      if (s0 + 2 < nst) iterate(s0 + 2, 2);
    }

    // The waves' sums, over the first stage's buffer.
    static_assert(NW * NT * 1024 <= ROWS * RUN, "sums fit a stage");
    f32x4 (*red)[NT][64] = reinterpret_cast<f32x4 (*)[NT][64]>(st0);
    __syncthreads();  // every wave's last reads of the stages
#pragma unroll
    for (int c = 0; c < NT; ++c) red[wave][c][lane] = acc[c];
    __syncthreads();
    float* tp = a.t + (static_cast<int64_t>(split) * a.M + m0 + r) * adapter_tstride(a.R);
    for (int c = wave; c < NT && 16 * c < rank; c += NW) {
      f32x4 sum = red[0][c][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) sum += red[w][c][lane];
      // Result lane 16 g + r: ranks 16 c + 4 g + i of row r.
      if (mine) *reinterpret_cast<f32x4*>(tp + 16 * c + 4 * g) = sum;
    }
    __syncthreads();  // the sums are read before the next adapter's stages
  }
}

// ---- out = y + s t . Bt^T ------------------------------------------------------
// A workgroup of four waves takes a tile of 16 rows (slot s: those of the
// adapter that row s leads) and `steps` x 256 columns, a wave 64 of each 256.
// Column q of the four column blocks of a wave is matrix column 4 c + q, so
// that a lane holds four consecutive columns of a row and the loads of y and
// the stores of out are runs of 256 bytes.

// Ranks [j0, j0 + FL) of row m's t, scaled, zero past the rank.
template <typename T>
__device__ __forceinline__ void load_t(const AdapterArgs& a, int64_t m, int j0, int rank, float s,
                                       float* v) {
  constexpr int FL = Frag<T>::FL;
  const int64_t ts = adapter_tstride(a.R);
#pragma unroll
  for (int e = 0; e < FL; ++e) v[e] = 0.f;
  if (j0 >= rank) return;
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

__device__ __forceinline__ f32x4 load_y(const float* row, int64_t n, int64_t N) {
  if (n + 4 <= N) return __builtin_nontemporal_load(reinterpret_cast<const vf4u*>(row + n));
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) v[i] = row[n + i];
  return v;
}

template <typename T, int NC>
__global__ void __launch_bounds__(256) expand_kernel(AdapterArgs a, int steps) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr bool F16 = F::FL == 8;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int my = row_adapter(a, m0, lane);
  const bool in_place = a.y == a.out;
  // Bit r of `rows`: row r is written here; of `todo`: and has an adapter.
  unsigned rows = a.M - m0 >= 16 ? 0xffffu : (1u << (a.M - m0)) - 1;
  unsigned todo = static_cast<unsigned>(__ballot(my >= 0)) & 0xffffu;
  if (gridDim.z > 1) {
    const int s = blockIdx.z;
    rows &= static_cast<unsigned>(__ballot(my == __builtin_amdgcn_readlane(my, s)));
    if (rows == 0 || static_cast<int>(__builtin_ctz(rows)) != s) return;  // led by another row
    todo &= rows;
  }
  if (in_place) rows = todo;
  if (rows == 0) return;

  // t as matrix operand: lane 16 g + r holds row r.
  V hi[NC], lo[NC];
  float un[4] = {1.f, 1.f, 1.f, 1.f};  // of rows 4 g + i
  if (todo != 0) {
    int rank = 0;
    float s = 1.f, unscale = 1.f;
    if (todo >> r & 1) {
      rank = a.ranks ? a.ranks[my] : a.R;
      rank = rank < 0 ? 0 : rank > a.R ? a.R : rank;
      if (a.scales) s = a.scales[my];
    }
    float v[NC][F::FL];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_t<T>(a, m0 + r, c * F::KC + F::FL * g, rank, s, v[c]);
    if constexpr (F16) {
      // The row's largest finite |t| is moved to [2^13, 2^14): t fits an fp16
      // pair whatever its magnitude.
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(v[c][e]) < INFINITY) big = fmaxf(big, fabsf(v[c][e]));
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
#pragma unroll
      for (int i = 0; i < 4; ++i) un[i] = __shfl(unscale, 4 * g + i);
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < F::FL; ++e) hi[c][e] = v[c][e];
    }
  }

  for (int step = 0; step < steps; ++step) {
    const int64_t n0 = (static_cast<int64_t>(blockIdx.y) * steps + step) * 256 + 64 * wave;
    if (n0 >= a.N) return;
    const int64_t n = n0 + 4 * r;
    f32x4 yv[4], acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      yv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (a.y && (rows >> (4 * g + i) & 1)) yv[i] = load_y(a.y + (m0 + 4 * g + i) * a.ldy, n, a.N);
    }
    unsigned rest = todo;
    while (rest != 0) {
      const int ad = __builtin_amdgcn_readlane(my, __builtin_ctz(rest));
      const unsigned same = static_cast<unsigned>(__ballot(my == ad)) & 0xffffu;
      const int rank = rank_of(a, ad);
      const T* bb = static_cast<const T*>(a.Bt) + static_cast<int64_t>(ad) * a.N * a.R;
      f32x4 d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c * F::KC >= rank) break;
        const int j = c * F::KC + g * F::FL;
        V b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t col = n + q < a.N ? n + q : a.N - 1;
          const T* p = bb + col * a.R + j;
          b[q] = V{};
          if (a.R % F::FL == 0) {
            if (j < a.R) b[q] = *reinterpret_cast<const V*>(p);
          } else {
#pragma unroll
            for (int e = 0; e < F::FL; ++e)
              if (j + e < a.R) b[q][e] = p[e];
          }
        }
        if (c * F::KC + F::KC > rank) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < F::FL; ++e) b[q][e] = j + e < rank ? b[q][e] : static_cast<T>(0.f);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          d[q] = F::mma(hi[c], b[q], d[q]);
          if constexpr (F16) d[q] = F::mma(lo[c], b[q], d[q]);
        }
      }
      // Result lane 16 g + c: row 4 g + i, column n0 + 4 c + q in d[q][i].
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool of = same >> (4 * g + i) & 1;  // other rows' values may be anything
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = of ? d[q][i] : acc[i][q];
      }
      rest &= ~same;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(rows >> (4 * g + i) & 1)) continue;
      const f32x4 v = yv[i] + acc[i] * un[i];
      float* p = a.out + (m0 + 4 * g + i) * a.ldo + n;
      if (n + 4 <= a.N) {
        __builtin_nontemporal_store(static_cast<vf4u>(v), reinterpret_cast<vf4u*>(p));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < a.N) p[q] = v[q];
      }
    }
  }
}

template <typename T, int NT, int RUN, int NW>
void launch_stage(const AdapterArgs& a, unsigned tiles, hipStream_t st) {
  hipLaunchKernelGGL((shrink_stage_kernel<T, NT, RUN, NW>), dim3(tiles, a.S, 2), dim3(64 * NW), 0, st, a);
}

template <typename T>
hipError_t launch_typed(const AdapterArgs& a, hipStream_t st) {
  const unsigned tiles = static_cast<unsigned>((a.M + 15) / 16);
  const unsigned slots = static_cast<unsigned>(a.M < 16 ? a.M : 16);
  if (tiles >= kStageTiles && a.R <= 128) {
    if (a.R <= 16) launch_stage<T, 1, 512, 8>(a, tiles, st);
    else if (a.R <= 32) launch_stage<T, 2, 512, 8>(a, tiles, st);
    else if (a.R <= 64) launch_stage<T, 4, 256, 4>(a, tiles, st);
    else launch_stage<T, 8, 256, 4>(a, tiles, st);
  } else {
    hipLaunchKernelGGL((shrink_block_kernel<T>), dim3(tiles, a.S * ((a.R + 15) / 16), slots),
                       dim3(64 * kBlockWaves), 0, st, a);
  }
  const int steps = tiles >= 64 ? 4 : 1;
  const dim3 grid(tiles, static_cast<unsigned>((a.N + 256 * steps - 1) / (256 * steps)), tiles >= 64 ? 1 : slots);
  const int chunks = static_cast<int>((a.R + Frag<T>::KC - 1) / Frag<T>::KC);
  if (chunks <= 1) hipLaunchKernelGGL((expand_kernel<T, 1>), grid, dim3(256), 0, st, a, steps);
  else if (chunks <= 2) hipLaunchKernelGGL((expand_kernel<T, 2>), grid, dim3(256), 0, st, a, steps);
  else if (chunks <= 4) hipLaunchKernelGGL((expand_kernel<T, 4>), grid, dim3(256), 0, st, a, steps);
  else if (chunks <= 8) hipLaunchKernelGGL((expand_kernel<T, 8>), grid, dim3(256), 0, st, a, steps);
  else hipLaunchKernelGGL((expand_kernel<T, 16>), grid, dim3(256), 0, st, a, steps);
  return hipGetLastError();
}

}  // namespace

// Parts that K is split into: the staged kernel's tiles fill the chip by
// themselves; a few rows need parts, at least 256 channels each.
int adapter_splits(int64_t M, int64_t K) {
  const int64_t tiles = (M + 15) / 16;
  if (tiles >= kStageTiles) return tiles >= 256 || K < 1024 ? 1 : 2;
  const int64_t want = (128 + M - 1) / M;
  const int64_t most = (K + 255) / 256;
  const int64_t s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > 8 ? 8 : s);
}

hipError_t launch_adapter_add(const AdapterArgs& a, bool f16, hipStream_t st) {
  return f16 ? launch_typed<_Float16>(a, st) : launch_typed<float>(a, st);
}

}  // namespace w4a4
