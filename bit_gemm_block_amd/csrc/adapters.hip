// adapters.hip — low-rank adapters of many requests beside one projection:
//   out[m] = y[m] + s_a (x[m] At[a]^T) Bt[a]^T,  a = index[m].
//
// Two launches: the first writes t = x At^T, the second adds s_a t Bt^T to y.
// Sums over K that several workgroups share are written apart and joined in
// order by the second launch.  No atomics: a row's result is the same from call
// to call.
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

typedef _Float16 half4 __attribute__((ext_vector_type(4)));

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

// Bytes of a row of x from which a call of few rows takes K in kParts parts: of
// every row (more workgroups for long rows: one row, K = 14336, rank 16: 7.8 ->
// 6.9 us; 64 rows of mixed adapters 20.8 -> 15.2 us; K = 4096, rank 64: 18.0 ->
// 23.5 us), and of groups of rows (whose slots have workgroups to spare: 100 rows
// of four adapters, K = 4096, rank 32: 15.4 -> 10.0 us; K = 64: 10.3 -> 12.0 us).
constexpr int kPartsBytes = 16384;
constexpr int kGroupPartsBytes = 2048;
// Rows of one adapter in a tile up to which they are multiplied one by one.
constexpr int kRowByRow = 3;
static_assert(kParts == kRowByRow + 1 && kPartsBytes >= kGroupPartsBytes, "a group has a row for every part");
// Rows (times groups of 64 ranks) from which two tiles of 16 share the factors'
// stages: with a tile for about every compute unit, half as many wide ones move
// fewer bytes through each (x . A of 4096 rows, K = 14336, rank 64: 65.5 -> 51.3 us, rank 32: 40.5 ->
// 37.8 us; 2048 rows, rank 32: 16.7 -> 21.4 us).
constexpr int64_t kWideTileRows = 2816;
// A workgroup of x . A takes up to 64 ranks of its rows (all 256 of them in one:
// 1000 rows, K = 4096: 72.5 -> 52.2 us, 4096 rows 169 -> 157 us).  Tiles (times such
// groups of ranks) up to which it takes 32: 592 rows, K = 12224, rank 40: 30.8 -> 22.0
// us, 256 rows, K = 14336, rank 64: 33.9 -> 24.1 us; with 128 tiles, K = 4096, rank
// 64: 31.4 -> 34.0 us.
constexpr int64_t kNarrowTiles = 64;
// Workgroups up to which a tile's adapters are shared out among several of them
// (tiles of one adapter leave the others with nothing to do, and a call of one adapter
// launches them all the same: the number of adapters is not looked at).  x . A, 512 against
// 1024: 1000 rows of eight mixed adapters, K = 4096, rank 16: 24.3 against 27.2 us;
// 2048 rows of eight requests, rank 32: 24.4 against 26.0 us.  t . B, 1024 against
// 2048: 300 rows of mixed adapters, N = 2048, rank 64: 12.5 against 14.5 us, 1000
// rows, N = 4096, rank 32: 34.5 against 38.3 us; 4096 costs the larger calls more
// (2048 rows: 51 -> 60 us).
constexpr unsigned kShareStages = 512;
constexpr int64_t kShareWorkgroups = 1024;

// What the low half of a pair is moved up by (see shrink_stage_kernel).
constexpr float kLowUp = 2048.f;

// P ranks of a row of Bt from rank k on (those past R: anything of the row).
// fp32 rows of any length: whole loads need only an element's alignment.
template <typename T, int P>
__device__ __forceinline__ void load_ranks(const T* row, int k, int R, T __attribute__((ext_vector_type(P)))& b) {
  typedef T V __attribute__((ext_vector_type(P)));
  typedef V VU __attribute__((aligned(sizeof(T) == 2 ? sizeof(V) : 4)));
  if constexpr (sizeof(T) == 2) {
    b = *reinterpret_cast<const VU*>(row + (k < R ? k : 0));
  } else if (k + P <= R) {
    b = *reinterpret_cast<const VU*>(row + k);
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e) b[e] = row[k + e < R ? k + e : 0];
  }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The first row of a workgroup's tile of `rows`.  Consecutive workgroups go to the eight
// XCDs in turn (grid.x is a multiple of eight); each XCD takes a contiguous
// eighth of the tiles, so that its L2 holds the factors of the few requests there.
// The grid's padding falls past the last row.
__device__ __forceinline__ int64_t tile_row(int rows) {
  return (static_cast<int64_t>(blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3)) * rows;
}

// The adapter of row m0 + lane % rows, -1 where there is none.
__device__ __forceinline__ int row_adapter(const AdapterArgs& a, int64_t m0, int lane, int rows = 16) {
  const int64_t m = m0 + (lane & (rows - 1));
  const int v = a.index[m < a.M ? m : a.M - 1];
  return m < a.M && v >= 0 && v < a.L ? v : -1;
}

// The adapters' ranks.  Up to 64 adapters: lane l holds l's, loaded beside the
// rows' adapters rather than after them.
struct Ranks {
  int of_lane;
  __device__ __forceinline__ Ranks(const AdapterArgs& a, int lane) {
    of_lane = a.ranks && a.L <= 64 && a.L > 0 ? a.ranks[lane < a.L ? lane : a.L - 1] : a.R;
  }
  // Of a wave-uniform adapter.
  __device__ __forceinline__ int operator()(const AdapterArgs& a, int ad) const {
    const int r = a.ranks && a.L > 64 ? uniform(a.ranks[ad]) : __builtin_amdgcn_readlane(of_lane, ad);
    return r < 0 ? 0 : r > a.R ? a.R : r;
  }
};

// ---- t = x . At^T: a few rows --------------------------------------------------
// A wave's load is one run of 1 KB of a rank's row of At or of a row of x; eight
// ranks are multiplied by up to MR rows in registers, and the lanes' parts of
// the eight sums are joined by halving: in each of the first three steps the
// lanes of a pair exchange the half of the sums that the other one keeps, after
// which a lane has one sum left and joins it with seven neighbours.  Larger
// groups of rows go to the matrix instruction (eight rows at a time in vector
// registers: 8 rows, K = 14336, 25.7 -> 16.4 us, but one row 7.7 -> 9.9 us).
// What bounds it: latency, a chain of index, factors and sums (one row, K = 4096,
// rank 16: 3.9 us with its launch), and factors read once a tile: 64 rows of 32 mixed
// adapters of rank up to 64 are about 46 groups of rows of 27 adapters, which read 17 MB
// of At for 10 MB of distinct ones (8.0 us).  Four or sixteen waves share K no better
// than eight.

// Ranks j0 to j0 + 7 (those past `rank`: its last one) of adapter ad with the
// first MR rows of `rows` (its last one again, if there are fewer), over chunks
// first, first + step, ... of K: out[8 i + j] for row i.
template <typename T, int MR>
__device__ __forceinline__ void rows_dot(const AdapterArgs& a, int64_t m0, unsigned rows, int ad,
                                         int rank, int j0, int first, int step, float* out) {
  constexpr int PL = 16 / sizeof(T), CH = 64 * PL, NJ = 8;
  typedef T V __attribute__((ext_vector_type(PL)));
  const int lane = threadIdx.x & 63;
  const T* xr[MR];
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    xr[i] = static_cast<const T*>(a.x) + (m0 + __builtin_ctz(rows)) * a.ldx;
    if (rows & (rows - 1)) rows &= rows - 1;
  }
  const T* ar = static_cast<const T*>(a.At) + static_cast<int64_t>(ad) * a.R * a.K;
  float v[MR][NJ];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[i][j] = 0.f;
  for (int c = first; c * CH < a.K; c += step) {
    const int k = c * CH + lane * PL;
    if (k < a.K) {
      V av[NJ], xv[MR];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int row = j0 + j < rank ? j0 + j : rank - 1;
        av[j] = *reinterpret_cast<const V*>(ar + static_cast<int64_t>(row) * a.K + k);
      }
#pragma unroll
      for (int i = 0; i < MR; ++i) xv[i] = *reinterpret_cast<const V*>(xr[i] + k);
#pragma unroll
      for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < PL; ++e)
            v[i][j] = fmaf(static_cast<float>(xv[i][e]), static_cast<float>(av[j][e]), v[i][j]);
    }
  }
  constexpr int LPS = 64 / NJ;  // lanes with the same sum after the halving
#pragma unroll
  for (int i = 0; i < MR; ++i) {
#pragma unroll
    for (int h = 32, cnt = NJ / 2; h >= LPS; h /= 2, cnt /= 2)
#pragma unroll
      for (int j = 0; j < cnt; ++j) {
        const float keep = lane & h ? v[i][j + cnt] : v[i][j];
        const float send = lane & h ? v[i][j] : v[i][j + cnt];
        v[i][j] = keep + __shfl_xor(send, h);
      }
#pragma unroll
    for (int h = LPS / 2; h >= 1; h /= 2) v[i][0] += __shfl_xor(v[i][0], h);
    if (lane % LPS == 0) out[NJ * i + lane / LPS] = v[i][0];
  }
}

// Ranks j0 to j0 + 15 (those past `rank`: its last one) with the rows `rows` of
// the tile, a part of K, on the matrix instruction: lane 16 g + r ends up with
// ranks j0 + 4 g + i of row r.  All loads are whole and unconditional, up to
// eight chunks of them in flight: rows of other adapters read the first of
// `rows` (their results are not stored).
template <typename T>
__device__ __forceinline__ f32x4 group_dot(const AdapterArgs& a, int64_t m0, unsigned rows, int ad,
                                           int rank, int j0, int part, int parts) {
  using F = Frag<T>;
  typedef typename F::V V;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int j = j0 + r < rank ? j0 + r : rank - 1;
  const int chunks = a.K / F::KC;
  int ch = chunks * part / parts;
  const int end = chunks * (part + 1) / parts;
  const T* xr = static_cast<const T*>(a.x) + (m0 + (rows >> r & 1 ? r : __builtin_ctz(rows))) * a.ldx + g * F::FL;
  const T* ar = static_cast<const T*>(a.At) + (static_cast<int64_t>(ad) * a.R + j) * a.K + g * F::FL;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto batch = [&](auto n) {
    V xv[n.value], av[n.value];
#pragma unroll
    for (int u = 0; u < n.value; ++u) {
      av[u] = *reinterpret_cast<const V*>(ar + (ch + u) * F::KC);
      xv[u] = *reinterpret_cast<const V*>(xr + (ch + u) * F::KC);
    }
#pragma unroll
    for (int u = 0; u < n.value; ++u) acc = F::mma(av[u], xv[u], acc);
    ch += n.value;
  };
  while (ch + 8 <= end) batch(std::integral_constant<int, 8>());
  if (ch + 4 <= end) batch(std::integral_constant<int, 4>());
  while (ch < end) batch(std::integral_constant<int, 1>());
  return acc;
}

// Workgroup (eight ranks and part of K, tile, slot): slot s takes the rows of the
// adapter that row s of the tile leads, a few of them one by one.  The waves share
// the part; their sums are joined in LDS.
constexpr int kRowsWaves = 8;

template <typename T>
__global__ void __launch_bounds__(64 * kRowsWaves) shrink_rows_kernel(AdapterArgs a) {
  __shared__ f32x4 red[kRowsWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 16;
  const int s = blockIdx.z;
  const int j0 = 8 * (a.parts > 1 ? blockIdx.x / kParts : blockIdx.x);
  int p = a.parts > 1 ? blockIdx.x % kParts : 0;
  if (m0 + s >= a.M) return;
  const int my = row_adapter(a, m0, lane);
  const Ranks ranks(a, lane);
  const int ad = __builtin_amdgcn_readlane(my, s);
  if (ad < 0) return;
  unsigned rows = static_cast<unsigned>(__ballot(my == ad)) & 0xffffu;
  const bool group = __builtin_popcount(rows) > kRowByRow;
  const int before = __builtin_popcount(rows & ((1u << s) - 1));  // rows that lead row s
  const int parts = group && a.K * sizeof(T) >= kGroupPartsBytes ? kParts : a.parts;
  if (group && (j0 & 8)) return;  // groups take sixteen ranks at a time
  if (parts > a.parts)
    p = before;  // the parts of a group: its first rows' slots
  else if (before != 0)
    return;
  if (p >= parts) return;
  const int rank = ranks(a, ad);
  if (j0 >= rank) return;
  const int64_t ts = adapter_tstride(a.R);
  float* t = a.t + p * a.M * ts;
  const int first = kRowsWaves * p + wave, step = kRowsWaves * parts;
  if (group) {
    red[wave][lane] = group_dot<T>(a, m0, rows, ad, rank, j0, first, step);
    __syncthreads();
    if (wave == 0) {
      f32x4 sum = red[0][lane];
#pragma unroll
      for (int w = 1; w < kRowsWaves; ++w) sum += red[w][lane];
      if (rows >> (lane & 15) & 1)
        *reinterpret_cast<f32x4*>(t + (m0 + (lane & 15)) * ts + j0 + 4 * (lane >> 4)) = sum;
    }
    return;
  }
  float* sums = reinterpret_cast<float*>(red);  // [kRowsWaves][kRowByRow][8]
  if (__builtin_popcount(rows) == 1)
    rows_dot<T, 1>(a, m0, rows, ad, rank, j0, first, step, sums + wave * 8 * kRowByRow);
  else
    rows_dot<T, kRowByRow>(a, m0, rows, ad, rank, j0, first, step, sums + wave * 8 * kRowByRow);
  __syncthreads();
  const int j = threadIdx.x;
  for (int i = 0; rows != 0; ++i, rows &= rows - 1) {
    if (j < 8 && j0 + j < rank) {
      float sum = sums[8 * i + j];
#pragma unroll
      for (int w = 1; w < kRowsWaves; ++w) sum += sums[(w * kRowByRow + i) * 8 + j];
      t[(m0 + __builtin_ctz(rows)) * ts + j0 + j] = sum;
    }
  }
}

// ---- t = x . At^T: many rows, one adapter for most tiles ------------------------
// A workgroup owns 16 RT rows and 16 NT ranks of an adapter in them (blockIdx.y
// says which), and streams K through LDS: stage s holds RUN bytes of each of the
// 16 RT rows of x and the 16 NT rows of At, every row one contiguous run that
// direct-to-LDS copies bring in (loads of the matrix operands themselves read 16
// rows x 64 bytes per instruction, which the caches serve at a fraction of the
// rate).  Three stages are in flight.  A row's 16-byte units are stored in the
// order u ^ (row & 15), chosen by the copies' addresses, so that the reads of
// one unit of 16 rows fall in distinct banks.
// What bounds it: the copies of the workgroups that there are.  4096 rows, K = 14336,
// rank 32: 128 tiles of 32 rows, one to a compute unit, so that half of the chip brings
// 117 MB of x in 38 to 42 us (copies of x alone on the same grid take 25 to 29; tiles with
// rows of two adapters stream their rows twice, about 10 us of it).  Four and five stages,
// staggered ones and non-temporal copies of x were level or slower.
template <typename T, int RT, int NT, int RUN>
__global__ void __launch_bounds__(512) shrink_stage_kernel(AdapterArgs a) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr int NW = 8, XR = 16 * RT, ROWS = XR + 16 * NT;
  constexpr int UNITS = RUN / 16;          // 16-byte units of a row in a stage
  constexpr int RPC = 1024 / RUN;          // rows of one copy
  constexpr int CPW = ROWS / RPC / NW;     // copies per wave and stage
  constexpr int CHUNKS = RUN / 64;         // matrix operands of a stage
  constexpr int WRITTEN = NT > 2 ? NT : 2;  // t is written in whole 32 ranks
  static_assert(ROWS % (RPC * NW) == 0, "whole copies per wave");
  static_assert(UNITS >= 16 && CHUNKS % NW == 0, "units of distinct banks, whole rounds of the waves");
  static_assert(CPW < 32, "copies in flight");
  __shared__ __attribute__((aligned(16))) uint8_t st0[ROWS * RUN];
  __shared__ __attribute__((aligned(16))) uint8_t st1[ROWS * RUN];
  __shared__ __attribute__((aligned(16))) uint8_t st2[ROWS * RUN];
  auto stage = [&](int i) -> uint8_t* { return i == 0 ? st0 : i == 1 ? st1 : st2; };
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = tile_row(XR);
  if (m0 >= a.M) return;
  const int j0 = 16 * NT * blockIdx.y;
  const int bytes = a.K * static_cast<int>(sizeof(T));
  const int nst = (bytes + RUN - 1) / RUN;
  const int my = row_adapter(a, m0, lane, XR);
  const Ranks ranks(a, lane);
  constexpr unsigned ALL = static_cast<unsigned>((uint64_t{1} << XR) - 1);
  unsigned rest = static_cast<unsigned>(__ballot(my >= 0)) & ALL;
  // Pass p of the tile's adapters runs in workgroup p mod grid.z.
  for (unsigned pass = 0; rest != 0; ++pass) {
    const int ad = __builtin_amdgcn_readlane(my, __builtin_ctz(rest));
    const unsigned same = static_cast<unsigned>(__ballot(my == ad)) & ALL;
    rest &= ~same;
    if (pass % gridDim.z != blockIdx.z) continue;
    const int rank = ranks(a, ad) - j0;  // of those from j0 on
    if (rank <= 0) continue;

    // Copy q of this wave: rows RPC (wave + NW q) to + RPC - 1 of the stage.
    const uint8_t* src[CPW];
    int off[CPW];
#pragma unroll
    for (int q = 0; q < CPW; ++q) {
      const int row = RPC * (wave + NW * q) + lane / UNITS;
      off[q] = 16 * ((lane % UNITS) ^ (row & 15));
      const T* p;
      if (row < XR) {
        const int64_t m = m0 + row < a.M ? m0 + row : a.M - 1;
        p = static_cast<const T*>(a.x) + m * a.ldx;
      } else {
        const int j = row - XR < rank ? row - XR : rank - 1;
        p = static_cast<const T*>(a.At) + (static_cast<int64_t>(ad) * a.R + j0 + j) * a.K;
      }
      src[q] = reinterpret_cast<const uint8_t*>(p);
    }
    auto issue = [&](int s, uint8_t* buf) {
      const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(buf));
      const int left = bytes - s * RUN;  // past the row's end: the stage's first unit again
#pragma unroll
      for (int q = 0; q < CPW; ++q)
        dma16(src[q] + s * RUN + (off[q] < left ? off[q] : 0), b + 1024 * (wave + NW * q));
    };
    f32x4 acc[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const uint8_t* buf, int s) {
      const int valid = (bytes - s * RUN) / 64;
#pragma unroll
      for (int u = 0; u < CHUNKS / NW; ++u) {
        const int ch = u * NW + wave;
        if (ch >= valid) break;
        const int at = r * RUN + 16 * ((4 * ch + g) ^ r);
        V xv[RT], av[NT];
#pragma unroll
        for (int t = 0; t < RT; ++t) xv[t] = *reinterpret_cast<const V*>(buf + 16 * t * RUN + at);
#pragma unroll
        for (int c = 0; c < NT; ++c) av[c] = *reinterpret_cast<const V*>(buf + (XR + 16 * c) * RUN + at);
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int c = 0; c < NT; ++c) acc[t][c] = F::mma(av[c], xv[t], acc[t][c]);
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

    // The waves' sums, over the first stage's buffer, 16 rows at a time.
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      static_assert(NW * NT * 1024 <= ROWS * RUN, "sums fit a stage");
      f32x4 (*red)[NT][64] = reinterpret_cast<f32x4 (*)[NT][64]>(st0);
      __syncthreads();  // every wave's last reads of the stages
#pragma unroll
      for (int c = 0; c < NT; ++c) red[wave][c][lane] = acc[t][c];
      __syncthreads();
      // Lane 16 g + r: ranks 16 c + 4 g + i of row 16 t + r, scaled, zero past the rank.
      const bool mine = same >> (16 * t + r) & 1;
      const int64_t m = m0 + 16 * t + r;
      const float scale = a.scales ? a.scales[ad] : 1.f;
      f32x4 (*joined)[64] = reinterpret_cast<f32x4 (*)[64]>(st1);
      for (int c = wave; c < NT; c += NW) {
        f32x4 sum = red[0][c][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum += red[w][c][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = 16 * c + 4 * g + i < rank ? sum[i] * scale : 0.f;
        joined[c][lane] = sum;
      }
      __syncthreads();
      const int64_t ts = adapter_tstride(a.R);
      if constexpr (sizeof(T) == 2) {
        // t as fp16 pair, hi + 2^-11 lo: the row's largest finite |t| here is moved
        // to [2^13, 2^14), and what hi leaves, at most 2^-11 of the value, up by
        // 2^11, so that it meets fp16's subnormal numbers no earlier than the value
        // itself does.  Every t keeps 22 bits down to 2^-27 of the row's largest,
        // smaller ones an error of 2^-49 of it or less.  (Under one power of two for
        // both halves a t 2^-21 of the largest kept 18 bits.)
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = fabsf(joined[c][lane][i]);
            big = fmaxf(big, v < INFINITY ? v : 0.f);
          }
        big = fmaxf(big, __shfl_xor(big, 16));
        big = fmaxf(big, __shfl_xor(big, 32));
        int e = 0;
        if (big > 0.f) {
          (void)frexpf(big, &e);  // big = f 2^e, f in [1/2, 1)
          e = 14 - e;
          e = e > 120 ? 120 : e;
        }
        _Float16* hi = reinterpret_cast<_Float16*>(a.t) + m * ts + j0 + 4 * g;
        for (int c = wave; c < WRITTEN && j0 + 16 * c < ts; c += NW) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          if (c < NT) v = joined[c][lane];
          half4 h, l;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = ldexpf(v[i], e);
            h[i] = static_cast<_Float16>(u);
            const float d = u - static_cast<float>(h[i]);
            l[i] = static_cast<_Float16>(fabsf(u) < INFINITY ? kLowUp * d : 0.f);
          }
          if (mine) {
            *reinterpret_cast<half4*>(hi + 16 * c) = h;
            *reinterpret_cast<half4*>(hi + a.M * ts + 16 * c) = l;
          }
        }
        if (mine && wave == 0 && 32 * g < 16 * WRITTEN && j0 + 32 * g < ts)
          a.t[a.M * ts + (j0 / 32 + g) * adapter_urows(a.M) + m] = ldexpf(1.f, -e);
      } else {
        float* tp = a.t + m * ts + j0 + 4 * g;
        for (int c = wave; c < WRITTEN && j0 + 16 * c < ts; c += NW) {
          f32x4 v = {0.f, 0.f, 0.f, 0.f};
          if (c < NT) v = joined[c][lane];
          if (mine) *reinterpret_cast<f32x4*>(tp + 16 * c) = v;
        }
      }
    }
    __syncthreads();  // the sums are read before the next adapter's stages
  }
}

// Four consecutive columns of a row, those past its end left alone.  y and out
// pass once.
__device__ __forceinline__ f32x4 load_y(const float* row, int64_t n, int64_t N) {
  if (n + 4 <= N) return __builtin_nontemporal_load(reinterpret_cast<const vf4u*>(row + n));
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < N) v[i] = row[n + i];
  return v;
}
__device__ __forceinline__ void store_out(float* row, int64_t n, int64_t N, f32x4 v) {
  if (n + 4 <= N) {
    __builtin_nontemporal_store(static_cast<vf4u>(v), reinterpret_cast<vf4u*>(row + n));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) row[n + i] = v[i];
  }
}

// ---- out = y + s t . Bt^T: a row at a time -------------------------------------
// For rows that share their adapter with few others the matrix instruction
// would multiply mostly zeros.  Here LPC lanes take a column: each holds PL
// (16 bytes) of its ranks, so that a wave's load is one run of 1 KB of Bt, eight
// of them in flight.  The dot products' parts are joined by halving: in
// every step the lanes of a pair exchange the half of their columns that the
// other one keeps, and a lane ends up with one column (or more, where LPC < 8).
// What bounds it: latency up to a few MB (one row, N = 4096, rank 16: 3.9 us with its
// launch), then the loads of Bt, which a group of rows reads for itself in every tile,
// to the call's rank (64 rows of 32 mixed adapters of rank up to 64, N = 6144: 10.3 us
// for 35 to 40 MB of loads, of which 15 MB are distinct and within the ranks).

// Columns [n0, n0 + 512 / LPC) of rows of adapter ad (or of none: ad < 0), by one
// wave.
template <typename T, int LPC>
struct RowProducts {
  static constexpr int PL = 16 / sizeof(T), CPI = 64 / LPC, NI = 8;
  static constexpr int KEEP = LPC < NI ? NI / LPC : 1;  // columns of a lane at the end
  typedef T V __attribute__((ext_vector_type(PL)));
  V b[NI];
  float scale = 1.f;
  int ad, rank, sub, j0;
  int64_t n;  // the lane's columns at the end: n + CPI i, i < KEEP
  bool last = true;  // of the lanes that hold the same column, the one that stores it

  __device__ __forceinline__ RowProducts(const AdapterArgs& a, int ad_, int rank_, int64_t n0)
      : ad(ad_), rank(rank_) {
    const int lane = threadIdx.x & 63;
    const int grp = lane / LPC;
    sub = lane % LPC;
    j0 = sub * PL;
    if (ad >= 0) {
      const T* bb = static_cast<const T*>(a.Bt) + (static_cast<int64_t>(ad) * a.N + n0) * a.R;
      const int most = a.N - n0 < 512 ? static_cast<int>(a.N - n0) - 1 : 511;  // last column from n0 on
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int col = i * CPI + grp < most ? i * CPI + grp : most;
        const T* p = bb + col * a.R;
        load_ranks<T, PL>(p, j0, a.R, b[i]);
      }
      if (a.scales) scale = a.scales[ad];
    }
    int first = 0;
#pragma unroll
    for (int h = LPC / 2, cnt = NI; h >= 1; h /= 2) {
      if (cnt > 1) {
        cnt /= 2;
        if (sub & h) first += cnt;
      } else if (sub & h) {
        last = false;
      }
    }
    n = n0 + CPI * first + grp;
  }
  // Zeroes what lies past the rank (anything), word by word.
  __device__ __forceinline__ void mask() {
    if (rank >= PL * LPC) return;
    constexpr int EPW = 4 / sizeof(T);
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int left = rank - (j0 + w * EPW);  // elements of this word that count
      const uint32_t keep = left >= EPW ? ~0u : left == 1 ? 0xffffu : 0u;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        Words v = __builtin_bit_cast(Words, b[i]);
        v[w] &= keep;
        b[i] = __builtin_bit_cast(V, v);
      }
    }
  }
  // Row m; get(e): t of the lane's rank e, before the scale (past the rank: anything).
  template <typename Get>
  __device__ __forceinline__ void row(const AdapterArgs& a, int64_t m, Get get) const {
    float y[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) y[i] = a.y && n + CPI * i < a.N ? a.y[m * a.ldy + n + CPI * i] : 0.f;
    float v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = 0.f;
    if (rank > 0) {
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const float t = j0 + e < rank ? get(e) * scale : 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) v[i] = fmaf(t, static_cast<float>(b[i][e]), v[i]);
      }
#pragma unroll
      for (int h = LPC / 2, cnt = NI; h >= 1; h /= 2) {
        if (cnt > 1) {
          cnt /= 2;
#pragma unroll
          for (int i = 0; i < cnt; ++i) {
            const float keep = sub & h ? v[i + cnt] : v[i];
            const float send = sub & h ? v[i] : v[i + cnt];
            v[i] = keep + __shfl_xor(send, h);
          }
        } else {
          v[0] += __shfl_xor(v[0], h);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (last && n + CPI * i < a.N) a.out[m * a.ldo + n + CPI * i] = y[i] + v[i];
  }
};

// Four of a row's t, from `at` on: of the sum of kParts parts, or as it is.
__device__ __forceinline__ f32x4 load_t(const AdapterArgs& a, const float* at, int64_t ts, bool parts) {
  f32x4 t = *reinterpret_cast<const f32x4*>(at);
  if (parts) {
    f32x4 p[kParts - 1];
#pragma unroll
    for (int i = 0; i < kParts - 1; ++i) p[i] = *reinterpret_cast<const f32x4*>(at + (i + 1) * a.M * ts);
#pragma unroll
    for (int i = 0; i < kParts - 1; ++i) t += p[i];
  }
  return t;
}

// The same rows, 64 columns from n0, by one wave with the float32 matrix
// instruction, t as it is (for groups of rows; about eight times the price of
// the fp16 pair per product, which few rows do not notice).
template <typename T, int RC>
__device__ __forceinline__ void group_pass(const AdapterArgs& a, int64_t m0, unsigned rows, int ad,
                                           int rank, int64_t n0) {
  constexpr int PL = sizeof(T) == 2 && RC > 16 ? 8 : 4;  // ranks of a lane in a chunk
  constexpr int KC = 4 * PL;
  typedef T V __attribute__((ext_vector_type(PL)));
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n = n0 + 4 * r, ts = adapter_tstride(a.R);
  const bool parts = a.K * sizeof(T) >= kGroupPartsBytes;
  f32x4 yv[4], d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    yv[i] = d[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.y && (rows >> (4 * g + i) & 1)) yv[i] = load_y(a.y + (m0 + 4 * g + i) * a.ldy, n, a.N);
  }
  if (ad >= 0) {
    const T* bb = static_cast<const T*>(a.Bt) + static_cast<int64_t>(ad) * a.N * a.R;
    const float* tp = a.t + (m0 + (rows >> r & 1 ? r : __builtin_ctz(rows))) * ts;
    const float scale = a.scales ? a.scales[ad] : 1.f;
#pragma unroll 1
    for (int c = 0; c * KC < rank; ++c) {
      const int k = c * KC + PL * g, at = k < a.R ? k : 0;
      V b[4];
      f32x4 w[PL / 4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const T* p = bb + (n + q < a.N ? n + q : a.N - 1) * a.R;
        load_ranks<T, PL>(p, k, a.R, b[q]);
      }
#pragma unroll
      for (int e = 0; e < PL / 4; ++e) w[e] = load_t(a, tp + at + 4 * e, ts, parts);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const float t = k + e < rank ? w[e / 4][e % 4] * scale : 0.f;  // past the rank: anything
#pragma unroll
        for (int q = 0; q < 4; ++q)
          d[q] = __builtin_amdgcn_mfma_f32_16x16x4f32(t, k + e < rank ? static_cast<float>(b[q][e]) : 0.f,
                                                      d[q], 0, 0, 0);
      }
    }
  }
  // Result lane 16 g + c: row 4 g + i, column n0 + 4 c + q in d[q][i].
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (rows >> (4 * g + i) & 1)
      store_out(a.out + (m0 + 4 * g + i) * a.ldo, n, a.N, yv[i] + f32x4{d[0][i], d[1][i], d[2][i], d[3][i]});
}

// Workgroup (4 x 512 / LPC columns, tile, slot): slot s takes the rows of the
// adapter that row s of the tile leads, a few of them one by one.  Larger groups
// share their columns, 256 at a time, among their rows' slots (100 rows of four
// adapters, K = 4096, N = 6144, rank 16: 22.1 -> 14.5 us).
template <typename T, int RC>
__global__ void __launch_bounds__(256) expand_rows_kernel(AdapterArgs a) {
  constexpr int LPC = RC * static_cast<int>(sizeof(T)) / 16, COLS = 4 * 512 / LPC;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 16;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * COLS;
  const int my = row_adapter(a, m0, lane);
  const Ranks ranks(a, lane);
  const int s = blockIdx.z;
  if (m0 + s >= a.M) return;
  const int ad = __builtin_amdgcn_readlane(my, s);
  unsigned rows = static_cast<unsigned>(__ballot(my == ad)) & 0xffffu;
  if (a.M - m0 < 16) rows &= (1u << (a.M - m0)) - 1;
  if (ad < 0 && a.y == a.out) return;  // in place, nothing to add
  const int rank = ad < 0 ? 0 : ranks(a, ad);
  const int count = __builtin_popcount(rows);
  const int before = __builtin_popcount(rows & ((1u << s) - 1));  // rows that lead row s
  if (count <= kRowByRow) {
    if (before != 0) return;
    const int64_t n = n0 + wave * (COLS / 4);
    if (n >= a.N) return;
    RowProducts<T, LPC> p(a, ad, rank, n);
    const int64_t ts = adapter_tstride(a.R);
    p.mask();
    for (; rows != 0; rows &= rows - 1) {
      const int64_t m = m0 + __builtin_ctz(rows);
      f32x4 t[p.PL / 4];
#pragma unroll
      for (int e = 0; e < p.PL / 4; ++e)
        t[e] = load_t(a, a.t + m * ts + (p.j0 < a.R ? p.j0 : 0) + 4 * e, ts, a.parts > 1);
      p.row(a, m, [&](int e) { return t[e / 4][e % 4]; });
    }
  } else {
    for (int64_t n = n0 + 256 * before + 64 * wave; n < n0 + COLS && n < a.N; n += 256 * count)
      group_pass<T, RC>(a, m0, rows, ad, rank, n);
  }
}

// ---- out = y + s t . Bt^T: many rows -------------------------------------------
// A workgroup of four waves takes 16 rows and 256 columns, a wave 64 of them;
// t comes ready as matrix operand (fp16: the pair, a product each, as the halves
// have powers of two of their own).  Column q of a wave's four column
// blocks is matrix column 4 c + q, so that a lane holds four consecutive columns
// of a row and the loads of y and the stores of out are runs of 256 bytes.
// Each wave brings its columns of Bt into its own part of LDS with direct copies,
// 128 bytes of every column at a time: matrix operands put neighbouring lanes
// into different columns, and loaded from memory as they are, each of a load's 64
// pieces of 16 bytes is a line of its own (2048 x 64 -> 28672 of 16 mixed adapters
// of rank 16: 325 -> 188 us; 4096 x 4096 -> 4096, one adapter in most tiles, rank
// 16 / 64 / 256: 40.6 / 58.1 / 209 -> 37.5 / 50.2 / 170 us).  Column 4 r + q lies
// at row 16 q + r, its units in the order u ^ r, so that an operand's reads fall in
// distinct banks.  No barriers: a wave waits for its own copies.
// What bounds it: y and out (4096 x 28672, rank 16: 940 MB in 165 to 188 us);
// with ranks of 64 and more the passes of Bt through the L2, one for every 16 rows
// (4096 x 4096 -> 4096: 36 us at rank 64, 117 us at rank 256).  Blocks of 64 rows and
// float32 products were slower (266 and 218 us where this kernel's first form took
// 191).
// RC: the ranks, rounded up (16, 32, ... 256).  SHARED: pass p of the tile's adapters
// runs in workgroup p mod grid.z, which then loads y for its rows only.
// Waves a SIMD whose registers a kernel keeps within: fp16 of rank 64 four (512 x 4096
// -> 4096: 18.2 -> 16.9 us), of rank 16 five (4096 x 4096 -> 28672: 202 -> 197 us); the
// other widths are within the next lower or far above.  fp32 is left alone: held to
// four waves, rank 64 kept about fifty registers in memory (4096 x 1024 -> 14336: 345
// against 203 us, 512 x 4096 -> 4096: 42.7 against 32.7 us).
template <typename T, int RC>
constexpr int kWaves = sizeof(T) != 2 ? 1 : RC == 16 ? 5 : RC == 64 ? 4 : 1;
template <typename T, int RC, bool SHARED>
__global__ void __launch_bounds__(256, (kWaves<T, RC>)) expand_many_kernel(AdapterArgs a) {
  using F = Frag<T>;
  typedef typename F::V V;
  constexpr bool F16 = sizeof(T) == 2;
  // One load brings hi as ranks 0 .. 15 of an operand and lo as 16 .. 31.
  constexpr bool BOTH = F16 && RC == 16;
  constexpr int NC = BOTH ? 1 : RC / F::KC;
  // A stage: RS ranks (UNITS units of 16 bytes, CS operands) of a wave's columns.
  constexpr int ROW = RC * static_cast<int>(sizeof(T)), UNITS = ROW < 128 ? ROW / 16 : 8;
  constexpr int RS = UNITS * 16 / static_cast<int>(sizeof(T)), CS = BOTH ? 1 : UNITS / 4;
  __shared__ __attribute__((aligned(16))) uint8_t staged[4 * 64 * 16 * UNITS];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = tile_row(16);
  const int64_t n0 = static_cast<int64_t>(blockIdx.y) * 256 + 64 * wave;
  if (m0 >= a.M || n0 >= a.N) return;
  const int64_t n = n0 + 4 * r;
  const int64_t ts = adapter_tstride(a.R);
  const uint32_t own = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(staged)) + 1024 * UNITS * wave;
  // Bit r of `rows`: row r is written here; of `todo`: and has an adapter.
  unsigned rows = a.M - m0 >= 16 ? 0xffffu : (1u << (a.M - m0)) - 1;

  f32x4 yv[4];
  auto load_rows = [&](unsigned of) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      yv[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (a.y && (of >> (4 * g + i) & 1)) yv[i] = load_y(a.y + (m0 + 4 * g + i) * a.ldy, n, a.N);
    }
  };
  if constexpr (!SHARED) load_rows(rows);
  // Row r's t (of a row without an adapter: anything, and not used).
  V hi[NC], lo[NC];
  const int64_t mt = m0 + r < a.M ? m0 + r : a.M - 1;
  const int j = BOTH ? 8 * (g & 1) : F::FL * g;  // the lane's first rank in a chunk
  const T* tp = reinterpret_cast<const T*>(a.t) + mt * ts + j;
  if constexpr (BOTH) {
    const V v = *reinterpret_cast<const V*>(tp + (g >> 1) * a.M * ts), zero = {};
    hi[0] = g < 2 ? v : zero;
    lo[0] = g < 2 ? zero : v;
  } else {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = c * F::KC < a.R ? c * F::KC : 0;
      hi[c] = *reinterpret_cast<const V*>(tp + at);
      if constexpr (F16) lo[c] = *reinterpret_cast<const V*>(tp + a.M * ts + at);
    }
  }
  f32x4 un[F16 ? NC : 1];
  if constexpr (F16) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      un[c] = *reinterpret_cast<const f32x4*>(a.t + a.M * ts + (32 * c < ts ? c : 0) * adapter_urows(a.M) + m0 + 4 * g);
  }
  const int my = row_adapter(a, m0, lane);
  const Ranks ranks(a, lane);
  const unsigned todo = static_cast<unsigned>(__ballot(my >= 0)) & 0xffffu;
  unsigned mine = todo;  // the rows that are multiplied here
  if constexpr (SHARED) {
    mine = 0;
    unsigned pass = 0;
    for (unsigned rest = todo; rest != 0; ++pass) {
      const unsigned same =
          static_cast<unsigned>(__ballot(my == __builtin_amdgcn_readlane(my, __builtin_ctz(rest)))) & 0xffffu;
      if (pass % gridDim.z == blockIdx.z) mine |= same;
      rest &= ~same;
    }
    rows = mine | (blockIdx.z == 0 ? rows & ~todo : 0);
  }
  if (a.y == a.out) rows = mine;
  if (rows == 0) return;
  if constexpr (SHARED) load_rows(rows);

  f32x4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (unsigned rest = mine; rest != 0;) {
    const int ad = __builtin_amdgcn_readlane(my, __builtin_ctz(rest));
    const unsigned same = static_cast<unsigned>(__ballot(my == ad)) & 0xffffu;
    const T* bb = static_cast<const T*>(a.Bt) + static_cast<int64_t>(ad) * a.N * a.R;
    const int rank = ranks(a, ad);
    rest &= ~same;
    if (rank == 0) continue;  // t was not written
    f32x4 sum[4];  // of the adapter's rows; the other rows' may be anything
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Chunk c's operands b: what lies past the rank may be anything.
    auto multiply = [&](int c, V(&b)[4]) {
      if (c * F::KC + (BOTH ? 16 : F::KC) > rank) {
        const int k = c * F::KC + j;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < F::FL; ++e) b[q][e] = k + e < rank ? b[q][e] : static_cast<T>(0.f);
      }
      f32x4 d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        d[q] = F::mma(hi[c], b[q], f32x4{0.f, 0.f, 0.f, 0.f});
        if constexpr (F16) {
          const f32x4 low = F::mma(lo[c], b[q], f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
          for (int i = 0; i < 4; ++i) d[q][i] = fmaf(low[i], 1.f / kLowUp, d[q][i]);
        }
      }
      // Result lane 16 g + c: row 4 g + i, column n0 + 4 c + q in d[q][i].
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sum[i][q] = F16 ? fmaf(d[q][i], un[F16 ? c : 0][i], sum[i][q]) : sum[i][q] + d[q][i];
    };
    if (F16 || a.R % F::FL == 0) {
#pragma unroll
      for (int h = 0; h < RC / RS; ++h) {
        if (RS * h >= rank) break;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last reads of the stage have returned
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
          const int row = (64 * i + lane) / UNITS, u = (lane % UNITS) ^ (row & (UNITS - 1));
          const int64_t col = n0 + 4 * (row & 15) + (row >> 4);
          const int k = RS * h + F::FL * u;
          dma16(reinterpret_cast<const uint8_t*>(bb + (col < a.N ? col : a.N - 1) * a.R + (k < a.R ? k : 0)), own + 1024 * i);
        }
        wait_vmcnt<0>();
#pragma unroll
        for (int c = CS * h; c < CS * (h + 1); ++c) {
          if (c * F::KC >= rank) break;
          V b[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int u = BOTH ? g & 1 : 4 * (c % CS) + g;
            b[q] = *reinterpret_cast<const V*>(staged + 1024 * UNITS * wave + 16 * (UNITS * (16 * q + r) + (u ^ (r & (UNITS - 1)))));
          }
          multiply(c, b);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c * F::KC >= rank) break;
        V b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          load_ranks<T, F::FL>(bb + (n + q < a.N ? n + q : a.N - 1) * a.R, c * F::KC + j, a.R, b[q]);
        multiply(c, b);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (same >> (4 * g + i) & 1) acc[i] = sum[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!(rows >> (4 * g + i) & 1)) continue;
    store_out(a.out + (m0 + 4 * g + i) * a.ldo, n, a.N, yv[i] + acc[i]);
  }
}

template <typename T, int RT, int NT, int RUN>
void launch_stage(const AdapterArgs& a, hipStream_t st) {
  const unsigned gx = static_cast<unsigned>(((a.M + 16 * RT - 1) / (16 * RT) + 7) / 8 * 8);
  const unsigned gy = static_cast<unsigned>((a.R + 16 * NT - 1) / (16 * NT));
  const unsigned share = kShareStages / (gx * gy);
  hipLaunchKernelGGL((shrink_stage_kernel<T, RT, NT, RUN>),
                     dim3(gx, gy, share < 2 ? 2 : share > 16 ? 16 : share), dim3(512), 0, st, a);
}

// Up to rank 32 three stages of 512 bytes a row leave room for a second workgroup
// on a compute unit; where there is no second one (few tiles), the double run
// halves the stages' latencies (512 rows, K = 14336, rank 16: 25.0 -> 20.9 us; 4096
// rows, rank 32: 74.8 -> 78.1 us).
template <typename T, int RC>
void launch_shrink(const AdapterArgs& a, hipStream_t st) {
  const int64_t tiles = (a.M + 15) / 16;
  if constexpr (RC <= 32) {
    if (a.M <= 16 * 128) return launch_stage<T, 1, RC / 16, 1024>(a, st);
    if constexpr (RC == 32) {
      if (a.M >= kWideTileRows) return launch_stage<T, 2, 2, 512>(a, st);
    }
    launch_stage<T, 1, RC / 16, 512>(a, st);
  } else {
    const int64_t groups = (a.R + 63) / 64;
    if (a.M * groups >= kWideTileRows) launch_stage<T, 2, 4, 512>(a, st);
    else if (tiles * groups <= kNarrowTiles) launch_stage<T, 1, 2, 1024>(a, st);
    else launch_stage<T, 1, 4, 512>(a, st);
  }
}

template <typename T, int RC>
void launch_rank(const AdapterArgs& a, hipStream_t st) {
  const unsigned tiles = static_cast<unsigned>((a.M + 15) / 16);
  if (a.M >= kManyRows) {
    launch_shrink<T, RC>(a, st);
    const unsigned gx = (tiles + 7) / 8 * 8;
    const unsigned gy = static_cast<unsigned>((a.N + 255) / 256);
    const int64_t share = kShareWorkgroups / (static_cast<int64_t>(gx) * gy);
    if (share <= 1)
      hipLaunchKernelGGL((expand_many_kernel<T, RC, false>), dim3(gx, gy), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((expand_many_kernel<T, RC, true>),
                         dim3(gx, gy, static_cast<unsigned>(share < 16 ? share : 16)), dim3(256), 0, st, a);
    return;
  }
  constexpr int WAVE_COLS = 512 * 16 / (RC * static_cast<int>(sizeof(T)));
  const unsigned slots = static_cast<unsigned>(a.M < 16 ? a.M : 16);
  hipLaunchKernelGGL((shrink_rows_kernel<T>), dim3(static_cast<unsigned>((a.R + 7) / 8 * a.parts), tiles, slots),
                     dim3(64 * kRowsWaves), 0, st, a);
  constexpr int COLS = 4 * WAVE_COLS;
  hipLaunchKernelGGL((expand_rows_kernel<T, RC>), dim3(static_cast<unsigned>((a.N + COLS - 1) / COLS), tiles, slots),
                     dim3(256), 0, st, a);
}

template <typename T>
hipError_t launch_typed(const AdapterArgs& a, hipStream_t st) {
  if (a.R <= 16) launch_rank<T, 16>(a, st);
  else if (a.R <= 32) launch_rank<T, 32>(a, st);
  else if (a.R <= 64) launch_rank<T, 64>(a, st);
  else if (a.R <= 128) launch_rank<T, 128>(a, st);
  else launch_rank<T, 256>(a, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_add(const AdapterArgs& a, bool f16, hipStream_t st) {
  AdapterArgs b = a;
  b.parts = a.M < kManyRows && a.K * (f16 ? 2 : 4) >= kPartsBytes ? kParts : 1;
  return f16 ? launch_typed<_Float16>(b, st) : launch_typed<float>(b, st);
}

}  // namespace w4a4
