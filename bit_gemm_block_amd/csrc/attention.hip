// attention.hip — how a call of the attention over the quantized cache is cut,
// and the joining of its parts.
//
// Where there are few rows, their tokens (a sequence's own, and the prefix) are
// shared among workgroups (attention_kernel.h).  Each leaves (ref, l, O) with
// p = 2^(t - ref) summed to l and p v to O, in float32;
//   out = sum_i 2^(ref_i - M) O_i / sum_i 2^(ref_i - M) l_i,  M = max ref_i,
// taken in the order of the tokens, the prefix last.
//
// The lengths are on the device.  For few rows the workgroups add them up and
// take equal runs; for many the host cuts by the tables' capacity and the rows
// there can be, and a workgroup whose sequence is shorter, or has fewer rows, ends
// at once.
#include "attention_kernel.h"

namespace w4a4 {
namespace {

constexpr int64_t kGrid = 1 << 24;   // workgroups of 256 threads: below 2^32 threads

// rows: of a sequence, at most; all: of the call.  `beside`: a prefix whose
// workgroups run beside those of the own tokens.
AttentionCut cut_tokens(int64_t rows, int64_t all, int64_t seqs, int64_t heads, int64_t capacity, int D, bool beside) {
  AttentionCut c{};
  // One tile of rows: waves share it and take tokens each (16 rows of 64 sequences
  // of up to 1024 tokens: 28.7 us, by rows 32.3; of 16 up to 2048: 19.5, 31.0).
  // More: waves share the tokens and take rows each (32 rows: 38.1 us, with two
  // tiles to every wave and tokens shared out 50.4; 32.6 and 31.6).
  c.rowsplit = rows > 16;
  if (seqs < 1) seqs = 1;
  const int64_t resident = 256 * (D == 256 ? 2 : 3);  // workgroups that fit the chip
  // Few rows: pieces of 256 tokens, two steps for each wave of a workgroup (64
  // sequences of 300 to 16384 tokens: 127 us, with 128 tokens 134, with 512 131).
  if (!c.rowsplit) {
    c.piece_log2 = 8;
    while ((seqs * capacity >> c.piece_log2) >= int64_t{1} << 30) ++c.piece_log2;
    const int64_t pieces = seqs * (capacity > 0 ? ((capacity - 1) >> c.piece_log2) + 1 : 1);
    int64_t groups = (resident + heads - 1) / heads;
    c.one_piece = groups >= pieces;
    groups = groups < pieces ? groups : pieces;
    c.groups = Divisor(static_cast<uint32_t>(groups));
    return c;
  }
  const int64_t groups = (rows + kGroupRows - 1) / kGroupRows;
  c.groups = Divisor(static_cast<uint32_t>(groups));
  // Rows' workgroups cost their queries' operands and a partial result each, so
  // parts are long (1024 tokens; 3 prompts of 1021 queries: 98 us, with 512 113,
  // with 2048 101), unless there are too few of them for the chip (256 tokens).
  // Then there are parts until the workgroups that fit at once are there (one
  // prompt of 512 queries behind 8192 tokens: 153 us with 768, 199 with 256; 44
  // drafts of 7 behind up to 4474: 24 and 41), but for a prefix only one to a
  // compute unit, since own tokens share the chip (64 sequences on a prefix of
  // 8192: 38 us with 256, 45 with 512, 50 with 1024).
  // And there are fewer parts the more row groups there are, down to one, so that
  // partial results are bounded by the chip and not by the queries: eight rounds of
  // what fits at once (a prompt of 8192 queries, 8 heads x 4 of 128: 806 us without
  // any, with 8 parts 1270 and 1.1 GB; of 4096 307, 342; 63 single queries of up to
  // 16384 tokens beside 2048 492, 440, beside 512 295, 290; with four rounds 96
  // sequences of group 20, one of 9000 tokens, 87 for 59).
  const int64_t units = seqs * heads * groups, through = all / kGroupRows + seqs;
  if (through < seqs * groups && through < kGrid) c.places = static_cast<int>(through);
  c.piece_log2 = units < 256 ? 8 : 10;
  int64_t parts = units < resident ? ((beside ? 256 : resident) + units - 1) / units : 8;
  const int64_t most = least64(capacity >> c.piece_log2, 8 * resident / (c.places ? heads * c.places : units));
  parts = parts < most ? parts : most;
  c.parts = Divisor(static_cast<uint32_t>(parts < 1 ? 1 : parts));
  return c;
}

// A row's partial results: of its own tokens and of the prefix.
struct Parts {
  int own, n, own_first, front_first;
  int64_t token;
  int query, head;
};
// False where the row has nothing to join: no such query, or stored at once.
__device__ __forceinline__ bool parts_of_row(const AttentionArgs& a, const AttentionPlan& plan, const Partial& partial,
                                             uint32_t id, Parts* p) {
  const uint32_t at = id / static_cast<uint32_t>(a.q_heads);
  p->head = id - at * a.q_heads;
  const int s = plan.join_by_place ? at / static_cast<uint32_t>(a.max_q)
                                   : first_above(a, at, [](int, int q) { return q; });
  if (s >= a.seqs) return false;
  const Span span = own_span(a, s);
  p->query = at - (plan.join_by_place ? s * a.max_q : span.first);
  if (p->query < 0 || p->query >= span.n || p->query >= a.max_q) return false;
  p->own_first = partial.slots(a, s)[0];
  p->own = p->n = partial.slots(a, s)[1];
  p->front_first = 0;
  if (a.prefix_table) {
    p->front_first = partial.slots(a, a.seqs)[0];
    p->n += partial.slots(a, a.seqs)[1];
  } else if (p->own == 1) {
    return false;
  }
  p->token = span.first + p->query;
  return true;
}
__device__ __forceinline__ int64_t row_of(const AttentionArgs& a, const AttentionPlan& plan, const Partial& partial,
                                          const Parts& p, int k) {
  const bool front = k >= p.own;
  return partial.row(a, plan, front, front ? p.front_first + k - p.own : p.own_first + k, p.token, p.query, p.head);
}
__device__ __forceinline__ void store_joined(const AttentionArgs& a, const Parts& p, int c, f4 o) {
  const int64_t to = p.token * a.ldo + static_cast<int64_t>(p.head) * a.D + c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.out_f16)
      static_cast<_Float16*>(a.out)[to + e] = static_cast<_Float16>(o[e]);
    else
      static_cast<float*>(a.out)[to + e] = o[e];
  }
}

// Many rows: one to a wave, D / 4 lanes to a part, the parts of 64 at a time.
template <int D>
__global__ void __launch_bounds__(256) attention_join_rows_kernel(AttentionArgs a, AttentionPlan plan, uint32_t rows) {
  constexpr int kLanes = D / 4, kGroups = 64 / kLanes;
  const uint32_t id = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (id >= rows) return;
  const Partial partial(a, plan);
  Parts p;
  if (!parts_of_row(a, plan, partial, id, &p)) return;
  const int c = lane % kLanes, grp = lane / kLanes;
  f4 o = {0.f, 0.f, 0.f, 0.f};
  float top = kUnset, sum = 0.f;
  for (int base = 0; base < p.n; base += 64) {
    const int here = p.n - base < 64 ? p.n - base : 64;
    float ref = kUnset, l = 0.f;
    if (lane < here) {
      const float* st = partial.stat(a, row_of(a, plan, partial, p, base + lane));
      ref = st[0];
      l = st[1];
    }
    float m = fmaxf(top, ref);
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor(m, w));
    const Lower before(m - top), mine(m - ref);
    top = m;
    const float f = lane < here ? mine.factor() : 0.f;
    float add = mine.sum(l);
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) add += __shfl_xor(add, w);
    sum = before.sum(sum) + add;
    o *= before.factor();
#pragma unroll 4
    for (int k = 0; k < here; k += kGroups) {
      const int at = k + grp < here ? k + grp : here - 1;
      const f4 v = *reinterpret_cast<const f4*>(partial.o(a, row_of(a, plan, partial, p, base + at)) + 4 * c);
      const float weight = __shfl(f, at);  // by all lanes: one that is switched off gives none
      o += (k + grp < here ? weight : 0.f) * v;
    }
  }
#pragma unroll
  for (int w = kLanes; w < 64; w <<= 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], w);
  }
  o *= sum == 0.f ? 0.f : 1.f / sum;
  if (grp == 0) store_joined(a, p, 4 * c, o);
}

// Few rows of many parts: 32 channels of a row to a workgroup, eight lanes to a
// part, the parts of 256 at a time.
template <int D>
__global__ void __launch_bounds__(256) attention_join_parts_kernel(AttentionArgs a, AttentionPlan plan) {
  __shared__ float weight[256];
  __shared__ float red[8];
  __shared__ f4 lds[4][8];
  const uint32_t id = blockIdx.x / (D / 32);
  const Partial partial(a, plan);
  Parts p;
  if (!parts_of_row(a, plan, partial, id, &p)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = static_cast<int>(blockIdx.x % (D / 32)) * 32 + 4 * (threadIdx.x & 7), grp = threadIdx.x >> 3;
  f4 o = {0.f, 0.f, 0.f, 0.f};
  float top = kUnset, sum = 0.f;
  for (int base = 0; base < p.n; base += 256) {
    const int here = p.n - base < 256 ? p.n - base : 256;
    float ref = kUnset, l = 0.f;
    if (static_cast<int>(threadIdx.x) < here) {
      const float* st = partial.stat(a, row_of(a, plan, partial, p, base + threadIdx.x));
      ref = st[0];
      l = st[1];
    }
    float m = fmaxf(top, ref);
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor(m, w));
    if (lane == 0) red[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const Lower before(m - top), mine(m - ref);
    top = m;
    weight[threadIdx.x] = static_cast<int>(threadIdx.x) < here ? mine.factor() : 0.f;
    float add = mine.sum(l);
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) add += __shfl_xor(add, w);
    if (lane == 0) red[4 + wave] = add;
    __syncthreads();
    sum = before.sum(sum) + ((red[4] + red[5]) + (red[6] + red[7]));
    o *= before.factor();
#pragma unroll 4
    for (int k = grp; k < here; k += 32)
      o += weight[k] * *reinterpret_cast<const f4*>(partial.o(a, row_of(a, plan, partial, p, base + k)) + c);
    __syncthreads();
  }
#pragma unroll
  for (int w = 8; w < 64; w <<= 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], w);
  }
  if (lane < 8) lds[wave][lane] = o;
  __syncthreads();
  if (threadIdx.x >= 8) return;
  o = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
  o *= sum == 0.f ? 0.f : 1.f / sum;
  store_joined(a, p, c, o);
}

template <int D>
void launch_join(const AttentionArgs& a, const AttentionPlan& plan, hipStream_t st) {
  const uint32_t rows = static_cast<uint32_t>(plan.join_queries) * a.q_heads;  // below 2^24
  // Few rows have lanes enough only if a row's channels and parts are spread (32
  // rows of 63 parts: 14.8 us with the attention, one wave to a row 26.2; 128
  // rows 18.5, 20.8; 512 rows 31.0, 29.1; 2048 rows 77.5, 68.7).
  if (rows < 512 && (plan.own.rowsplit ? plan.own_slots : plan.own.groups.d) + plan.front_slots > 8)
    hipLaunchKernelGGL((attention_join_parts_kernel<D>), dim3(rows * (D / 32)), dim3(256), 0, st, a, plan);
  else
    hipLaunchKernelGGL((attention_join_rows_kernel<D>), dim3((rows + 3) / 4), dim3(256), 0, st, a, plan, rows);
}

}  // namespace

bool attention_plan(const AttentionArgs& a, AttentionPlan* plan) {
  const int64_t own_rows = static_cast<int64_t>(a.max_q) * a.group.d;
  const int64_t front_rows = static_cast<int64_t>(a.tokens) * a.group.d;
  *plan = AttentionPlan{};
  AttentionCut& own = plan->own;
  AttentionCut& front = plan->front;
  own = cut_tokens(own_rows, front_rows, a.seqs, a.heads, a.width << a.page_log2, a.D, false);
  const int64_t cap = a.width << a.page_log2;
  const bool split = own.rowsplit ? own.parts.d > 1 : cap > int64_t{1} << own.piece_log2;
  plan->join = split || a.prefix_width > 0;
  // Few rows: run w of sequence s is slot w + s.
  if (plan->join) plan->own_slots = own.rowsplit ? own.parts.d : static_cast<int64_t>(own.groups.d) + a.seqs;
  if (a.prefix_width > 0) {
    front = cut_tokens(front_rows, front_rows, 1, a.heads, a.prefix_width << a.page_log2, a.D, !own.rowsplit);
    plan->front_slots = front.rowsplit ? front.parts.d : front.groups.d;
  }
  // No more queries than rows of q, and than max_q of every sequence.
  const int64_t places = static_cast<int64_t>(a.seqs) * a.max_q;
  plan->join_by_place = places <= a.tokens;
  const int64_t queries = least64(places, a.tokens);
  plan->join_queries = static_cast<int>(queries);
  return cut_blocks(a, own, a.seqs) + (a.prefix_width > 0 ? cut_blocks(a, front, 1) : 0) < kGrid &&
         queries * a.q_heads < kGrid;
}

size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& plan) {
  if (!plan.join) return 0;
  const size_t rows = static_cast<size_t>(plan.own_slots * (plan.own.rowsplit ? a.tokens : a.max_q) +
                                          plan.front_slots * a.tokens) * static_cast<size_t>(a.q_heads);
  return rows * static_cast<size_t>(a.D + 2) * 4 + (static_cast<size_t>(a.seqs) + 1) * 8;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, bool q_f16, hipStream_t st) {
  if (a.D == 64)
    launch_attention_64(a, plan, !q_f16, st);
  else if (a.D == 128)
    launch_attention_128(a, plan, !q_f16, st);
  else
    launch_attention_256(a, plan, !q_f16, st);
  if (plan.join) {
    if (a.D == 64)
      launch_join<64>(a, plan, st);
    else if (a.D == 128)
      launch_join<128>(a, plan, st);
    else
      launch_join<256>(a, plan, st);
  }
  return hipGetLastError();
}

}  // namespace w4a4
