// attention.hip — how a call of the attention over the quantized cache is cut,
// and the joining of its parts.
//
// A row's tokens (its sequence's own, and the prefix) are cut into parts where
// there are few rows, each a workgroup's (attention_kernel.h).  A part leaves
// (ref, l, O) with p = 2^(t - ref) summed to l and p v to O, in float32;
//   out = sum_i 2^(ref_i - M) O_i / sum_i 2^(ref_i - M) l_i,  M = max ref_i,
// taken in the order of the parts.
//
// The lengths are on the device: the host cuts by the tables' capacity, and a
// workgroup whose sequence is shorter than its part's share ends at once.
#include "attention_kernel.h"

namespace w4a4 {
namespace {

constexpr int kMaxParts = 256;       // of the own tokens, and of the prefix
constexpr int64_t kGrid = 1 << 24;   // workgroups of 256 threads: below 2^32 threads

AttentionCut cut_rows(int64_t rows, int64_t seqs, int64_t heads, int64_t capacity, int D) {
  AttentionCut c{};
  c.rowsplit = rows > 32 || (D == 256 && rows > 16);
  c.tiles = D < 256 && rows > (c.rowsplit ? 64 : 16) ? 2 : 1;
  const int64_t group_rows = 16 * c.tiles * (c.rowsplit ? kAttnWaves : 1);
  c.row_groups = (rows + group_rows - 1) / group_rows;
  if (c.row_groups < 1) c.row_groups = 1;
  const int64_t units = seqs > 0 ? seqs * heads * c.row_groups : 1;
  c.least = c.rowsplit ? 256 : 128;
  const int64_t most = (capacity + c.least - 1) / c.least;
  int64_t parts = (4096 + units - 1) / units;
  parts = parts < most ? parts : most;
  c.parts = static_cast<int>(parts < 1 ? 1 : parts < kMaxParts ? parts : kMaxParts);
  return c;
}

template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(AttentionArgs a, AttentionPlan plan) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ float weight[2 * kMaxParts];
  __shared__ float red[4];
  __shared__ f4 lds[kGroups][kLanes];
  const int head = blockIdx.x % a.q_heads;
  const uint32_t at = blockIdx.x / a.q_heads;
  const int s = at / static_cast<uint32_t>(a.max_q), i = at % static_cast<uint32_t>(a.max_q);
  const Span span = own_span(a, s);
  if (i >= span.n) return;
  const int own = parts_of(span.length, plan.own.parts, plan.own.least);
  if (own == 1 && !a.prefix_table) return;  // stored at once
  const int front = a.prefix_table ? parts_of(front_span(a).length, plan.front.parts, plan.front.least) : 0;
  const int n = own + front;
  const int64_t row = static_cast<int64_t>(span.first + i) * a.q_heads + head;
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.q_heads;
  const float* stats = a.partial + plan.slots * rows * D;
  auto slot = [&](int k) -> int64_t { return (k < own ? k : plan.own.parts + k - own) * rows + row; };

  auto reduce = [&](float v, bool max) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = max ? fmaxf(v, __shfl_xor(v, o)) : v + __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = max ? fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])) : (red[0] + red[1]) + (red[2] + red[3]);
    __syncthreads();
    return v;
  };
  float top = -INFINITY;
  for (int k = threadIdx.x; k < n; k += 256) top = fmaxf(top, stats[2 * slot(k)]);
  top = reduce(top, true);
  float sum = 0.f;
  for (int k = threadIdx.x; k < n; k += 256) {
    const float f = __builtin_amdgcn_exp2f(stats[2 * slot(k)] - top);
    weight[k] = f;
    sum += f * stats[2 * slot(k) + 1];
  }
  sum = reduce(sum, false);
  const int c = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  f4 o = {0.f, 0.f, 0.f, 0.f};
  for (int k = grp; k < n; k += kGroups)
    o += weight[k] * *reinterpret_cast<const f4*>(a.partial + slot(k) * D + 4 * c);
  lds[grp][c] = o;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) o += lds[k][c];
  o *= sum == 0.f ? 0.f : 1.f / sum;
  const int64_t to = (span.first + i) * a.ldo + static_cast<int64_t>(head) * D + 4 * c;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.out_f16)
      static_cast<_Float16*>(a.out)[to + e] = static_cast<_Float16>(o[e]);
    else
      static_cast<float*>(a.out)[to + e] = o[e];
  }
}

void launch_part(const AttentionArgs& a, const AttentionCut& c, int front, int slot0, int slots, bool pair,
                 hipStream_t st) {
  if (a.D == 64)
    launch_attention_64(a, c, front, slot0, slots, pair, st);
  else if (a.D == 128)
    launch_attention_128(a, c, front, slot0, slots, pair, st);
  else
    launch_attention_256(a, c, front, slot0, slots, pair, st);
}

}  // namespace

bool attention_plan(const AttentionArgs& a, AttentionPlan* plan) {
  plan->own = cut_rows(static_cast<int64_t>(a.max_q) * a.group, a.seqs, a.heads, a.width << a.page_log2, a.D);
  plan->front = AttentionCut{};
  plan->slots = plan->own.parts > 1 ? plan->own.parts : 0;
  if (a.prefix_width > 0) {
    plan->front = cut_rows(static_cast<int64_t>(a.tokens) * a.group, 1, a.heads, a.prefix_width << a.page_log2, a.D);
    plan->slots = plan->own.parts + plan->front.parts;
  }
  return static_cast<int64_t>(a.seqs) * a.heads * plan->own.row_groups * plan->own.parts < kGrid &&
         a.heads * plan->front.row_groups * plan->front.parts < kGrid &&
         static_cast<int64_t>(a.seqs) * a.max_q * a.q_heads < kGrid;
}

size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& plan) {
  return static_cast<size_t>(plan.slots) * static_cast<size_t>(a.tokens) * static_cast<size_t>(a.q_heads) *
         static_cast<size_t>(a.D + 2) * 4;
}

hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& plan, bool q_f16, hipStream_t st) {
  const int slots = static_cast<int>(plan.slots);
  if (a.prefix_table) launch_part(a, plan.front, 1, plan.own.parts, slots, !q_f16, st);
  launch_part(a, plan.own, 0, 0, slots, !q_f16, st);
  if (slots > 0) {
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.seqs) * a.max_q * a.q_heads)), block(256);
    if (a.D == 64)
      hipLaunchKernelGGL((attention_join_kernel<64>), grid, block, 0, st, a, plan);
    else if (a.D == 128)
      hipLaunchKernelGGL((attention_join_kernel<128>), grid, block, 0, st, a, plan);
    else
      hipLaunchKernelGGL((attention_join_kernel<256>), grid, block, 0, st, a, plan);
  }
  return hipGetLastError();
}

}  // namespace w4a4
