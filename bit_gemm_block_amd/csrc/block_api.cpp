// block_api.cpp — the C ABI declared in include/w4a4_block.h: argument
// validation and stream-ordered launches.  No allocation happens here.
#include "w4a4_block.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "block_internal.h"
#include "w4a4_internal.h"

namespace {

constexpr int64_t kMaxK = 16384;
constexpr int64_t kMaxRank = 256;
// The grids' limits: tiles of 16 rows along x, 512 threads each, below 2^32
// threads; 256 columns a workgroup along y, 65535 of them.
constexpr int64_t kMaxM = int64_t{8388600} * 16;
constexpr int64_t kMaxN = 65535 * 256;
constexpr int64_t kMaxC = 16384;

bool dtype_ok(int d) { return d == W4A4_F32 || d == W4A4_F16; }
uintptr_t esize(int dtype) { return dtype == W4A4_F16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int status(hipError_t e) { return e == hipSuccess ? W4A4_OK : w4a4::hip_status(e); }

}  // namespace

extern "C" {

size_t w4a4_adapter_workspace_size(int64_t M, int64_t K, int64_t rank) {
  if (M <= 0 || K <= 0 || rank <= 0) return 0;
  // t (of few rows: of every part of K), and one float32 for 32 ranks of a row
  // (whole tiles of 16 rows).  What serves M rows serves fewer.
  const int64_t few = w4a4::kParts * (M < w4a4::kManyRows ? M : w4a4::kManyRows - 1);
  return (static_cast<size_t>(M > few ? M : few) * static_cast<size_t>(w4a4::adapter_tstride(rank)) +
          static_cast<size_t>(w4a4::adapter_urows(M) * w4a4::adapter_tstride(rank) / 32)) * 4;
}

int w4a4_adapter_add(const void* x, int x_dtype, int64_t ldx, const void* At, const void* Bt,
                     int64_t adapters, int64_t rank, const int32_t* index, const int32_t* ranks,
                     const float* scales, int64_t M, int64_t N, int64_t K, const float* y,
                     int64_t ldy, float* out, int64_t ldo, void* workspace, size_t ws_bytes,
                     void* stream) {
  if (!dtype_ok(x_dtype) || M < 0 || N < 0 || K <= 0 || rank <= 0 || adapters < 0 || ldx < K ||
      ldo < N || (y && ldy < N))
    return W4A4_ERR_INVALID_ARG;
  if (K % 64 != 0 || K > kMaxK || rank > kMaxRank || (x_dtype == W4A4_F16 && rank % 8 != 0) ||
      adapters > INT32_MAX || M > kMaxM || N > kMaxN)
    return W4A4_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return W4A4_OK;
  if (!x || !index || !out || !workspace || (adapters > 0 && (!At || !Bt)))
    return W4A4_ERR_INVALID_ARG;
  if (y == out && ldy != ldo) return W4A4_ERR_INVALID_ARG;
  const uintptr_t e = esize(x_dtype);
  if (!aligned(x, 16) || static_cast<uintptr_t>(ldx) * e % 16 != 0 || !aligned(At, 16) ||
      !aligned(Bt, 16) || !aligned(workspace, 16) || !aligned(index, 4) || !aligned(ranks, 4) ||
      !aligned(scales, 4) || !aligned(y, 4) || !aligned(out, 4))
    return W4A4_ERR_MISALIGNED;
  if (ws_bytes < w4a4_adapter_workspace_size(M, K, rank)) return W4A4_ERR_WORKSPACE;
  int s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::AdapterArgs a{};
  a.x = x; a.ldx = ldx; a.At = At; a.Bt = Bt;
  a.L = static_cast<int>(adapters); a.R = static_cast<int>(rank);
  a.index = index; a.ranks = ranks; a.scales = scales;
  a.M = M; a.N = N; a.K = static_cast<int>(K);
  a.y = y; a.ldy = ldy; a.out = out; a.ldo = ldo;
  a.t = static_cast<float*>(workspace);
  return status(w4a4::launch_adapter_add(a, x_dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

int w4a4_norm_residual(const void* h, int h_dtype, int64_t ldh, const void* y, int y_dtype,
                       int64_t ldy, int post_norm, const void* post_w, const void* post_b,
                       const void* gate, int gate_dtype, int64_t ldg, int64_t gate_rows,
                       float residual_scale, int pre_norm, const void* pre_w, const void* pre_b,
                       int p_dtype, float offset, float eps, int64_t M, int64_t C, void* h_out,
                       int64_t ldho, void* x_out, int x_dtype, int64_t ldx, void* stream) {
  if (!dtype_ok(h_dtype) || !dtype_ok(y_dtype) || !dtype_ok(gate_dtype) || !dtype_ok(p_dtype) ||
      !dtype_ok(x_dtype))
    return W4A4_ERR_INVALID_ARG;
  if (post_norm < W4A4_NORM_NONE || post_norm > W4A4_NORM_LAYER || pre_norm < W4A4_NORM_NONE ||
      pre_norm > W4A4_NORM_LAYER)
    return W4A4_ERR_INVALID_ARG;
  if (M < 0 || C <= 0 || !(eps >= 0.f) || std::isinf(eps)) return W4A4_ERR_INVALID_ARG;
  if ((h && ldh < C) || (y && ldy < C) || (gate && (ldg < C || gate_rows <= 0)) ||
      (h_out && ldho < C) || (x_out && ldx < C))
    return W4A4_ERR_INVALID_ARG;
  if (post_norm == W4A4_NORM_NONE && (post_w || post_b)) return W4A4_ERR_INVALID_ARG;
  if (pre_norm == W4A4_NORM_NONE && (pre_w || pre_b)) return W4A4_ERR_INVALID_ARG;
  if (!y && M > 0 && (post_norm != W4A4_NORM_NONE || gate)) return W4A4_ERR_INVALID_ARG;
  if (!x_out && M > 0 && pre_norm != W4A4_NORM_NONE) return W4A4_ERR_INVALID_ARG;
  if (C > kMaxC) return W4A4_ERR_UNSUPPORTED;
  if (M == 0) return W4A4_OK;
  if ((!h && !y) || (!h_out && !x_out)) return W4A4_ERR_INVALID_ARG;
  if (h && h == h_out && ldh != ldho) return W4A4_ERR_INVALID_ARG;
  if (!aligned(h, esize(h_dtype)) || !aligned(y, esize(y_dtype)) ||
      !aligned(gate, esize(gate_dtype)) || !aligned(h_out, esize(h_dtype)) ||
      !aligned(x_out, esize(x_dtype)) || !aligned(post_w, 16) || !aligned(post_b, 16) ||
      !aligned(pre_w, 16) || !aligned(pre_b, 16))
    return W4A4_ERR_MISALIGNED;
  int s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::NormArgs a{};
  a.h = h; a.ldh = ldh; a.y = y; a.ldy = ldy;
  a.post_w = post_w; a.post_b = post_b; a.pre_w = pre_w; a.pre_b = pre_b;
  a.gate = gate; a.ldg = ldg; a.gate_rows = gate_rows;
  a.h_out = h_out; a.ldho = ldho; a.x_out = x_out; a.ldx = ldx;
  a.M = M; a.C = static_cast<int>(C);
  a.post = post_norm; a.pre = pre_norm;
  a.gate_f16 = gate_dtype == W4A4_F16; a.x_f16 = x_dtype == W4A4_F16;
  a.rs = residual_scale; a.offset = offset; a.eps = eps;
  return status(w4a4::launch_norm_residual(a, h_dtype == W4A4_F16, y_dtype == W4A4_F16,
                                           p_dtype == W4A4_F16, static_cast<hipStream_t>(stream)));
}

int w4a4_gated_activation(const void* gate, int64_t ldg, const void* up, int64_t ldu, int in_dtype,
                          int act, int64_t M, int64_t F, void* out, int64_t ldo, int out_dtype,
                          void* stream) {
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype) || act < W4A4_ACT_SILU || act > W4A4_ACT_RELU ||
      M < 0 || F < 0 || ldg < F || ldo < F || (up && ldu < F))
    return W4A4_ERR_INVALID_ARG;
  if (M == 0 || F == 0) return W4A4_OK;
  if (!gate || !out) return W4A4_ERR_INVALID_ARG;
  if (!aligned(gate, esize(in_dtype)) || !aligned(up, esize(in_dtype)) ||
      !aligned(out, esize(out_dtype)))
    return W4A4_ERR_MISALIGNED;
  int s = w4a4::device_status();
  if (s != W4A4_OK) return s;
  w4a4::GatedArgs a{gate, ldg, up, ldu, out, ldo, M, F};
  return status(w4a4::launch_gated_activation(a, in_dtype == W4A4_F16, out_dtype == W4A4_F16, act,
                                              static_cast<hipStream_t>(stream)));
}

}  // extern "C"
