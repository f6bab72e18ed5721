// Internal launch interface of the operators beside the layer: block_api.cpp
// validates, adapters.hip, norm_residual.hip and gated.hip run.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

// W4A4_OK if the current device is a gfx950, else W4A4_ERR_UNSUPPORTED (api.cpp).
int device_status();

// ---- low-rank adapters of many requests (adapters.hip) ----------------------
struct AdapterArgs {
  const void* x;  // [M, K], row distance ldx
  int64_t ldx;
  const void* At;  // [L, R, K]
  const void* Bt;  // [L, N, R]
  int L, R;
  const int32_t* index;  // [M]
  const int32_t* ranks;  // [L] or null
  const float* scales;   // [L] or null
  int64_t M, N;
  int K;
  const float* y;  // [M, N] or null
  int64_t ldy;
  float* out;
  int64_t ldo;
  // x . A, [M, adapter_tstride(R)].  Few rows: `parts` such matrices of float32 to
  // be added up, not scaled, defined up to the row's rank.  Many rows, fp32: scaled,
  // zero past the rank; fp16: the same as fp16 pair (hi, then 2^11 times what hi
  // leaves), times a power of two whose inverse follows, one float32 per row for
  // every 32 ranks: [adapter_tstride(R) / 32][adapter_urows(M)].
  float* t;
  int parts;
};

// Rows from which x . A is staged and t enters as a matrix operand.  Above and
// below it, K = 4096: 256 rows of eight requests, rank 64: 17.1 us staged against
// 24.0, 256 rows of mixed adapters 22.3 against 31.7; 64 rows of mixed adapters,
// N = 6144, rank 64: 25.6 against 18.2, N = 28672, rank 16: 22.2 against 17.4 us.
constexpr int64_t kManyRows = 128;
// Parts of K of a call of few rows with long rows.
constexpr int kParts = 4;

// The row distance of t.
__host__ __device__ inline int64_t adapter_tstride(int64_t R) { return (R + 31) / 32 * 32; }
// The row distance of the powers of two: whole tiles of 16.
__host__ __device__ inline int64_t adapter_urows(int64_t M) { return (M + 15) / 16 * 16; }
hipError_t launch_adapter_add(const AdapterArgs& a, bool f16, hipStream_t st);

// ---- norms joined with gate and residual (norm_residual.hip) -----------------
struct NormArgs {
  const void* h;
  int64_t ldh;
  const void* y;
  int64_t ldy;
  const void* post_w;
  const void* post_b;
  const void* gate;
  int64_t ldg, gate_rows;
  const void* pre_w;
  const void* pre_b;
  void* h_out;
  int64_t ldho;
  void* x_out;
  int64_t ldx;
  int64_t M;
  int C;
  int post, pre;  // w4a4_norm
  int gate_f16, x_f16;
  float rs, offset, eps;
};
hipError_t launch_norm_residual(const NormArgs& a, bool h_f16, bool y_f16, bool p_f16,
                                hipStream_t st);

// ---- gated activation (gated.hip) ---------------------------------------------
struct GatedArgs {
  const void* gate;
  int64_t ldg;
  const void* up;  // or null
  int64_t ldu;
  void* out;
  int64_t ldo;
  int64_t M, F;
};
hipError_t launch_gated_activation(const GatedArgs& a, bool in_f16, bool out_f16, int act,
                                   hipStream_t st);

}  // namespace w4a4
