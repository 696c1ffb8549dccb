// Internal interface of the RMS norm with weight, SiLU gate and residual scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dynconv.h"

namespace dynconv {

// Rows [n0, n1, n2] of D elements; strides of the three leading dimensions.
struct NormTensor {
  const void* p;
  int64_t s0, s1, s2;
};

struct NormParams {
  NormTensor x;      // forward: x; backward: what was normalised (x, or h with the residual before)
  NormTensor gate;   // p == null: none
  NormTensor res;    // forward: residual, p == null: none
  NormTensor dy, dh; // backward; dh.p may be null
  NormTensor y, h;   // forward outputs; h.p null unless the residual is added before
  NormTensor dx, dres, dgate;  // backward outputs; dres.p, dgate.p may be null
  const void* weight;  // [D] or null (ones)
  float* dw_part;      // backward: [blocks][D] partial sums, or null
  int64_t rows;
  int32_t n1, n2, D;
  int32_t before, after;  // where the residual is added
  float alpha, eps;
};

// Workgroups of the backward (each writes one row of partial sums).
int64_t norm_bwd_blocks(int64_t rows, int64_t D, dynconv_dtype dt, bool vec);
// The most that norm_bwd_blocks returns for any alignment.
int64_t norm_bwd_blocks_max(int64_t rows, int64_t D, dynconv_dtype dt);
// out[D]: the sums over n partial rows.
hipError_t norm_dweight(const float* part, int64_t n, int32_t D, float* out, hipStream_t s);
hipError_t norm_fwd(const NormParams& p, dynconv_dtype dt, bool vec, hipStream_t s);
hipError_t norm_bwd(const NormParams& p, dynconv_dtype dt, bool vec, hipStream_t s);

}  // namespace dynconv
