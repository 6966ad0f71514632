// Products with 4-bit weights (moe_grouped_matvec_w4, moe_grouped_swiglu_w4,
// moe_forward_w4): the arguments and the launchers of their kernels.
#pragma once

#include "gmm.cuh"

namespace moe {

// One grouped launch: [0] routed experts (rows by offsets), [1] the shared MLP
// (one matrix, rows 0..t_shared-1 of its own x; t_shared == 0: none).
struct W4Args {
  const __nv_bfloat16* x[2];  // rows' activations [x_rows, k] / [t_shared, k]
  const int32_t* src;         // routed row r reads x row src[r]; null: row r
  int64_t x_rows;
  const uint8_t* q1[2];       // codes of w (SWIGLU: w1) [E, n, k/2]
  const uint8_t* q3[2];       // SWIGLU: of w3
  const __nv_bfloat16* s1[2]; // scales [E, k/group, n]
  const __nv_bfloat16* s3[2];
  __nv_bfloat16* out[2];      // [rows, n] / [t_shared, n]
  int n[2], k[2];
  const int32_t* offsets;
  int64_t rows;
  int E, group;
  int64_t t_shared;
  int stall;                  // test hook: CTA 0's first multiplying warp lets a wait run out
  uint32_t* err;
};

cudaError_t launch_w4(bool swiglu, const W4Args& g, int num_sms, cudaStream_t st);
cudaError_t launch_quantize_w4(bool bf16, const void* w, int64_t E, int n, int k, int group,
                               uint8_t* q, __nv_bfloat16* scales, cudaStream_t st);

}  // namespace moe
