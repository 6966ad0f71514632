// Grouped products by expert (moe_grouped_matmul and its gradients): the
// arguments and the launchers of their kernels.
#pragma once

#include "common.cuh"

namespace moe {

// Which product: the rows' (FWD), their input's gradient (DX), or the
// weights' gradient (DW).
enum { GMM_FWD = 0, GMM_DX = 1, GMM_DW = 2 };

struct GmmArgs {
  const void* a;   // FWD x [R, K]; DX dy [R, N]; DW dy [R, N]
  const void* b;   // FWD, DX w [E, N, K]; DW x [R, K]
  void* out;       // FWD y [R, N]; DX dx [R, K]; DW dw [E, N, K]
  const int32_t* offsets;
  int64_t rows;
  int E, n, k;
  int out_f32;     // DW: dw in fp32 (else in act)
  int accumulate;  // DW: dw += (else dw =)
  uint32_t* err;
};

// Every kernel of these calls is launched as a programmatic dependent of what
// is before it in the stream: it may start (its launch, barriers and other
// set-up overlap that kernel's end), lets the next one start, and waits for the
// grids before it to complete before it reads or writes any tensor.
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Expert e's rows [b, b + count), or none when its offsets are not
// 0 <= offsets[e] <= offsets[e + 1] <= rows (`bad` then says so).
struct Span {
  int32_t b, count;
  bool bad;
};
__device__ __forceinline__ Span expert_span(const int32_t* offsets, int e, int64_t rows) {
  const int32_t b = offsets[e], z = offsets[e + 1];
  Span s;
  s.bad = b < 0 || z < b || (int64_t)z > rows;
  s.b = s.bad ? 0 : b;
  s.count = s.bad ? 0 : z - b;
  return s;
}

// CUDA cores: fp32 and, as a cross-check of the tensor-core kernel, bf16.
cudaError_t launch_gmm_simt(int mode, bool bf16, const GmmArgs& g, int num_sms, cudaStream_t st);
// Tensor cores: bf16. maps: 2 E TMA maps of workspace (DW).
cudaError_t launch_gmm_tc(int mode, const GmmArgs& g, void* maps, int num_sms, cudaStream_t st);

}  // namespace moe
