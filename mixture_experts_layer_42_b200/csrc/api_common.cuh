// Host helpers shared by the C ABI's entry points.
#pragma once

#include "common.cuh"

namespace moe {

inline bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(ws) + off);
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Make this thread's current device the one the caller's work lives on: the
// device of `ptr` (a device buffer of the call), else the stream's device.
moe_status bind_device(cudaStream_t s, const void* ptr);

// SMs of the current device.
int num_sms_current();

// Whether moe_select_expert_kernel chose the CUDA-core kernels.
bool simt_selected();

// A layer's shape and batch (see moe_config's limits).
moe_status check_config(const moe_config* c, int64_t T);

}  // namespace moe
