// Host helpers shared by the C ABI's entry points.
#pragma once

#include <atomic>

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

// Let `kernel` use `bytes` of dynamic shared memory on the current device:
// asked of the runtime once per kernel and device (`done`: the kernel's own).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Whether moe_select_expert_kernel chose the CUDA-core kernels.
bool simt_selected();

// A layer's shape and batch (see moe_config's limits).
moe_status check_config(const moe_config* c, int64_t T);

}  // namespace moe
