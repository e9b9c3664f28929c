// Host-side helpers shared by the libmedusa translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "medusa.h"

namespace medusa {

// Record a message for medusa_last_error() and return `code`.
int fail(int code, const char* fmt, ...);
// Map a CUDA error after a launch to MEDUSA_ERR_CUDA (or MEDUSA_OK).
int check_launch(const char* what);
// Streaming multiprocessors of the current device (cached per device).
int sm_count();
// Validate a medusa_tree_t (host fields and non-null device arrays).
int check_tree(const medusa_tree_t* tree, const char* what);
// Validate a medusa_pages_t (host fields and non-null device arrays).
int check_pages(const medusa_pages_t* pages, const char* what);
// Validate the pools of a paged cache.
int check_pool(const void* k_pages, const void* v_pages, int num_pages, int page_size, int Hkv, int Dh,
               medusa_dtype dtype, const char* what);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Launch through cudaLaunchKernelEx (arguments coerced to the kernel's types).
template <typename... KArgs, typename... Args>
cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                          Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
// The same for a kernel that may start while the one before it on the stream
// still runs, and waits for that one's end itself (griddepcontrol.wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         Args&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
// In clusters of `cl` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), int cl, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                           Args&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
// Opt a kernel in to `smem` bytes of shared memory, once per device (`done`: a
// static of the caller's, a bit per device).  Returns the kernel's attributes'
// status, MEDUSA_OK or MEDUSA_ERR_CUDA, and with min_regs > 0 checks that it
// was built with at least that many registers a thread, with smem_base > 0 that
// its dynamic shared memory begins at that byte of the block's.
int prepare_kernel(const void* kernel, size_t smem, int min_regs, int smem_base, std::atomic<uint64_t>* done,
                   const char* what);
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace medusa
