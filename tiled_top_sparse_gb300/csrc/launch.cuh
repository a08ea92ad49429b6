// Host side of launches: kernels set up while the stream's previous kernel still runs, and what is
// asked about a kernel once.
#pragma once
#include <atomic>

#include <cuda_runtime.h>

namespace tts {

// Waits until the grids this one may have been launched ahead of are complete and their writes
// visible (launch_ahead); returns at once for a plain launch.
__device__ __forceinline__ void wait_for_prior_grids() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel that begins with wait_for_prior_grids(): the launch may be set up while the
// stream's previous kernel still runs, which takes about 2 us off a short kernel behind another.
// Under stream capture the launch is a plain one (a graph's launches are set up already, and
// its edges stay full dependencies).
template <typename... P, typename... A>
cudaError_t launch_ahead(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, A... args) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(stream, &capture);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = capture == cudaStreamCaptureStatusNone ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A property of a compiled kernel, asked for once and kept in `known` (0: not known yet). A query
// that fails is not kept: its error is returned, and the next call asks again.
template <typename Query>
cudaError_t ask_once(std::atomic<int>& known, int* value, Query query) {
  *value = known.load(std::memory_order_relaxed);
  if (*value != 0) return cudaSuccess;
  const cudaError_t e = query(value);
  if (e == cudaSuccess) known.store(*value, std::memory_order_relaxed);
  return e;
}

}  // namespace tts
