// Launches that overlap the end of the kernel before them in the stream.
//
// Every kernel launched here begins with grid_wait(), before it reads or
// writes any global memory, and so runs its set-up (barriers, tensor memory,
// shared memory) while the kernel before it ends: a few microseconds of a
// short call.  grid_go() lets the next kernel in the stream begin its own
// set-up; what that one reads is still only valid after its grid_wait(), which
// returns when this kernel has ended and its writes are visible.  A kernel
// that has begun while its inputs are still being written reads them with
// plain loads after grid_wait(), never with loads for data that is constant
// for the kernel's whole life (__ldg, __restrict__).
//
// A kernel may wait late, before it ends instead of before it begins, when it
// needs nothing of the kernel before it and that one (or the first of a chain
// of such) waited early: what lies before the chain is then complete, and the
// two run beside each other.  A later kernel's wait still covers both.  What a
// late kernel reads before its wait it reads from L2 (TMA, __ldcg): no wait of
// its own has made the writes before the chain visible to its L1.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace bra {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned grid, unsigned threads,
                              size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(std::forward<Args>(args))...);
}

}  // namespace bra
