// Launches of the vocabulary losses' and the embedding's kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace zl {

// Programmatic launches: every kernel of a call lets the next one start when
// its own blocks run, and waits for the one before it (complete, and so for all
// before that) before it touches what they wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// `dependent`: a programmatic launch behind the kernel before it.
template <typename... P, typename... A>
inline cudaError_t launch(void (*kernel)(P...), dim3 blocks, int threads, size_t shared, cudaStream_t s, bool dependent,
                   const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = blocks;
  c.blockDim = dim3(unsigned(threads));
  c.dynamicSmemBytes = shared;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

inline bool aligned16(const void* p, int64_t stride_bytes) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

}  // namespace zl
