// ssm_chain.cuh -- kernels of one call that start while their predecessor ends
// (programmatic dependent launch). Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

namespace ssm {

// A kernel of a call whose predecessor on the stream is the call's own: it may
// start while that one's last blocks run, and waits for it (chain_wait) before
// it reads anything.
template <typename P>
inline cudaError_t launch_chained(void (*kern)(P), dim3 grid, int threads, int bytes,
                                  cudaStream_t stream, const P& p) {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)bytes;
  c.stream = stream;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, p);
}

// Before the first read of what the preceding kernel of the call wrote.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's blocks may take the places that this kernel's leave. A kernel
// that holds tensor memory calls it once a block has its columns, so that none of
// them can wait for columns that a waiting successor has taken; the others at once.
__device__ __forceinline__ void chain_go() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace ssm
