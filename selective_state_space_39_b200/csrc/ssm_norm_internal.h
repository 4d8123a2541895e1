// ssm_norm_internal.h -- parameters of the gated norm shared by the C entry
// points (ssm_api.cu) and its kernels (ssm_norm.cu). Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssm {

constexpr int kNormMaxWidth = 49152;  // values per group

enum NormGate { kGateNone = 0, kGateFirst = 1, kGateLast = 2 };

struct NormParams {
  int64_t rows;          // rows of dim elements
  int dim, groups, width;  // width = dim / groups
  int gate;              // NormGate
  float eps, residual_scale;
  const void* x;         // (rows, dim) io; backward: null
  const void* residual;  // (rows, dim) residual type, or null
  const void* z;         // (rows, dim) io, with a gate
  const float* w;        // (dim)
  void* y;               // (rows, dim) io
  void* h_out;           // (rows, dim) residual type, with a residual
  // backward
  const void* h;         // (rows, dim) residual type (io without a residual)
  const void* dy;        // (rows, dim) io
  const void* dh;        // (rows, dim) like h, or null
  void* dx;              // (rows, dim) io
  void* dresidual;       // (rows, dim) like h, or null
  void* dz;              // (rows, dim) io, with a gate
  float* dw;             // (dim) or null
  float* ws;             // (slices, dim) partial dw
  int slices;            // norm_bwd_slices (set by the launch)
};

// types: 0 io bf16, h bf16; 1 io bf16, h fp32; 2 both fp32
cudaError_t launch_norm_fwd(const NormParams& p, int types, bool vec, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormParams& p, int types, bool vec, cudaStream_t stream);
// Row slices of the backward pass (partial sums of dw per slice).
int norm_bwd_slices(int64_t rows, int groups);

}  // namespace ssm
