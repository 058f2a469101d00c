// norm.h - parameters and host launchers of the residual RMSNorm.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace vdn {

struct NormParams {
  const void *x, *res;
  void *res_out, *out;
  float* scales;
  const float* weight;
  long long rows;
  int W;
  float eps;
  long long sx, sres, sres_out, sout;  // row strides, elements
};

struct NormBwdParams {
  const void *h, *dy, *dh;
  void* dx;
  float* dweight;
  float* parts;          // [n_parts, W]
  const float* weight;
  long long rows;
  int W;
  float eps;
  long long sh, sdy, sdh, sdx;
  int n_parts;
};

// vec: rows and pointers are 16-byte aligned and W % 8 == 0
cudaError_t launch_norm_fwd(const NormParams& p, int fp32, int output, int vec, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormBwdParams& p, int fp32, int vec, cudaStream_t st);
// blocks of launch_norm_bwd, each of which leaves a partial weight gradient (also the count in NormBwdParams)
int norm_parts(long long rows, int W);
// bytes of launch_norm_bwd's parts (rows wider than registers: and two factors of each row)
size_t norm_workspace(long long rows, int W);

}  // namespace vdn
