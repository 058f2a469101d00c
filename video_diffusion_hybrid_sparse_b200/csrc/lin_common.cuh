// lin_common.cuh - device helpers shared by the kernels of the causal linear
// memory: decay powers, walk order and element loads.
#pragma once

#include "linear.h"

namespace vdn {

// log2(lambda).  -infinity (lambda = 0) becomes a finite number whose first
// power underflows to 0 and whose power 0 is 1; a NaN stays one.
__device__ __forceinline__ float lin_log2_decay(float log_decay) {
  const float l = log_decay < -1e30f ? -1e30f : log_decay;
  return l * 1.4426950408889634f;
}

// lambda^n.  The product's rounding is a relative error of n |log lambda| 2^-24
// of the power: at most 1e-5 before the power itself is below 2^-126.
__device__ __forceinline__ float lin_pow(float log2_decay, int n) { return exp2f(log2_decay * (float)n); }

__device__ __forceinline__ int lin_length(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

// Chunks before the end of a walk beyond which a token's decay to that end is 0 in fp32 (2^-150 and less).
__device__ __forceinline__ int lin_horizon(float log2_decay, int chunk) {
  return log2_decay < 0.f ? (int)fminf(160.f / -log2_decay / (float)chunk, 1e9f) + 2 : 1 << 30;
}

// A stretch of one CTA's range inside one head: chunks [u0, u1) in walk order.
struct LinPiece {
  int bh, u0, u1;
  __device__ __forceinline__ LinPiece(long long t, long long t_end, const LinPlan& pl) {
    bh = (int)(t / pl.nc);
    u0 = (int)(t - (long long)bh * pl.nc);
    const long long left = t_end - t;
    u1 = left < pl.nc - u0 ? u0 + (int)left : pl.nc;
  }
};

}  // namespace vdn
