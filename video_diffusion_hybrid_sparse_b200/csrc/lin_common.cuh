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

// Chunks with real rows among [u0, u1), walk order.
__device__ __forceinline__ void lin_real(int u0, int u1, int len, const LinPlan& pl, int reverse, int& a, int& b) {
  const int n = (len + pl.chunk - 1) / pl.chunk;
  a = reverse ? max(u0, pl.nc - n) : u0;
  b = reverse ? u1 : min(u1, n);
  if (a > b) a = b = u0;
}

// Range j's stretch (len: its head's tokens).
__device__ __forceinline__ LinStretch lin_stretch(int j, int len, float log2_decay, const LinPlan& pl, int reverse) {
  const long long t1 = pl.start(j + 1), head0 = (t1 - 1) / pl.nc * pl.nc, t0 = max(pl.start(j), head0);
  LinStretch s;
  s.bh = (int)(head0 / pl.nc);
  if (t1 == head0 + pl.nc) {
    s.u0 = s.u1 = s.end = 0;
    return s;
  }
  lin_real((int)(t0 - head0), (int)(t1 - head0), len, pl, reverse, s.u0, s.u1);
  s.u0 = max(s.u0, s.u1 - lin_horizon(log2_decay, pl.chunk));
  s.end = s.u1;
  return s;
}
// Its piece i of pl.sub.
__device__ __forceinline__ LinStretch lin_piece_of(LinStretch s, int i, const LinPlan& pl) {
  const int n = s.u1 - s.u0, u = s.u0;
  s.u0 = u + n * i / pl.sub;
  s.u1 = u + n * (i + 1) / pl.sub;
  return s;
}

}  // namespace vdn
