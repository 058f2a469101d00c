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

// lambda^n as a state is multiplied by it: s * lambda^n = base s + m s.  Where a state keeps its tokens over many such
// products (|n log lambda| < 1/2), m is lambda^n - 1 and base 1: a rounded power, which is off by up to 2^-24 in the same
// direction each time, is 1e-5 off after a thousand chunks, and 1e-3 after 100000 single tokens.
struct LinFall {
  float m, base;
  __device__ __forceinline__ LinFall(float2 v) : m(v.x), base(v.y) {}
  __device__ __forceinline__ LinFall(float log_decay, int n) {
    const float y = log_decay * (float)n;
    const bool slow = fabsf(y) < 0.5f;
    base = slow ? 1.f : 0.f;
    m = slow ? expm1f(y) : lin_pow(lin_log2_decay(log_decay), n);
  }
  // `s` decayed, plus `a`; an infinite s stays so (m s is the other infinity, or 0 times it)
  __device__ __forceinline__ float operator()(float s, float a) const {
    const float t = fmaf(m, s, a);
    return base == 0.f ? t : fabsf(s) == INFINITY ? s + a : t + s;
  }
};

// The same power as one factor for each of many chunks, rounded so that what one rounding leaves out the next makes up for:
// the product of any number of them in a row is off by a rounding or two.
class LinFactors {
 public:
  __device__ __forceinline__ LinFactors(float log_decay, int n) : f_(log_decay, n), left_(0.f) {}
  __device__ __forceinline__ float next() {
    const float t = f_.m + left_, g = f_.base + t;
    left_ = t - (g - f_.base);
    return g;
  }

 private:
  LinFall f_;
  float left_;
};

__device__ __forceinline__ int lin_length(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

// Chunks before the end of a walk beyond which a token's decay to that end is 0 in fp32 (2^-150 and less).
__device__ __forceinline__ int lin_horizon(float log2_decay, int chunk) {
  return log2_decay < 0.f ? (int)fminf(160.f / -log2_decay / (float)chunk, 1e9f) + 2 : 1 << 30;
}

// Where the ranges of a split plan begin, and which of them hold a head's ends.  With lengths, a list cut into equal
// parts would leave the CTAs of the padding without work: it is cut into parts of equal cost, a chunk without tokens (its
// output rows are zeros, nothing is read) an eighth of one with tokens.  Every kernel of a call cuts by this rule.  Not for
// batches above kLinCutBatch, nor where a part would be less than one chunk with tokens (two ranges
// could begin at one).  Whole warps make and use it, with the same arguments in all lanes unless it says otherwise.
class LinCuts {
 public:
  __device__ __forceinline__ LinCuts(const LinPlan& plan, const int* lengths, int B, int H, int N, int reverse)
      : pl_(plan), H_(H), rev_(reverse), n_(0), cost_(0) {
    if (!pl_.split || !lengths || B > kLinCutBatch) return;
    const int lane = threadIdx.x & 31;
    if (lane < B) n_ = (lin_length(lengths, lane, N) + pl_.chunk - 1) / pl_.chunk;
    to_ = lane < B ? (long long)head_cost(n_) * H : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, to_, o);
      if (lane >= o) to_ += v;
    }
    cost_ = __shfl_sync(0xffffffffu, to_, 31);
    if (cost_ < (long long)kWhole * pl_.grid) cost_ = 0;
  }
  __device__ __forceinline__ long long start(int j) const {
    if (cost_ == 0) return pl_.start(j);
    if (j >= pl_.grid) return pl_.total;
    const long long c = cost_ * j / pl_.grid;
    const int b = __popc(__ballot_sync(0xffffffffu, to_ <= c)), n = __shfl_sync(0xffffffffu, n_, b), cost = head_cost(n);
    const long long in = c - (__shfl_sync(0xffffffffu, to_, b) - (long long)cost * H_);
    const int h = (int)(in / cost);
    return ((long long)b * H_ + h) * pl_.nc + chunk_at((int)(in - (long long)h * cost), n);
  }

  // Head bh: the ranges that hold its first and its last chunk; chunk (of the head) at which range j, another one in each
  // lane, begins, if it begins inside.
  struct Head {
    int first, last, n;
    long long before;
  };
  __device__ __forceinline__ Head head(int bh) const {
    Head r = {0, 0, 0, 0};
    if (cost_ == 0) {
      r.first = pl_.range_of((long long)bh * pl_.nc);
      r.last = pl_.range_of((long long)bh * pl_.nc + pl_.nc - 1);
      return r;
    }
    const int b = bh / H_;
    r.n = __shfl_sync(0xffffffffu, n_, b);
    r.before = __shfl_sync(0xffffffffu, to_, b) - (long long)head_cost(r.n) * (H_ - (bh - b * H_));
    r.first = below(r.before + ((rev_ ? r.n == pl_.nc : r.n > 0) ? kWhole : 1));
    r.last = below(r.before + head_cost(r.n));
    return r;
  }
  __device__ __forceinline__ int start_in(const Head& a, int bh, int j) const {
    const long long u = cost_ == 0 ? pl_.start(j) - (long long)bh * pl_.nc : cost_ * j / pl_.grid - a.before;
    return u <= 0 ? 0 : cost_ == 0 ? (int)u : chunk_at((int)u, a.n);
  }

 private:
  static constexpr int kWhole = 8;
  __device__ __forceinline__ int head_cost(int n) const { return n * (kWhole - 1) + pl_.nc; }
  // the chunk (walk order) at which r of a head's cost is spent, of a head with n chunks with tokens
  __device__ __forceinline__ int chunk_at(int r, int n) const {
    const int pad = pl_.nc - n;
    return rev_ ? (r < pad ? r : pad + (r - pad) / kWhole) : r < n * kWhole ? r / kWhole : r - n * (kWhole - 1);
  }
  // the last range that begins before cost c
  __device__ __forceinline__ int below(long long c) const { return (int)((c * pl_.grid + cost_ - 1) / cost_ - 1); }
  const LinPlan& pl_;
  int H_, rev_, n_;           // n_: chunks with tokens of the lane's sequence
  long long to_ = 0, cost_;   // cost of the sequences up to the lane's, of all; 0: equal parts
};

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

// The stretch of a range that has chunks [u0, u1) of its last head (len: that head's tokens).
__device__ __forceinline__ LinStretch lin_stretch(int u0, int u1, int len, float log2_decay, const LinPlan& pl, int reverse) {
  LinStretch s;
  if (u1 == pl.nc) {
    s.u0 = s.u1 = s.end = 0;
    return s;
  }
  lin_real(u0, u1, len, pl, reverse, s.u0, s.u1);
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
