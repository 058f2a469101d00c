// norm.cu - RMSNorm with the residual's addition and an output in the tensors'
// type or in e4m3 with scales, and its backward pass.
//
// Both are bound by memory.  A row is held in the registers of G threads (8
// elements a vector, up to 4 vectors a thread), so that each tensor is read and
// written once: sum of squares, scale and conversion need no second look.  G is
// the smallest power of two from 32 on that holds the row with 2 vectors a
// thread (4 from width 16384 on, where a block ends); blocks of 256 threads hold
// several rows where G is smaller.  Rows wider than 32768 are read again by a
// looping kernel.  Rows whose width or address no 16-byte vector fits take the
// same layout with element loads.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "norm.h"
#include "sm100.cuh"

namespace vdn {
namespace {

constexpr int kE = 8;  // elements of a vector

template <typename T, bool kVec>
__device__ __forceinline__ void load8(float (&f)[kE], const T* p, int col, int W) {
  if constexpr (!kVec) {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = col + e < W ? (float)p[col + e] : 0.f;
  } else if (col >= W) {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = 0.f;
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p + col), b = *reinterpret_cast<const float4*>(p + col + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(p + col);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[2 * e] = bf16_lo(u[e]), f[2 * e + 1] = bf16_hi(u[e]);
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* p, const float (&f)[kE], int col, int W) {
  if constexpr (!kVec) {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (col + e < W) p[col + e] = (T)f[e];
  } else if (col < W) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p + col) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(p + col + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(p + col) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                      pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
  }
}

// e4m3 of f * inv, rounded to nearest even; the product's own rounding can carry
// the largest element past 448 by an ulp, which saturates to 448
template <bool kVec>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&f)[kE], float inv, int col, int W) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  if constexpr (kVec) {
    if (col < W) *reinterpret_cast<uint2*>(p + col) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (col + e < W) p[col + e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
}

template <bool kVec>
__device__ __forceinline__ void load8_weight(float (&f)[kE], const float* w, int col, int W) {
  if (w) {
    load8<float, kVec>(f, w, col, W);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = 1.f;
  }
}

// The scale of a group whose largest magnitude is `most`: 448 is e4m3's largest
// number.  Not below 2^-126, so that its inverse is finite; 1 for zeros.
__device__ __forceinline__ float e4m3_scale(float most) {
  return most == 0.f ? 1.f : most < 448.0f * 1.17549435e-38f ? 1.17549435e-38f : most / 448.0f;
}

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum (or maximum) over the G threads of a row.  `slot`: shared memory of the
// block's warps, another one for each use in flight.
template <int G, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  if constexpr (G > 32) {
    const int warp = threadIdx.x >> 5, first = threadIdx.x / G * (G / 32);
    if ((threadIdx.x & 31) == 0) slot[warp] = v;
    __syncthreads();
    v = slot[first];
#pragma unroll
    for (int i = 1; i < G / 32; ++i) v = kMax ? max_nan(v, slot[first + i]) : v + slot[first + i];
  }
  return v;
}

constexpr int block_of(int G) { return G < 256 ? 256 : G; }

constexpr float kBigDown = 0x1p-64f, kSmallUp = 0x1p64f;

// Factor that brings a row's elements back where 32 bits hold their squares: 1
// unless the sum of squares has overflowed, or vanishes and eps does not cover it.
__device__ __forceinline__ float rescue(float sum, float eps) {
  if (!(sum < INFINITY)) return kBigDown;
  return sum < 0x1p-80f && eps < 0x1p-80f ? kSmallUp : 1.f;
}

// 1 / rms of the row whose G threads hold h, where the elements may have been
// multiplied by `mul` (a power of two) on return: mul / rms belongs to them.
// The second look at the registers is a choice of the whole block (it has a
// barrier), which each thread reads from all warps' sums.
template <int G, int kV>
__device__ __forceinline__ float row_rstd(float (&h)[kV][kE], int W, float eps, float* slot, float& mul) {
  mul = 1.f;
  auto squares = [&] {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) s = fmaf(h[i][e], h[i][e], s);
    return s;
  };
  float sum = row_reduce<G, false>(squares(), slot);
  bool again = rescue(sum, eps) != 1.f;
  if constexpr (G > 32 && G < 256) {
    constexpr int kWarps = G / 32, kRows = block_of(G) / G;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float s = slot[r * kWarps];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) s += slot[r * kWarps + i];
      again |= rescue(s, eps) != 1.f;
    }
  }
  if (again) {
    mul = rescue(sum, eps);
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int e = 0; e < kE; ++e) h[i][e] *= mul;
    if constexpr (G > 32) __syncthreads();  // the first sums have been read
    sum = row_reduce<G, false>(squares(), slot);
  }
  return rsqrtf(sum / (float)W + eps * mul * mul);
}

}  // namespace

// kOut: 0 the tensors' type, 1 e4m3 with a scale a row, 2 e4m3 with a scale for each 128 columns
template <typename T, int G, int kV, int kOut, bool kVec>
__global__ void __launch_bounds__(block_of(G)) norm_fwd(const __grid_constant__ NormParams p) {
  constexpr int kRows = block_of(G) / G;
  __shared__ float s_sum[32], s_max[32];
  const int t = threadIdx.x % G;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / G;
  const bool real = row < p.rows;
  const long long r = real ? row : 0;
  const T* x = static_cast<const T*>(p.x) + r * p.sx;
  float h[kV][kE];
#pragma unroll
  for (int i = 0; i < kV; ++i) load8<T, kVec>(h[i], x, (i * G + t) * kE, real ? p.W : 0);
  if (p.res) {
    const T* res = static_cast<const T*>(p.res) + r * p.sres;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float a[kE];
      load8<T, kVec>(a, res, (i * G + t) * kE, real ? p.W : 0);
#pragma unroll
      for (int e = 0; e < kE; ++e) h[i][e] += a[e];
    }
  }
  if (p.res_out && real) {
    T* ro = static_cast<T*>(p.res_out) + r * p.sres_out;
#pragma unroll
    for (int i = 0; i < kV; ++i) store8<T, kVec>(ro, h[i], (i * G + t) * kE, p.W);
  }
  float mul;
  const float rstd = row_rstd<G, kV>(h, p.W, p.eps, s_sum, mul);
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int col = (i * G + t) * kE;
    float w[kE];
    load8_weight<kVec>(w, p.weight, col, p.W);
#pragma unroll
    for (int e = 0; e < kE; ++e) h[i][e] = h[i][e] * rstd * w[e];
  }
  if constexpr (kOut == 0) {
    if (real) {
      T* out = static_cast<T*>(p.out) + r * p.sout;
#pragma unroll
      for (int i = 0; i < kV; ++i) store8<T, kVec>(out, h[i], (i * G + t) * kE, p.W);
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(p.out) + r * p.sout;
    if constexpr (kOut == 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if ((i * G + t) * kE + e < p.W) most = max_nan(most, fabsf(h[i][e]));
      most = row_reduce<G, true>(most, s_max);
      const float scale = e4m3_scale(most);
      if (real) {
        if (t == 0) p.scales[r] = scale;
#pragma unroll
        for (int i = 0; i < kV; ++i) store8_e4m3<kVec>(out, h[i], 1.0f / scale, (i * G + t) * kE, p.W);
      }
    } else {
      const int groups = (p.W + 127) / 128;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int col = (i * G + t) * kE;
        most = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (col + e < p.W) most = max_nan(most, fabsf(h[i][e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float scale = e4m3_scale(most);
        if (real) {
          if ((t & 15) == 0 && col < p.W) p.scales[r * groups + col / 128] = scale;
          store8_e4m3<kVec>(out, h[i], 1.0f / scale, col, p.W);
        }
      }
    }
  }
}

// Rows of more than 32768 elements: a block of 1024 threads reads the row up to
// three times (sum; largest magnitude, for a scale a row; result).  Nothing is
// written before the last pass, so that x may be residual_out.
template <typename T, int kOut>
__global__ void __launch_bounds__(1024) norm_fwd_wide(const __grid_constant__ NormParams p) {
  constexpr int G = 1024;
  __shared__ float s_sum[32], s_max[32];
  const int t = threadIdx.x;
  const long long r = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + r * p.sx;
  const T* res = p.res ? static_cast<const T*>(p.res) + r * p.sres : nullptr;
  auto load = [&](float (&h)[kE], int col) {
    load8<T, false>(h, x, col, p.W);
    if (res) {
      float a[kE];
      load8<T, false>(a, res, col, p.W);
#pragma unroll
      for (int e = 0; e < kE; ++e) h[e] += a[e];
    }
  };
  float h[kE], mul = 1.f;
  auto squares = [&] {
    float sum = 0.f;
    for (int col = t * kE; col < p.W; col += G * kE) {
      load(h, col);
#pragma unroll
      for (int e = 0; e < kE; ++e) sum = fmaf(mul * h[e], mul * h[e], sum);
    }
    return row_reduce<G, false>(sum, s_sum);
  };
  float sum = squares();
  if ((mul = rescue(sum, p.eps)) != 1.f) {
    __syncthreads();
    sum = squares();
  }
  const float rstd = rsqrtf(sum / (float)p.W + p.eps * mul * mul);
  auto scaled = [&](int col) {
    float w[kE];
    load8_weight<false>(w, p.weight, col, p.W);
#pragma unroll
    for (int e = 0; e < kE; ++e) h[e] = mul * h[e] * rstd * w[e];
  };
  float scale = 1.f;
  if constexpr (kOut == 1) {
    float most = 0.f;
    for (int col = t * kE; col < p.W; col += G * kE) {
      load(h, col);
      scaled(col);
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (col + e < p.W) most = max_nan(most, fabsf(h[e]));
    }
    scale = e4m3_scale(row_reduce<G, true>(most, s_max));
    if (t == 0) p.scales[r] = scale;
  }
  const int groups = (p.W + 127) / 128;
  for (int c0 = 0; c0 < p.W; c0 += G * kE) {
    const int col = c0 + t * kE;
    load(h, col);
    if (p.res_out) store8<T, false>(static_cast<T*>(p.res_out) + r * p.sres_out, h, col, p.W);
    scaled(col);
    if constexpr (kOut == 0) {
      store8<T, false>(static_cast<T*>(p.out) + r * p.sout, h, col, p.W);
    } else {
      if constexpr (kOut == 2) {
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (col + e < p.W) most = max_nan(most, fabsf(h[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        scale = e4m3_scale(most);
        if ((t & 15) == 0 && col < p.W) p.scales[r * groups + col / 128] = scale;
      }
      store8_e4m3<false>(static_cast<uint8_t*>(p.out) + r * p.sout, h, 1.0f / scale, col, p.W);
    }
  }
}

// Backward: groups of G threads go through rows `n_parts` apart; sum h^2 and
// sum g h come from one look at the row, and each thread keeps the weight's
// gradient of its own columns over all its rows (fixed order, no atomics).
template <typename T, int G, int kV, bool kVec>
__global__ void __launch_bounds__(block_of(G)) norm_bwd(const __grid_constant__ NormBwdParams p) {
  constexpr int kRows = block_of(G) / G;
  __shared__ float s_sq[32], s_gh[32];
  const int t = threadIdx.x % G;
  const int part = blockIdx.x * kRows + threadIdx.x / G;
  float acc[kV][kE] = {};
  // the block's row groups make the same number of turns (they share barriers)
  for (long long first = (long long)blockIdx.x * kRows; first < p.rows; first += p.n_parts) {
    const long long row = first + threadIdx.x / G;
    const bool real = row < p.rows;
    const long long r = real ? row : 0;
    const int W = real ? p.W : 0;
    float h[kV][kE], g[kV][kE];
    float gh = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      load8<T, kVec>(h[i], static_cast<const T*>(p.h) + r * p.sh, (i * G + t) * kE, W);
      load8<T, kVec>(g[i], static_cast<const T*>(p.dy) + r * p.sdy, (i * G + t) * kE, W);
    }
    float mul;
    // h * rn is the normed row; a row that does not exist is zeros (eps may be 0)
    const float rn = row_rstd<G, kV>(h, p.W, real ? p.eps : 1.f, s_sq, mul);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float w[kE];
      load8_weight<kVec>(w, p.weight, (i * G + t) * kE, p.W);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        h[i][e] *= rn;
        gh = fmaf(g[i][e] * w[e], h[i][e], gh);
      }
    }
    const float c = row_reduce<G, false>(gh, s_gh) / (float)p.W, rstd = rn * mul;
    T* dx = static_cast<T*>(p.dx) + r * p.sdx;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int col = (i * G + t) * kE;
      float w[kE], d[kE] = {};
      load8_weight<kVec>(w, p.weight, col, p.W);
      if (p.dh) load8<T, kVec>(d, static_cast<const T*>(p.dh) + r * p.sdh, col, W);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        acc[i][e] = fmaf(g[i][e], h[i][e], acc[i][e]);
        d[e] = fmaf(rstd, g[i][e] * w[e] - h[i][e] * c, d[e]);
      }
      if (real) store8<T, kVec>(dx, d, col, p.W);
    }
  }
  if (p.parts) {
    float* dst = p.parts + (long long)part * p.W;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int col = (i * G + t) * kE;
#pragma unroll
      for (int e = 0; e < kE; ++e)
        if (col + e < p.W) dst[col + e] = acc[i][e];
    }
  }
}

// Backward of rows of more than 32768 elements: a block a row, read twice; the
// weight's gradient by norm_dweight_wide from each row's factors (rescue's and 1 / rms).
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_wide(const __grid_constant__ NormBwdParams p, float2* rstds) {
  constexpr int G = 1024;
  __shared__ float s_sq[32], s_gh[32];
  const long long r = blockIdx.x;
  const T* h0 = static_cast<const T*>(p.h) + r * p.sh;
  const T* dy0 = static_cast<const T*>(p.dy) + r * p.sdy;
  float h[kE], g[kE], w[kE], mul = 1.f, sq, gh;
  auto sums = [&] {
    sq = 0.f, gh = 0.f;
    for (int col = threadIdx.x * kE; col < p.W; col += G * kE) {
      load8<T, false>(h, h0, col, p.W);
      load8<T, false>(g, dy0, col, p.W);
      load8_weight<false>(w, p.weight, col, p.W);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        sq = fmaf(mul * h[e], mul * h[e], sq);
        gh = fmaf(g[e] * w[e], mul * h[e], gh);
      }
    }
    sq = row_reduce<G, false>(sq, s_sq);
    gh = row_reduce<G, false>(gh, s_gh);
  };
  sums();
  if ((mul = rescue(sq, p.eps)) != 1.f) {
    __syncthreads();
    sums();
  }
  const float rn = rsqrtf(sq / (float)p.W + p.eps * mul * mul), rstd = rn * mul;
  const float c = gh * rn / (float)p.W;
  if (rstds && threadIdx.x == 0) rstds[r] = make_float2(mul, rn);
  for (int col = threadIdx.x * kE; col < p.W; col += G * kE) {
    float d[kE] = {};
    load8<T, false>(h, h0, col, p.W);
    load8<T, false>(g, dy0, col, p.W);
    load8_weight<false>(w, p.weight, col, p.W);
    if (p.dh) load8<T, false>(d, static_cast<const T*>(p.dh) + r * p.sdh, col, p.W);
#pragma unroll
    for (int e = 0; e < kE; ++e) d[e] = fmaf(rstd, g[e] * w[e] - mul * h[e] * rn * c, d[e]);
    store8<T, false>(static_cast<T*>(p.dx) + r * p.sdx, d, col, p.W);
  }
}

// h and dy are read again: dx must not have overwritten them (outputs do not overlap inputs)
template <typename T>
__global__ void __launch_bounds__(256) norm_dweight_wide(const __grid_constant__ NormBwdParams p, const float2* rstds) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= p.W) return;
  float acc = 0.f;
  for (long long r = blockIdx.y; r < p.rows; r += p.n_parts) {
    const float2 f = rstds[r];  // two factors: their product may be below 32 bits' range
    acc = fmaf((float)static_cast<const T*>(p.dy)[r * p.sdy + col],
               f.x * (float)static_cast<const T*>(p.h)[r * p.sh + col] * f.y, acc);
  }
  p.parts[(long long)blockIdx.y * p.W + col] = acc;
}

// dweight[col] = sum of the parts, in order
__global__ void __launch_bounds__(256) norm_dweight(const float* parts, int n_parts, int W, float* dweight) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < W)
#pragma unroll 8
    for (int i = warp; i < n_parts; i += 8) a += parts[(long long)i * W + col];
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < W) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += s[i][lane];
    dweight[col] = a;
  }
}

namespace {

constexpr int kWide = 32768;

// threads of a row: at most 2 vectors a thread up to width 16384, then 4
int group_of(int W) {
  int g = 32;
  while (g < 1024 && g * 2 * kE < W) g *= 2;
  return g;
}
int vectors_of(int W, int g) { return W <= g * kE ? 1 : W <= g * 2 * kE ? 2 : 4; }

// Calls f with (G, vectors) as compile-time numbers.
template <typename F>
cudaError_t by_width(int W, F f) {
  const int g = group_of(W), v = vectors_of(W, g);
#define VDN_NORM_CASE(GG)                                                     \
  if (g == GG) {                                                              \
    if (GG == 32 && v == 1) return f(std::integral_constant<int, GG>(), std::integral_constant<int, 1>()); \
    if (GG == 1024 && v == 4) return f(std::integral_constant<int, GG>(), std::integral_constant<int, 4>()); \
    return f(std::integral_constant<int, GG>(), std::integral_constant<int, 2>()); \
  }
  VDN_NORM_CASE(32)
  VDN_NORM_CASE(64)
  VDN_NORM_CASE(128)
  VDN_NORM_CASE(256)
  VDN_NORM_CASE(512)
  VDN_NORM_CASE(1024)
#undef VDN_NORM_CASE
  return cudaErrorInvalidValue;
}

template <typename T, int kOut>
cudaError_t fwd(const NormParams& p, int vec, cudaStream_t st) {
  if (p.W > kWide) {
    norm_fwd_wide<T, kOut><<<(unsigned)p.rows, 1024, 0, st>>>(p);
    return cudaGetLastError();
  }
  return by_width(p.W, [&](auto G, auto V) {
    constexpr int g = decltype(G)::value, v = decltype(V)::value, block = block_of(g), rows = block / g;
    const unsigned grid = (unsigned)((p.rows + rows - 1) / rows);
    if (vec)
      norm_fwd<T, g, v, kOut, true><<<grid, block, 0, st>>>(p);
    else
      norm_fwd<T, g, v, kOut, false><<<grid, block, 0, st>>>(p);
    return cudaGetLastError();
  });
}

long long norm_factors_at(int n_parts, int W) { return ((long long)n_parts * W + 1) / 2 * 2; }  // 8-byte aligned

template <typename T>
cudaError_t bwd(const NormBwdParams& p, int vec, cudaStream_t st) {
  cudaError_t e;
  if (p.W > kWide) {
    float2* rstds = p.parts ? reinterpret_cast<float2*>(p.parts + norm_factors_at(p.n_parts, p.W)) : nullptr;
    norm_bwd_wide<T><<<(unsigned)p.rows, 1024, 0, st>>>(p, rstds);
    if (p.parts) norm_dweight_wide<T><<<dim3((p.W + 255) / 256, p.n_parts), 256, 0, st>>>(p, rstds);
    e = cudaGetLastError();
  } else {
    e = by_width(p.W, [&](auto G, auto V) {
      constexpr int g = decltype(G)::value, v = decltype(V)::value, block = block_of(g), rows = block / g;
      const unsigned grid = (unsigned)(p.n_parts / rows);
      if (vec)
        norm_bwd<T, g, v, true><<<grid, block, 0, st>>>(p);
      else
        norm_bwd<T, g, v, false><<<grid, block, 0, st>>>(p);
      return cudaGetLastError();
    });
  }
  if (e != cudaSuccess || !p.parts) return e;
  norm_dweight<<<(p.W + 31) / 32, 256, 0, st>>>(p.parts, p.n_parts, p.W, p.dweight);
  return cudaGetLastError();
}

}  // namespace

size_t norm_workspace(long long rows, int W) {
  const int n = norm_parts(rows, W);
  return (size_t)(W > kWide ? norm_factors_at(n, W) + 2 * rows : (long long)n * W) * 4;
}

int norm_parts(long long rows, int W) {
  if (W > kWide) return (int)std::min<long long>(rows, 64);
  const int g = group_of(W), block = block_of(g), per = block / g;
  const long long blocks = std::min<long long>((rows + per - 1) / per, 148 * (block == 256 ? 3 : block == 512 ? 2 : 1));
  return (int)(blocks * per);
}

cudaError_t launch_norm_fwd(const NormParams& p, int fp32, int output, int vec, cudaStream_t st) {
  if (fp32)
    return output == 0 ? fwd<float, 0>(p, vec, st) : output == 1 ? fwd<float, 1>(p, vec, st) : fwd<float, 2>(p, vec, st);
  return output == 0   ? fwd<__nv_bfloat16, 0>(p, vec, st)
         : output == 1 ? fwd<__nv_bfloat16, 1>(p, vec, st)
                       : fwd<__nv_bfloat16, 2>(p, vec, st);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, int fp32, int vec, cudaStream_t st) {
  return fp32 ? bwd<float>(p, vec, st) : bwd<__nv_bfloat16>(p, vec, st);
}

}  // namespace vdn
