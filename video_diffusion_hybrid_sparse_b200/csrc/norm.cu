// norm.cu - RMSNorm with the residual's addition and an output in the tensors'
// type or in e4m3 with scales, and its backward pass.
//
// Both are bound by memory.  A row is held in the registers of G threads (8
// elements a vector, up to 4 vectors a thread), so that each tensor is read and
// written once: sum of squares, scale and conversion need no second look.  G is
// the smallest power of two from 8 on that holds the row with one vector a
// thread up to width 256, with two from there (four from width 16384 on, where a
// block ends); blocks of 256 threads hold several rows where G is smaller.  Rows
// wider than 32768 are read again by a looping kernel.  A row whose width or
// address no 16-byte vector fits takes element loads, 32 neighbours at a time
// (eight neighbours a thread: 1.7 TB/s at width 500).  Arithmetic goes by packed
// pairs: with single operations the e4m3 output is bound by the issue of
// instructions (118 us for 100 million elements, whatever is read).  Measured:
// 60480 x 2048 bf16 to e4m3 with groups in 141-158 us (0.84-0.95 of the copy
// rate), gradients at 46080 x 2048 in 147-150 us (0.78: a row's two sums cross
// the threads one after the other, which the second does not need: it could go
// with the first and be multiplied by 1 / rms after).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "norm.h"
#include "norm_range.h"
#include "pdl.cuh"
#include "sm100.cuh"

namespace vdn {
namespace {

constexpr int kE = 8;  // elements of a vector

// Eight neighbours from column `col` of a row (rows wider than registers).
template <typename T>
__device__ __forceinline__ void load8(float (&f)[kE], const T* p, int col, int W) {
#pragma unroll
  for (int e = 0; e < kE; ++e) f[e] = col + e < W ? (float)p[col + e] : 0.f;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[kE], int col, int W) {
#pragma unroll
  for (int e = 0; e < kE; ++e)
    if (col + e < W) p[col + e] = (T)f[e];
}
__device__ __forceinline__ void load8_weight(float (&f)[kE], const float* w, int col, int W) {
#pragma unroll
  for (int e = 0; e < kE; ++e) f[e] = !w ? 1.f : col + e < W ? w[col + e] : 0.f;
}

// two e4m3, rounded to nearest even; a product's own rounding can carry the largest element past 448 by an ulp, which
// saturates to 448
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&f)[kE], float inv, int col, int W) {
#pragma unroll
  for (int e = 0; e < kE; e += 2) {
    const uint32_t v = e4m3x2(f[e] * inv, f[e + 1] * inv);
    if (col + e < W) p[col + e] = (uint8_t)v;
    if (col + e + 1 < W) p[col + e + 1] = (uint8_t)(v >> 8);
  }
}

// The scale of a group whose largest magnitude is `most`: 448 is e4m3's largest
// number.  Not below 2^-126, so that its inverse is finite; 1 for zeros.
__device__ __forceinline__ float e4m3_scale(float most) {
  return most == 0.f ? 1.f : most < 448.0f * 1.17549435e-38f ? 1.17549435e-38f : most * (1.0f / 448.0f);
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
  for (int o = G < 32 ? G / 2 : 16; o > 0; o >>= 1) {
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
// Forward blocks on an SM (60480 x 2048 bf16 to e4m3: 162, 154 and 177 us with 3, 4 and 5); fp32 rows ahead take more
// registers, element loads more still.
template <typename T, bool kVec>
constexpr int blocks_of(int G) {
  return block_of(G) == 256 ? (!kVec ? 2 : sizeof(T) == 2 ? 4 : 3) : block_of(G) == 512 && kVec && sizeof(T) == 2 ? 2 : 1;
}

// Eight elements of a thread in fp32, as pairs.
struct Pairs {
  uint64_t p[kE / 2];
};

// Columns of a thread t of G: its vector i holds the neighbours from column(i, t), or (element loads) those 1, 2, .. 7
// lane widths on, so that a warp's loads are neighbours.
template <int G, bool kVec>
struct Columns {
  static constexpr int kLanes = G < 32 ? G : 32;
  static constexpr int kStep = kVec ? 1 : kLanes;
  static __device__ __forceinline__ int first(int i, int t) {
    return kVec ? (i * G + t) * kE : (i * G + t / kLanes * kLanes) * kE + t % kLanes;
  }
};

// Eight elements as they lie in memory, and fp32 pairs of them.
template <typename T, int G, bool kVec>
struct Raw {
  using C = Columns<G, kVec>;
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int col, int W) {
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        v[i] = col < W ? __ldcs(reinterpret_cast<const uint4*>(p + col) + i) : make_uint4(0, 0, 0, 0);
    } else {
      T f[kE];
#pragma unroll
      for (int e = 0; e < kE; ++e) f[e] = col + e * C::kStep < W ? p[col + e * C::kStep] : (T)0.f;
      if constexpr (sizeof(T) == 4) {
        v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      } else {
        auto two = [&](int e) {
          return (uint32_t)__bfloat16_as_ushort(f[e]) | (uint32_t)__bfloat16_as_ushort(f[e + 1]) << 16;
        };
        v[0] = make_uint4(two(0), two(2), two(4), two(6));
      }
    }
  }
  __device__ __forceinline__ Pairs get() const {
    Pairs r;
    if constexpr (sizeof(T) == 4) {
      const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) r.p[e] = f32x2_pack(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]));
    } else {
      const uint32_t u[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) r.p[e] = f32x2_pack(bf16_lo(u[e]), bf16_hi(u[e]));
    }
    return r;
  }
};

template <typename T, int G, bool kVec>
__device__ __forceinline__ void store_pairs(T* p, const Pairs& f, int col, int W) {
  float a[kE];
#pragma unroll
  for (int e = 0; e < 4; ++e) f32x2_unpack(f.p[e], a[2 * e], a[2 * e + 1]);
  if constexpr (!kVec) {
    constexpr int kStep = Columns<G, kVec>::kStep;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (col + e * kStep < W) p[col + e * kStep] = (T)a[e];
  } else if (col < W) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p + col) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4*>(p + col + 4) = make_float4(a[4], a[5], a[6], a[7]);
    } else {
      *reinterpret_cast<uint4*>(p + col) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                      pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
    }
  }
}

template <int G, bool kVec>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const Pairs& f, float inv, int col, int W) {
  const uint64_t i2 = f32x2_pack(inv, inv);
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    f32x2_unpack(f32x2_mul(f.p[e], i2), a, b);
    u[e] = e4m3x2(a, b);
  }
  if constexpr (kVec) {
    if (col < W) *reinterpret_cast<uint2*>(p + col) = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
  } else {
    constexpr int kStep = Columns<G, kVec>::kStep;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (col + e * kStep < W) p[col + e * kStep] = (uint8_t)(u[e >> 1] >> (8 * (e & 1)));
  }
}

template <int G, bool kVec>
__device__ __forceinline__ Pairs load_weight(const float* w, int col, int W) {
  Pairs r;
  if (!w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r.p[e] = f32x2_pack(1.f, 1.f);
  } else if constexpr (kVec) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = col < W ? *reinterpret_cast<const float4*>(w + col) : z, b = col < W ? *reinterpret_cast<const float4*>(w + col + 4) : z;
    r.p[0] = f32x2_pack(a.x, a.y), r.p[1] = f32x2_pack(a.z, a.w), r.p[2] = f32x2_pack(b.x, b.y), r.p[3] = f32x2_pack(b.z, b.w);
  } else {
    constexpr int kStep = Columns<G, kVec>::kStep;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      r.p[e] = f32x2_pack(col + 2 * e * kStep < W ? w[col + 2 * e * kStep] : 0.f,
                          col + (2 * e + 1) * kStep < W ? w[col + (2 * e + 1) * kStep] : 0.f);
  }
  return r;
}

// Largest magnitude of pairs a..b as the bits of a float: as integers, magnitudes have their order and a NaN is the largest.
__device__ __forceinline__ uint32_t most_bits(const Pairs& f, int a, int b, uint32_t m) {
#pragma unroll
  for (int e = a; e < b; ++e) {
    float x, y;
    f32x2_unpack(f.p[e], x, y);
    m = max(m, max(__float_as_uint(x) & 0x7FFFFFFFu, __float_as_uint(y) & 0x7FFFFFFFu));
  }
  return m;
}

// 1 / rms of the row whose G threads hold h, where the elements may have been
// multiplied by `mul` (a power of two) on return: mul / rms belongs to them.
// The second look at the registers is a choice of the whole block (it has
// barriers), made of the sums of its real rows: `left` rows are left from the
// block's first on, and this row exists if `real` (one that does not is zeros,
// and is normed with eps 1: eps may be 0).
template <int G, int kV>
__device__ __forceinline__ float row_rstd(Pairs (&h)[kV], int W, float eps, bool real, long long left, float* slot,
                                          float& mul) {
  mul = 1.f;
  const float own_eps = real ? eps : 1.f;
  auto squares = [&] {
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) s = f32x2_fma(h[i].p[e], h[i].p[e], s);
    float a, b;
    f32x2_unpack(s, a, b);
    return a + b;
  };
  float sum = row_reduce<G, false>(squares(), slot);
  const float own = norm_rescue(sum, own_eps);
  bool again = own != 1.f;
  if constexpr (G > 32 && G < 256) {
    constexpr int kRows = block_of(G) / G;
    again = norm_look_again<kRows, G / 32>(slot, left < kRows ? (int)left : kRows, eps);
  }
  if constexpr (G < 32) again = __any_sync(0xffffffffu, again);  // the warp's rows share shuffles
  if (again) {
    mul = own;
    const uint64_t m2 = f32x2_pack(mul, mul);
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int e = 0; e < kE / 2; ++e) h[i].p[e] = f32x2_mul(h[i].p[e], m2);
    if constexpr (G > 32) __syncthreads();  // the first sums have been read
    sum = row_reduce<G, false>(squares(), slot);
  }
  return rsqrtf(sum / (float)W + own_eps * mul * mul);
}

}  // namespace

// A block's row groups of G threads go through rows gridDim apart, the next
// row's loads on their way while the sum crosses the threads.
// kOut: 0 the tensors' type, 1 e4m3 with a scale a row, 2 e4m3 with a scale for each 128 columns
template <typename T, int G, int kV, int kOut, bool kVec>
__global__ void __launch_bounds__(block_of(G), blocks_of<T, kVec>(G)) norm_fwd(const __grid_constant__ NormParams p) {
  constexpr int kRows = block_of(G) / G;
  constexpr bool kAhead = G < 1024;  // 1024 threads have no registers for a row ahead
  __shared__ float s_sum[2][32], s_max[32];
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  const long long step = (long long)gridDim.x * kRows;
  using C = Columns<G, kVec>;
  Raw<T, G, kVec> rx[kV], rr[kV];
  auto fetch = [&](long long row) {
    const bool real = row < p.rows;
    const long long r = real ? row : 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) rx[i].load(static_cast<const T*>(p.x) + r * p.sx, C::first(i, t), real ? p.W : 0);
    if (p.res)
#pragma unroll
      for (int i = 0; i < kV; ++i) rr[i].load(static_cast<const T*>(p.res) + r * p.sres, C::first(i, t), real ? p.W : 0);
  };
  if constexpr (kAhead) fetch((long long)blockIdx.x * kRows + group);
  int par = 0;
  // the block's row groups make the same number of turns (they share barriers)
  for (long long first = (long long)blockIdx.x * kRows; first < p.rows; first += step, par ^= 1) {
    const long long r = first + group;
    const bool real = r < p.rows;
    Pairs h[kV];
    if constexpr (!kAhead) fetch(r);
#pragma unroll
    for (int i = 0; i < kV; ++i) h[i] = rx[i].get();
    if (p.res)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const Pairs a = rr[i].get();
#pragma unroll
        for (int e = 0; e < 4; ++e) h[i].p[e] = f32x2_add(h[i].p[e], a.p[e]);
      }
    if constexpr (kAhead) fetch(r + step);
    if (p.res_out && real) {
      T* ro = static_cast<T*>(p.res_out) + r * p.sres_out;
#pragma unroll
      for (int i = 0; i < kV; ++i) store_pairs<T, G, kVec>(ro, h[i], C::first(i, t), p.W);
    }
    float mul;
    const float rstd = row_rstd<G, kV>(h, p.W, p.eps, real, p.rows - first, s_sum[par], mul);
    const uint64_t rstd2 = f32x2_pack(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const Pairs w = load_weight<G, kVec>(p.weight, C::first(i, t), p.W);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[i].p[e] = f32x2_mul(f32x2_mul(h[i].p[e], rstd2), w.p[e]);
    }
    if constexpr (kOut == 0) {
      if (real) {
        T* out = static_cast<T*>(p.out) + r * p.sout;
#pragma unroll
        for (int i = 0; i < kV; ++i) store_pairs<T, G, kVec>(out, h[i], C::first(i, t), p.W);
      }
    } else {
      uint8_t* out = static_cast<uint8_t*>(p.out) + r * p.sout;
      if constexpr (kOut == 1) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) m = most_bits(h[i], 0, 4, m);
        const float scale = e4m3_scale(row_reduce<G, true>(__uint_as_float(m), s_max)), inv = __fdividef(1.0f, scale);
        if (real) {
          if (t == 0) p.scales[r] = scale;
#pragma unroll
          for (int i = 0; i < kV; ++i) store_e4m3<G, kVec>(out, h[i], inv, C::first(i, t), p.W);
        }
      } else {
        const int groups = (p.W + 127) / 128;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int col = C::first(i, t);
          if constexpr (kVec || G < 32) {
            // 128 columns: the vectors of 16 neighbours, or the row
            uint32_t m = most_bits(h[i], 0, 4, 0);
#pragma unroll
            for (int o = G < 16 ? G / 2 : 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float scale = e4m3_scale(__uint_as_float(m));
            if (real) {
              if ((t & 15) == 0 && col < p.W) p.scales[r * groups + col / 128] = scale;
              store_e4m3<G, kVec>(out, h[i], __fdividef(1.0f, scale), col, p.W);
            }
          } else {
            // 128 columns: four elements of each lane of a warp
            float scale[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              scale[k] = e4m3_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, most_bits(h[i], 2 * k, 2 * k + 2, 0))));
              const int c0 = col - (int)(threadIdx.x & 31) + 128 * k;
              if (real && (threadIdx.x & 31) == 0 && c0 < p.W) p.scales[r * groups + c0 / 128] = scale[k];
              const float inv = __fdividef(1.0f, scale[k]);
              const uint64_t i2 = f32x2_pack(inv, inv);
              h[i].p[2 * k] = f32x2_mul(h[i].p[2 * k], i2);
              h[i].p[2 * k + 1] = f32x2_mul(h[i].p[2 * k + 1], i2);
            }
            if (real) store_e4m3<G, kVec>(out, h[i], 1.f, col, p.W);
          }
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
    load8<T>(h, x, col, p.W);
    if (res) {
      float a[kE];
      load8<T>(a, res, col, p.W);
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
  if ((mul = norm_rescue(sum, p.eps)) != 1.f) {
    __syncthreads();
    sum = squares();
  }
  const float rstd = rsqrtf(sum / (float)p.W + p.eps * mul * mul);
  auto scaled = [&](int col) {
    float w[kE];
    load8_weight(w, p.weight, col, p.W);
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
    if (p.res_out) store8<T>(static_cast<T*>(p.res_out) + r * p.sres_out, h, col, p.W);
    scaled(col);
    if constexpr (kOut == 0) {
      store8<T>(static_cast<T*>(p.out) + r * p.sout, h, col, p.W);
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
      store8_e4m3(static_cast<uint8_t*>(p.out) + r * p.sout, h, 1.0f / scale, col, p.W);
    }
  }
}

// Backward: a block's row groups of G threads go through rows gridDim apart.
// The next row's loads are on their way while a row's two sums cross the
// threads; each thread keeps the weight's gradient of its own columns over all
// its rows, and a block leaves one partial gradient (fixed order, no atomics).
template <typename T, int G, int kV, bool kVec>
__global__ void __launch_bounds__(block_of(G), G <= 256 ? 2 : 1) norm_bwd(const __grid_constant__ NormBwdParams p) {
  constexpr int kRows = block_of(G) / G;
  constexpr bool kAhead = G < 1024;  // 1024 threads have no registers for a row ahead
  __shared__ float s_sq[32], s_gh[32];
  __shared__ uint64_t s_acc[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? G * kV * kE / 2 : 1];
  const int t = threadIdx.x % G, group = threadIdx.x / G;
  pdl_release();
  using C = Columns<G, kVec>;
  Pairs acc[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i].p[e] = 0;
  Raw<T, G, kVec> rh[kV], rg[kV], rd[kV];
  auto fetch = [&](long long row) {
    const bool real = row < p.rows;
    const long long r = real ? row : 0;
    const int W = real ? p.W : 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      rh[i].load(static_cast<const T*>(p.h) + r * p.sh, C::first(i, t), W);
      rg[i].load(static_cast<const T*>(p.dy) + r * p.sdy, C::first(i, t), W);
      if constexpr (kAhead) rd[i].load(static_cast<const T*>(p.dh) + r * p.sdh, C::first(i, t), p.dh ? W : 0);
    }
  };
  const long long step = (long long)gridDim.x * kRows;
  if constexpr (kAhead) fetch((long long)blockIdx.x * kRows + group);
  // the block's row groups make the same number of turns (they share barriers)
  for (long long first = (long long)blockIdx.x * kRows; first < p.rows; first += step) {
    const long long row = first + group;
    const bool real = row < p.rows;
    Pairs h[kV], g[kV], d[kV];
    if constexpr (!kAhead) fetch(row);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      h[i] = rh[i].get();
      g[i] = rg[i].get();
      if constexpr (kAhead) d[i] = rd[i].get();
    }
    if constexpr (kAhead) fetch(row + step);
    float mul;
    const float rn = row_rstd<G, kV>(h, p.W, p.eps, real, p.rows - first, s_sq, mul);  // h * rn is the normed row
    const uint64_t rn2 = f32x2_pack(rn, rn);
    uint64_t gh = 0;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const Pairs w = load_weight<G, kVec>(p.weight, C::first(i, t), p.W);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[i].p[e] = f32x2_mul(h[i].p[e], rn2);
        acc[i].p[e] = f32x2_fma(g[i].p[e], h[i].p[e], acc[i].p[e]);
        g[i].p[e] = f32x2_mul(g[i].p[e], w.p[e]);
        gh = f32x2_fma(g[i].p[e], h[i].p[e], gh);
      }
    }
    float gh0, gh1;
    f32x2_unpack(gh, gh0, gh1);
    const float c = row_reduce<G, false>(gh0 + gh1, s_gh) / (float)p.W, rstd = rn * mul;
    const uint64_t c2 = f32x2_pack(-c, -c), rstd2 = f32x2_pack(rstd, rstd);
    T* dx = static_cast<T*>(p.dx) + row * p.sdx;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if constexpr (!kAhead) {
        rd[i].load(static_cast<const T*>(p.dh) + row * p.sdh, C::first(i, t), p.dh && real ? p.W : 0);
        d[i] = rd[i].get();
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i].p[e] = f32x2_fma(rstd2, f32x2_fma(h[i].p[e], c2, g[i].p[e]), d[i].p[e]);
      if (real) store_pairs<T, G, kVec>(dx, d[i], C::first(i, t), p.W);
    }
  }
  if (!p.parts) return;
  if constexpr (kRows > 1) {
    if (group > 0)
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_acc[group - 1][(i * 4 + e) * G + t] = acc[i].p[e];
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i].p[e] = f32x2_add(acc[i].p[e], s_acc[k][(i * 4 + e) * G + t]);
  }
  float* dst = p.parts + (long long)blockIdx.x * p.W;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int col = C::first(i, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      f32x2_unpack(acc[i].p[e], a, b);
      if (col + 2 * e * C::kStep < p.W) dst[col + 2 * e * C::kStep] = a;
      if (col + (2 * e + 1) * C::kStep < p.W) dst[col + (2 * e + 1) * C::kStep] = b;
    }
  }
}

// Backward of rows of more than 32768 elements: a block a row, read twice; the
// weight's gradient by norm_dweight_wide from each row's factors (norm_rescue's and 1 / rms).
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
      load8<T>(h, h0, col, p.W);
      load8<T>(g, dy0, col, p.W);
      load8_weight(w, p.weight, col, p.W);
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
  if ((mul = norm_rescue(sq, p.eps)) != 1.f) {
    __syncthreads();
    sums();
  }
  const float rn = rsqrtf(sq / (float)p.W + p.eps * mul * mul), rstd = rn * mul;
  const float c = gh * rn / (float)p.W;
  if (rstds && threadIdx.x == 0) rstds[r] = make_float2(mul, rn);
  for (int col = threadIdx.x * kE; col < p.W; col += G * kE) {
    float d[kE] = {};
    load8<T>(h, h0, col, p.W);
    load8<T>(g, dy0, col, p.W);
    load8_weight(w, p.weight, col, p.W);
    if (p.dh) load8<T>(d, static_cast<const T*>(p.dh) + r * p.sdh, col, p.W);
#pragma unroll
    for (int e = 0; e < kE; ++e) d[e] = fmaf(rstd, g[e] * w[e] - mul * h[e] * rn * c, d[e]);
    store8<T>(static_cast<T*>(p.dx) + r * p.sdx, d, col, p.W);
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

// dweight[col] = sum of the parts, in a fixed order
__global__ void __launch_bounds__(1024) norm_dweight(const float* parts, int n_parts, int W, float* dweight) {
  __shared__ float s[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < W)
#pragma unroll 8
    for (int i = warp; i < n_parts; i += 32) a += parts[(long long)i * W + col];
  s[warp][lane] = a;
  __syncthreads();
  a = s[lane][warp];  // column `warp`: its 32 sums across the lanes
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0 && blockIdx.x * 32 + warp < W) dweight[blockIdx.x * 32 + warp] = a;
}

namespace {

constexpr int kWide = 32768;

// Threads of a row: one vector a thread up to width 256, two up to 16384, then four.
int group_of(int W) {
  int g = 8;
  while (g < 1024 && g * (g < 32 ? 1 : 2) * kE < W) g *= 2;
  return g;
}
int vectors_of(int W, int g) { return W <= g * kE ? 1 : W <= g * 2 * kE ? 2 : 4; }

// Calls f with (G, vectors) as compile-time numbers.
template <typename F>
cudaError_t by_width(int W, F f) {
  const int g = group_of(W), v = vectors_of(W, g);
#define VDN_NORM_CASE(GG)                                                                                  \
  if (g == GG) {                                                                                           \
    if constexpr (GG <= 32)                                                                                \
      if (v == 1) return f(std::integral_constant<int, GG>(), std::integral_constant<int, 1>());           \
    if constexpr (GG == 1024)                                                                              \
      if (v == 4) return f(std::integral_constant<int, GG>(), std::integral_constant<int, 4>());           \
    if constexpr (GG >= 32) return f(std::integral_constant<int, GG>(), std::integral_constant<int, 2>()); \
  }
  VDN_NORM_CASE(8)
  VDN_NORM_CASE(16)
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
    const long long need = (p.rows + rows - 1) / rows;
    if (vec)
      norm_fwd<T, g, v, kOut, true><<<(unsigned)std::min<long long>(need, 148 * blocks_of<T, true>(g)), block, 0, st>>>(p);
    else
      norm_fwd<T, g, v, kOut, false><<<(unsigned)std::min<long long>(need, 148 * blocks_of<T, false>(g)), block, 0, st>>>(p);
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
      (void)rows;
      const unsigned grid = (unsigned)p.n_parts;
      if (vec)
        norm_bwd<T, g, v, true><<<grid, block, 0, st>>>(p);
      else
        norm_bwd<T, g, v, false><<<grid, block, 0, st>>>(p);
      return cudaGetLastError();
    });
  }
  if (e != cudaSuccess || !p.parts) return e;
  return launch_after(norm_dweight, (p.W + 31) / 32, 1024, 0, st, (const float*)p.parts, p.n_parts, p.W, p.dweight);
}

}  // namespace

size_t norm_workspace(long long rows, int W) {
  const int n = norm_parts(rows, W);
  return (size_t)(W > kWide ? norm_factors_at(n, W) + 2 * rows : (long long)n * W) * 4;
}

int norm_parts(long long rows, int W) {
  if (W > kWide) return (int)std::min<long long>(rows, 64);
  const int g = group_of(W), block = block_of(g), per = block / g;
  return (int)std::min<long long>((rows + per - 1) / per, 148 * (block == 256 ? 2 : 1));
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
