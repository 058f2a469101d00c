// lin_step.cu - one token for each of many sequences: the recurrent form of the
// causal linear memory, on a pool of states updated in place.
//
//   S = lambda S + k^T v,   out = scale q S
//
// Bound by memory: the state is read and written once (8 D^2 bytes a row and
// head, against 4 D values of tensors).  A CTA takes a slice of the state's
// columns: column slices need nothing of one another (out's element j is a sum
// over rows of column j), so small batches spread over the SMs without a join.
// A thread owns four columns (16 bytes) of every kRows-th row and keeps them in
// registers from the load to the store; all its loads are in flight at once.
// Measured: 192 x 16 x 128 of a pool of 256 in 68 us as a call, 0.91 of the copy
// rate.
//
// With slots, a CTA looks all of them through for rows that share its own (4 B
// bytes, from L2, once for each of its tokens): B^2 H D / 32 reads in all, which
// are nothing for some hundred rows and outweigh the states from about 64 D rows
// on.  Measured, with slots and without: 700 x 1 x 32 8.5 and 8.9 us, 4096 x 16 x
// 128 2210 and 1245, 20000 x 1 x 32 236 and 28, 65536 x 1 x 32 3870 and 91.
#include "lin_common.cuh"

namespace vdn {
namespace {

constexpr int kStepThreads = 128;

template <typename T>
__device__ __forceinline__ float load1(const void* p, long long i) {
  if constexpr (sizeof(T) == 4)
    return static_cast<const float*>(p)[i];
  else
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace

template <typename T, int D, int kCols>
__global__ void __launch_bounds__(kStepThreads) lin_step(const __grid_constant__ LinStepParams p) {
  constexpr int kQuads = kCols / 4;              // threads of a row
  constexpr int kRows = kStepThreads / kQuads;   // rows at a time
  constexpr int kN = D / kRows;                  // float4s of a thread
  __shared__ float sq[D], sk[D];
  __shared__ float red[kRows][kCols];
  __shared__ int s_next;
  const int tid = threadIdx.x;
  const int slice = blockIdx.x % (D / kCols);
  const long long row = blockIdx.x / (D / kCols);
  const int h = (int)(row % p.H), b0 = (int)(row / p.H);
  const int c0 = slice * kCols + (tid % kQuads) * 4, r0 = tid / kQuads;
  const int slot = p.slots ? p.slots[b0] : b0;
  if (slot < 0 || slot >= p.n_slots) {
    T* o = static_cast<T*>(p.o.p) + b0 * p.o.sb + h * p.o.sh;
    if (tid < kCols) store1(o + slice * kCols + tid, 0.f);
    if (slot >= p.n_slots && p.status && tid == 0) *p.status = 1;  // VDN_ERR_INVALID_ARG
    return;
  }
  float* S = p.pool + slot * p.slot_stride + (long long)h * D * D;
  float4 s[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) s[i] = *reinterpret_cast<const float4*>(S + (r0 + kRows * i) * D + c0);
  const LinFall decayed(p.log_decay[h], 1);
  int b = b0;
  while (true) {
    if (tid == 0) s_next = p.B;
    for (int i = tid; i < D; i += kStepThreads) {
      sq[i] = load1<T>(p.q.p, b * p.q.sb + h * p.q.sh + i);
      sk[i] = load1<T>(p.k.p, b * p.k.sb + h * p.k.sh + i);
    }
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = load1<T>(p.v.p, b * p.v.sb + h * p.v.sh + c0 + e);
    // Rows of the same slot: the first of them takes all, in order.
    bool later = false;
    if (p.slots) {
      int next = p.B;
      for (int i = tid; i < p.B; i += kStepThreads)
        if (i != b && p.slots[i] == slot) {
          if (i < b0) later = true;
          if (i > b) next = min(next, i);
        }
      later = __syncthreads_or(later);
      if (later) return;  // an earlier row has taken this one (seen on the first pass, before any store)
      if (next < p.B) atomicMin(&s_next, next);
    }
    __syncthreads();
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float k = sk[r0 + kRows * i], q = sq[r0 + kRows * i];
      s[i].x = decayed(s[i].x, k * v[0]);
      s[i].y = decayed(s[i].y, k * v[1]);
      s[i].z = decayed(s[i].z, k * v[2]);
      s[i].w = decayed(s[i].w, k * v[3]);
      o[0] = fmaf(q, s[i].x, o[0]);
      o[1] = fmaf(q, s[i].y, o[1]);
      o[2] = fmaf(q, s[i].z, o[2]);
      o[3] = fmaf(q, s[i].w, o[3]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[r0][(tid % kQuads) * 4 + e] = o[e];
    const int next = s_next;
    __syncthreads();
    if (tid < kCols) {
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) sum += red[r][tid];
      store1(static_cast<T*>(p.o.p) + b * p.o.sb + h * p.o.sh + slice * kCols + tid, p.scale * sum);
    }
    if (next >= p.B) break;
    b = next;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) *reinterpret_cast<float4*>(S + (r0 + kRows * i) * D + c0) = s[i];
}

namespace {

template <typename T, int D>
cudaError_t step(const LinStepParams& p, cudaStream_t st) {
  const long long rows = (long long)p.B * p.H;
  lin_step<T, D, 32><<<(unsigned)(rows * (D / 32)), kStepThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_step(const LinStepParams& p, int D, int fp32, cudaStream_t st) {
  if (D == 32) return fp32 ? step<float, 32>(p, st) : step<__nv_bfloat16, 32>(p, st);
  if (D == 64) return fp32 ? step<float, 64>(p, st) : step<__nv_bfloat16, 64>(p, st);
  return fp32 ? step<float, 128>(p, st) : step<__nv_bfloat16, 128>(p, st);
}

}  // namespace vdn
