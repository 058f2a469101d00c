// lin_simt.cu - the causal linear memory on the FMA pipes: fp32 tensors, and
// bf16 tensors of head_dim 32.
//
// A CTA walks its range of 32-row chunks with the state W (D x D, fp32) in
// shared memory.  Per chunk: X, Y, Z rows (converted to fp32) are staged, the
// scores X Y^T are formed, decayed and masked, then out = scores Z + X W and
// W = lambda^n W + (decayed Y)^T Z.  32 rows keep the quadratic part (2 * 32 * D
// multiply-adds a row) at a quarter to a half of the state's (2 * D * D) for D =
// 128 and 64.  Bound by the FMA pipe: fp32 has no tensor-core form that keeps
// fp32's products, which is what a caller of fp32 tensors asks for here.
#include "lin_common.cuh"
#include "pdl.cuh"

namespace vdn {
namespace {

constexpr int kC = kLinSimtChunk;
constexpr int kThreads = 256;

template <int D>
struct SimtLayout {
  static constexpr int kPitch = D + 4;  // X, Y, Z rows: float4 reads of 8 rows at once meet no bank twice
  static constexpr int kTile = kC * kPitch;
  static constexpr int kPP = kC + 1;
  static constexpr int kFloats = 3 * kTile + D * D + kC * kPP + 2 * kC + 4;
  static constexpr int kBytes = kFloats * 4;
};

// rows [row0, row0 + kC) of a view's (b, h) as fp32 into dst, zeros from n_valid on
template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, const LinView& v, int b, int h, int row0, int n_valid) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kPerRow = D / kVec;
  const T* base = static_cast<const T*>(v.p) + b * v.sb + h * v.sh;
  for (int i = threadIdx.x; i < kC * kPerRow; i += kThreads) {
    const int r = i / kPerRow, c = (i - r * kPerRow) * kVec;
    float* d = dst + r * SimtLayout<D>::kPitch + c;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r < n_valid) w = *reinterpret_cast<const uint4*>(base + (long long)(row0 + r) * v.sn + c);
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint4*>(d) = w;
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[2 * e] = __uint_as_float(u[e] << 16);
        d[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// W = decay W + sum_r w[r] Y[r]^T Z[r] over the n real rows
template <int D>
__device__ __forceinline__ void update_state(float* W, const float* Y, const float* Z, const float* w, float decay, int n) {
  constexpr int kT = D / 16;
  constexpr int kPitch = SimtLayout<D>::kPitch;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[kT][kT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) acc[i][j] = 0.f;
  for (int r = 0; r < n; ++r) {
    float y[kT], z[kT];
#pragma unroll
    for (int i = 0; i < kT; ++i) y[i] = w[r] * Y[r * kPitch + ty + 16 * i];
#pragma unroll
    for (int j = 0; j < kT; ++j) z[j] = Z[r * kPitch + tx + 16 * j];
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int j = 0; j < kT; ++j) acc[i][j] = fmaf(y[i], z[j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      float* p = W + (ty + 16 * i) * D + tx + 16 * j;
      *p = fmaf(decay, *p, acc[i][j]);
    }
}

// weights lambda^(n - p - e) of the rows of a chunk (p: place in walk order)
__device__ __forceinline__ void row_weights(float* w, float l2, int n, int reverse) {
  if (threadIdx.x < kC) {
    const int r = threadIdx.x;
    w[r] = r < n ? lin_pow(l2, reverse ? r + 1 : n - 1 - r) : 0.f;
  }
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lin_states_simt(const __grid_constant__ LinStateParams p) {
  using L = SimtLayout<D>;
  extern __shared__ float sm[];
  float *Y = sm, *Z = Y + L::kTile, *W = Z + L::kTile, *w = W + D * D;
  const LinPlan& pl = p.pl;
  const LinWalk& wk = p.walk[blockIdx.y];
  pdl_release();
  const int range = blockIdx.x / pl.sub;
  const int bh = (int)((pl.start(range + 1) - 1) / pl.nc), b = bh / p.H, h = bh % p.H, len = lin_length(p.lengths, b, p.N);
  const float l2 = lin_log2_decay(p.log_decay[h]);
  const LinStretch st = lin_piece_of(lin_stretch(range, len, l2, pl, wk.reverse), blockIdx.x % pl.sub, pl);
  if (st.u0 == st.u1) return;
  for (int i = threadIdx.x; i < D * D; i += kThreads) W[i] = 0.f;
  for (int u = st.u0; u < st.u1; ++u) {
    const int row0 = (wk.reverse ? pl.nc - 1 - u : u) * kC, n = min(max(len - row0, 0), kC);
    __syncthreads();
    load_rows<T, D>(Y, wk.y, b, h, row0, n);
    load_rows<T, D>(Z, wk.z, b, h, row0, n);
    row_weights(w, l2, n, wk.reverse);
    __syncthreads();
    update_state<D>(W, Y, Z, w, lin_pow(l2, n), n);
  }
  __syncthreads();
  const float left = lin_pow(l2, lin_rows(st.u1, st.end, len, pl, wk.reverse));  // decay to the stretch's end
  float* dst = wk.parts + (long long)blockIdx.x * D * D;
  for (int i = threadIdx.x; i < D * D; i += kThreads) dst[i] = left * W[i];
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lin_out_simt(const __grid_constant__ LinOutParams p) {
  using L = SimtLayout<D>;
  extern __shared__ float sm[];
  float *X = sm, *Y = X + L::kTile, *Z = Y + L::kTile, *W = Z + L::kTile, *P = W + D * D, *w = P + kC * L::kPP,
        *pw = w + kC;  // pw[k] = lambda^k, k <= kC
  const LinPlan& pl = p.pl;
  const LinJob& jb = p.job[blockIdx.y];
  const int tid = threadIdx.x, rev = jb.reverse;
  long long t = pl.start(blockIdx.x);
  const long long t_end = pl.start(blockIdx.x + 1);
  pdl_wait();
  while (t < t_end) {
    const LinPiece pc(t, t_end, pl);
    t += pc.u1 - pc.u0;
    const int b = pc.bh / p.H, h = pc.bh % p.H, len = lin_length(p.lengths, b, p.N);
    const float l2 = lin_log2_decay(p.log_decay[h]);
    __syncthreads();
    if (tid <= kC) pw[tid] = lin_pow(l2, tid);
    const float* src = nullptr;
    float mul = 1.f;
    if (pc.u0 > 0) {
      src = jb.s_in + (long long)blockIdx.x * D * D;
    } else if (jb.s_head && pc.u1 < pl.nc) {
      src = jb.s_head + (long long)blockIdx.x * D * D;
    } else if (jb.init) {
      src = jb.init + b * jb.init_stride + (long long)h * D * D;
      mul = jb.init_mul;
    }
    for (int i = tid; i < D * D; i += kThreads)
      W[i] = src ? mul * (jb.transposed ? src[(i % D) * D + i / D] : src[i]) : 0.f;
    for (int u = pc.u0; u < pc.u1; ++u) {
      const int row0 = (rev ? pl.nc - 1 - u : u) * kC;
      const int n_rows = min(p.N - row0, kC), n = min(max(len - row0, 0), kC);
      __syncthreads();
      load_rows<T, D>(X, jb.x, b, h, row0, n);
      load_rows<T, D>(Y, jb.y, b, h, row0, n);
      load_rows<T, D>(Z, jb.z, b, h, row0, n);
      row_weights(w, l2, n, rev);
      __syncthreads();
      // scores: row r, columns c and c + 16, decayed by the rows between, 0 past the row in walk order
      {
        const int c0 = tid & 15, r0 = tid >> 4;
        float acc[2][2] = {};
        for (int k = 0; k < D; k += 4) {
          float4 x[2], y[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[i] = *reinterpret_cast<const float4*>(X + (r0 + 16 * i) * L::kPitch + k);
            y[i] = *reinterpret_cast<const float4*>(Y + (c0 + 16 * i) * L::kPitch + k);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
              acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
              acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
              acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = r0 + 16 * i, c = c0 + 16 * j, gap = rev ? c - r : r - c;
            P[r * L::kPP + c] = gap >= 0 && r < n && c < n ? acc[i][j] * pw[gap] : 0.f;
          }
      }
      __syncthreads();
      {
        constexpr int kCols = D / 4, kRowGroups = kThreads / kCols, kRpt = kC / kRowGroups;
        const int c = (tid % kCols) * 4, r0 = tid / kCols;
        float o[kRpt][4];
#pragma unroll
        for (int i = 0; i < kRpt; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        for (int k = 0; k < D; ++k) {
          const float4 s = *reinterpret_cast<const float4*>(W + k * D + c);
#pragma unroll
          for (int i = 0; i < kRpt; ++i) {
            const float x = X[(r0 + kRowGroups * i) * L::kPitch + k];
            o[i][0] = fmaf(x, s.x, o[i][0]);
            o[i][1] = fmaf(x, s.y, o[i][1]);
            o[i][2] = fmaf(x, s.z, o[i][2]);
            o[i][3] = fmaf(x, s.w, o[i][3]);
          }
        }
#pragma unroll
        for (int i = 0; i < kRpt; ++i) {
          const int r = r0 + kRowGroups * i;
          const float f = r < n ? pw[rev ? n - 1 - r : r + 1] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f;
        }
        for (int k = 0; k < n; ++k) {
          const float4 z = *reinterpret_cast<const float4*>(Z + k * L::kPitch + c);
#pragma unroll
          for (int i = 0; i < kRpt; ++i) {
            const float q = P[(r0 + kRowGroups * i) * L::kPP + k];
            o[i][0] = fmaf(q, z.x, o[i][0]);
            o[i][1] = fmaf(q, z.y, o[i][1]);
            o[i][2] = fmaf(q, z.z, o[i][2]);
            o[i][3] = fmaf(q, z.w, o[i][3]);
          }
        }
        T* out = static_cast<T*>(jb.o.p) + b * jb.o.sb + h * jb.o.sh;
#pragma unroll
        for (int i = 0; i < kRpt; ++i) {
          const int r = r0 + kRowGroups * i;
          if (r >= n_rows) continue;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = r < n ? p.alpha * o[i][e] : 0.f;
          store4(out + (long long)(row0 + r) * jb.o.sn + c, v);
        }
      }
      __syncthreads();
      if (n > 0) update_state<D>(W, Y, Z, w, pw[n], n);
    }
    if (pc.u1 == pl.nc && jb.final_out) {
      __syncthreads();
      float* dst = jb.final_out + b * jb.final_stride + (long long)h * D * D;
      for (int i = tid; i < D * D; i += kThreads)
        dst[jb.transposed ? (i % D) * D + i / D : i] = jb.final_mul * W[i];
    }
  }
}

// State before each range that begins inside a head: s_in[j] = lambda^rows(j - 1)
// s_in[j - 1] + part[j - 1] along the head's ranges, from the state before the
// walk.  A thread owns four elements and goes through the ranges.  Bound by the
// latency of its loads, which do not depend on one another: eight are in flight.
__global__ void __launch_bounds__(128) lin_scan(const __grid_constant__ LinStateParams p, int DD) {
  constexpr int kAhead = 8;
  const LinPlan& pl = p.pl;
  const LinWalk& wk = p.walk[blockIdx.y];
  pdl_release();
  const int per = (DD + 4 * (int)blockDim.x - 1) / (4 * (int)blockDim.x);  // blocks of a head
  const int bh = blockIdx.x / per, b = bh / p.H, h = bh % p.H, sub = pl.sub;
  const long long head0 = (long long)bh * pl.nc;
  const int j0 = pl.range_of(head0), j1 = pl.range_of(head0 + pl.nc - 1);
  if (j1 == j0) return;
  const int len = lin_length(p.lengths, b, p.N);
  const float l2 = lin_log2_decay(p.log_decay[h]);
  // the head's ranges j0 .. j1 - 1: decay over each, and whether the pieces of its part have been written
  __shared__ float fall[kLinMaxGrid];
  __shared__ bool has[kLinMaxGrid * kLinMaxSub];
  const int n = (j1 - j0) * sub;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int j = j0 + i / sub;
    const LinStretch st = lin_piece_of(lin_stretch(j, len, l2, pl, wk.reverse), i % sub, pl);
    has[i] = st.u0 < st.u1;
    if (i % sub == 0)
      fall[i / sub] = lin_pow(l2, lin_rows((int)(max(pl.start(j), head0) - head0), (int)(pl.start(j + 1) - head0), len, pl, wk.reverse));
  }
  __syncthreads();
  pdl_wait();
  const int e = (blockIdx.x % per * blockDim.x + threadIdx.x) * 4;
  if (e >= DD) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (wk.init) {
    s = *reinterpret_cast<const float4*>(wk.init + b * wk.init_stride + (long long)h * DD + e);
    s = make_float4(s.x * wk.init_mul, s.y * wk.init_mul, s.z * wk.init_mul, s.w * wk.init_mul);
  }
  if (wk.s_head) *reinterpret_cast<float4*>(wk.s_head + (long long)j0 * DD + e) = s;
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    float4 a[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < n && has[i0 + i])
        a[i] = *reinterpret_cast<const float4*>(wk.parts + ((long long)j0 * sub + i0 + i) * DD + e);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= n) continue;
      const int k = (i0 + i) / sub;
      if (i0 + i == k * sub) s = make_float4(fall[k] * s.x, fall[k] * s.y, fall[k] * s.z, fall[k] * s.w);
      s = make_float4(s.x + a[i].x, s.y + a[i].y, s.z + a[i].z, s.w + a[i].w);
      if (i0 + i == k * sub + sub - 1) *reinterpret_cast<float4*>(wk.s_in + (long long)(j0 + k + 1) * DD + e) = s;
    }
  }
}

namespace {

template <typename T, int D>
cudaError_t states_simt(const LinStateParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = lin_prepare((const void*)lin_states_simt<T, D>, SimtLayout<D>::kBytes, 0, done);
  if (e != cudaSuccess) return e;
  lin_states_simt<T, D><<<dim3(p.pl.grid * p.pl.sub, p.n_walks), kThreads, SimtLayout<D>::kBytes, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t out_simt(const LinOutParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = lin_prepare((const void*)lin_out_simt<T, D>, SimtLayout<D>::kBytes, 0, done);
  if (e != cudaSuccess) return e;
  if (p.pl.split) return launch_after(lin_out_simt<T, D>, dim3(p.pl.grid, p.n_jobs), kThreads, SimtLayout<D>::kBytes, st, p);
  lin_out_simt<T, D><<<dim3(p.pl.grid, p.n_jobs), kThreads, SimtLayout<D>::kBytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_states_simt(const LinStateParams& p, int D, int fp32, cudaStream_t st) {
  if (D == 32) return fp32 ? states_simt<float, 32>(p, st) : states_simt<__nv_bfloat16, 32>(p, st);
  if (D == 64) return fp32 ? states_simt<float, 64>(p, st) : states_simt<__nv_bfloat16, 64>(p, st);
  return fp32 ? states_simt<float, 128>(p, st) : states_simt<__nv_bfloat16, 128>(p, st);
}

cudaError_t launch_lin_out_simt(const LinOutParams& p, int D, int fp32, cudaStream_t st) {
  if (D == 32) return fp32 ? out_simt<float, 32>(p, st) : out_simt<__nv_bfloat16, 32>(p, st);
  if (D == 64) return fp32 ? out_simt<float, 64>(p, st) : out_simt<__nv_bfloat16, 64>(p, st);
  return fp32 ? out_simt<float, 128>(p, st) : out_simt<__nv_bfloat16, 128>(p, st);
}

cudaError_t launch_lin_scan(const LinStateParams& p, int D, cudaStream_t st) {
  return launch_after(lin_scan, dim3((D * D + 511) / 512 * p.B * p.H, p.n_walks), 128, 0, st, p, D * D);
}

}  // namespace vdn
