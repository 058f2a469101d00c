// lin_simt.cu - the causal linear memory on the FMA pipes: fp32 tensors (and
// bf16 tensors without a TMA view).
//
// A CTA walks its range of 64-row chunks with the state W (D x D, fp32) in
// shared memory.  Per chunk: X, Y, Z rows (as fp32) are staged, the scores X Y^T
// are formed, decayed and masked, then out = scores Z + X W and W = lambda^n W +
// (decayed Y)^T Z.  A tensor-core form that keeps fp32's products would take
// every operand, P and W among them, in three bf16 parts and six products for
// one (271 TFLOP/s of the measured bf16 rate, against 74 of the FMA pipe); it is
// not written.  The kernel is bound by the FMA pipe, at 2 D (2 D + 64 + 32)
// operations a row: 64 rows keep the quadratic part at a quarter (D = 128) to a
// half (64) of it, with the masked blocks of 16 columns and rows behind left out.
// To be bound by it, a thread's tile has to turn each load from shared memory
// into eight operations and more: 8 x 8 of the state and 8 x 4 of the output at
// D = 128.  fp32 rows come by cp.async, the next
// chunk's X while the state is updated.  Measured: 4 x 20000 x 8 x 128 in 1910 us
// (walk 1560, parts 390), about 40 TFLOP/s executed, 22 of the 4 D^2 operations a
// row that the formula needs.
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
  static constexpr int kPP = kC + 4;
  static constexpr int kFloats = 3 * kTile + D * D + kC * kPP + 2 * kC + 4;
  static constexpr int kBytes = kFloats * 4;
  static constexpr int kCtas = D == 128 ? 1 : 2;  // on an SM: shared memory at D = 128, registers
};

// rows [row0, row0 + kC) of a view's (b, h) as fp32 into dst, zeros from n_valid on; fp32 rows are on their way on return
template <typename T, int D>
__device__ __forceinline__ void load_rows(float* dst, const LinView& v, int b, int h, int row0, int n_valid) {
  constexpr int kVec = 16 / sizeof(T);
  constexpr int kPerRow = D / kVec;
  const T* base = static_cast<const T*>(v.p) + b * v.sb + h * v.sh;
#pragma unroll 4
  for (int i = threadIdx.x; i < kC * kPerRow; i += kThreads) {
    const int r = i / kPerRow, c = (i - r * kPerRow) * kVec;
    float* d = dst + r * SimtLayout<D>::kPitch + c;
    const T* src = base + (long long)(row0 + (r < n_valid ? r : 0)) * v.sn + c;
    if constexpr (sizeof(T) == 4) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(d)), "l"(src),
                   "r"(r < n_valid ? 16 : 0)
                   : "memory");
    } else {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < n_valid) w = *reinterpret_cast<const uint4*>(src);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[2 * e] = __uint_as_float(u[e] << 16);
        d[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
  }
}
__device__ __forceinline__ void rows_arrived() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

// A thread's tile of the state: kT x kT elements, in runs of four (two at D = 32) 64 apart, so that the runs of a warp's
// threads are neighbours.
template <int D>
struct StateTile {
  static constexpr int kT = D / 16, kRun = kT < 4 ? kT : 4, kRuns = kT / kRun;
  float a[kT][kT];
  __device__ __forceinline__ static int at(int thread, int i) { return thread * kRun + i / kRun * 64 + i % kRun; }
  __device__ __forceinline__ static void load(float (&f)[kT], const float* p, int thread) {
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      if constexpr (kRun == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + thread * 4 + 64 * k);
        f[4 * k] = v.x, f[4 * k + 1] = v.y, f[4 * k + 2] = v.z, f[4 * k + 3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(p + thread * 2);
        f[0] = v.x, f[1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kT; ++i)
#pragma unroll
      for (int j = 0; j < kT; ++j) a[i][j] = 0.f;
  }
  // a += sum_r w[r] Y[r]^T Z[r] over n rows
  __device__ __forceinline__ void add(const float* Y, const float* Z, const float* w, int n) {
    constexpr int kPitch = SimtLayout<D>::kPitch;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
      float y[kT], z[kT];
      load(y, Y + r * kPitch, ty);
      load(z, Z + r * kPitch, tx);
      const float f = w[r];
#pragma unroll
      for (int i = 0; i < kT; ++i) y[i] *= f;
#pragma unroll
      for (int i = 0; i < kT; ++i)
#pragma unroll
        for (int j = 0; j < kT; ++j) a[i][j] = fmaf(y[i], z[j], a[i][j]);
    }
  }
};

// weights lambda^(n - p - e) of the rows of a chunk (p: place in walk order)
__device__ __forceinline__ void row_weights(float* w, float l2, int n, int reverse) {
  if (threadIdx.x < kC) {
    const int r = threadIdx.x;
    w[r] = r < n ? lin_pow(l2, reverse ? r + 1 : n - 1 - r) : 0.f;
  }
}

// P = scores, decayed by the rows between and 0 past the row in walk order: 4 x 4 a thread, rows and columns 16 apart, so
// that whole blocks of 16 x 16 fall to the mask and are left out.
template <int D, bool kRev>
__device__ __forceinline__ void scores(float* P, const float* X, const float* Y, const float* pw, int n) {
  using L = SimtLayout<D>;
  const int c0 = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  float acc[4][4] = {};
#pragma unroll 2
  for (int k = 0; k < D; k += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = *reinterpret_cast<const float4*>(X + (r0 + 16 * i) * L::kPitch + k);
      y[i] = *reinterpret_cast<const float4*>(Y + (c0 + 16 * i) * L::kPitch + k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kRev ? j < i : j > i) continue;
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + 16 * i, c = c0 + 16 * j, gap = kRev ? c - r : r - c;
      P[r * L::kPP + c] = gap >= 0 && r < n && c < n ? acc[i][j] * pw[gap] : 0.f;
    }
}

// o[i] += sum_k A[row i][k] B[k][4 columns], k0 <= k < k1 (multiples of 4); A's rows are the same for a warp's neighbours
template <int kR>
__device__ __forceinline__ void rows_times(float (&o)[kR][4], const float* A, int a_pitch, const float* B, int b_pitch, int k0,
                                           int k1) {
#pragma unroll 2
  for (int k = k0; k < k1; k += 4) {
    float4 a[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) a[i] = *reinterpret_cast<const float4*>(A + i * a_pitch + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 v = *reinterpret_cast<const float4*>(B + (k + e) * b_pitch);
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float f = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
        o[i][0] = fmaf(f, v.x, o[i][0]);
        o[i][1] = fmaf(f, v.y, o[i][1]);
        o[i][2] = fmaf(f, v.z, o[i][2]);
        o[i][3] = fmaf(f, v.w, o[i][3]);
      }
    }
  }
}

}  // namespace

// A range's part, in pieces (linear.h); the state stays in registers.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lin_states_simt(const __grid_constant__ LinStateParams p) {
  using L = SimtLayout<D>;
  extern __shared__ float sm[];
  float *Y = sm, *Z = Y + L::kTile, *w = Z + L::kTile;
  const LinPlan& pl = p.pl;
  const LinWalk& wk = p.walk[blockIdx.y];
  pdl_release();
  const int range = blockIdx.x / pl.sub;
  const LinCuts cuts(pl, p.lengths, p.B, p.H, p.N, wk.reverse);
  const long long t0 = cuts.start(range), t1 = cuts.start(range + 1);
  const int bh = (int)((t1 - 1) / pl.nc), b = bh / p.H, h = bh % p.H, len = lin_length(p.lengths, b, p.N);
  const long long head0 = (long long)bh * pl.nc;
  const float log_decay = p.log_decay[h], l2 = lin_log2_decay(log_decay);
  const LinStretch st = lin_piece_of(lin_stretch((int)(max(t0, head0) - head0), (int)(t1 - head0), len, l2, pl, wk.reverse), blockIdx.x % pl.sub, pl);
  if (st.u0 == st.u1) return;
  LinFactors whole(log_decay, kC);
  StateTile<D> W;
  W.zero();
  for (int u = st.u0; u < st.u1; ++u) {
    const int row0 = (wk.reverse ? pl.nc - 1 - u : u) * kC, n = min(max(len - row0, 0), kC);
    __syncthreads();
    load_rows<T, D>(Y, wk.y, b, h, row0, n);
    load_rows<T, D>(Z, wk.z, b, h, row0, n);
    row_weights(w, l2, n, wk.reverse);
    const float fall = n == kC ? whole.next() : lin_pow(l2, n);
#pragma unroll
    for (int i = 0; i < W.kT; ++i)
#pragma unroll
      for (int j = 0; j < W.kT; ++j) W.a[i][j] *= fall;
    rows_arrived();
    W.add(Y, Z, w, n);
  }
  const float left = lin_pow(l2, lin_rows(st.u1, st.end, len, pl, wk.reverse));  // decay to the stretch's end
  float* dst = wk.parts + (long long)blockIdx.x * D * D;
#pragma unroll
  for (int i = 0; i < W.kT; ++i)
#pragma unroll
    for (int j = 0; j < W.kT; ++j) dst[W.at(threadIdx.x >> 4, i) * D + W.at(threadIdx.x & 15, j)] = left * W.a[i][j];
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
  // output tile of a thread: kR rows of four columns
  constexpr int kQuads = D / 4, kR = kC / (kThreads / kQuads);
  const int c = tid % kQuads * 4, r0 = tid / kQuads * kR;
  const LinCuts cuts(pl, p.lengths, p.B, p.H, p.N, rev);
  long long t = cuts.start(blockIdx.x);
  const long long t_end = cuts.start(blockIdx.x + 1);
  pdl_wait();
  while (t < t_end) {
    const LinPiece pc(t, t_end, pl);
    t += pc.u1 - pc.u0;
    const int b = pc.bh / p.H, h = pc.bh % p.H, len = lin_length(p.lengths, b, p.N);
    const float log_decay = p.log_decay[h], l2 = lin_log2_decay(log_decay);
    LinFactors whole(log_decay, kC);
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
    auto first_row = [&](int u) { return (rev ? pl.nc - 1 - u : u) * kC; };
    auto rows_of = [&](int u) { return min(max(len - first_row(u), 0), kC); };
    load_rows<T, D>(X, jb.x, b, h, first_row(pc.u0), rows_of(pc.u0));
    load_rows<T, D>(Y, jb.y, b, h, first_row(pc.u0), rows_of(pc.u0));
    load_rows<T, D>(Z, jb.z, b, h, first_row(pc.u0), rows_of(pc.u0));
    for (int u = pc.u0; u < pc.u1; ++u) {
      const int row0 = first_row(u), n_rows = min(p.N - row0, kC), n = rows_of(u);
      row_weights(w, l2, n, rev);
      rows_arrived();
      if (n > 0) {
        if (rev)
          scores<D, true>(P, X, Y, pw, n);
        else
          scores<D, false>(P, X, Y, pw, n);
      }
      __syncthreads();
      float o[kR][4];
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
      if (n > 0) {
        rows_times<kR>(o, X + r0 * L::kPitch, L::kPitch, W + c, D, 0, D);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          const int r = r0 + i;
          const float f = r < n ? pw[rev ? n - 1 - r : r + 1] : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= f;
        }
        // columns of P that these rows see
        rows_times<kR>(o, P + r0 * L::kPP, L::kPP, Z + c, L::kPitch, rev ? r0 / 4 * 4 : 0,
                       rev ? (n + 3) / 4 * 4 : min((r0 + kR + 3) / 4 * 4, (n + 3) / 4 * 4));
      }
      T* out = static_cast<T*>(jb.o.p) + b * jb.o.sb + h * jb.o.sh;
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int r = r0 + i;
        if (r >= n_rows) continue;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = r < n ? p.alpha * o[i][e] : 0.f;
        store4(out + (long long)(row0 + r) * jb.o.sn + c, v);
      }
      __syncthreads();
      const bool more = u + 1 < pc.u1;
      if (more) load_rows<T, D>(X, jb.x, b, h, first_row(u + 1), rows_of(u + 1));
      if (n > 0) {
        StateTile<D> S;
        S.zero();
        S.add(Y, Z, w, n);
        const float fall = n == kC ? whole.next() : pw[n];
#pragma unroll
        for (int i = 0; i < S.kT; ++i)
#pragma unroll
          for (int j = 0; j < S.kT; ++j) {
            float* q = W + S.at(tid >> 4, i) * D + S.at(tid & 15, j);
            *q = fmaf(fall, *q, S.a[i][j]);
          }
      }
      __syncthreads();
      if (more) {
        load_rows<T, D>(Y, jb.y, b, h, first_row(u + 1), rows_of(u + 1));
        load_rows<T, D>(Z, jb.z, b, h, first_row(u + 1), rows_of(u + 1));
      }
    }
    if (pc.u1 == pl.nc && jb.final_out) {
      float* dst = jb.final_out + b * jb.final_stride + (long long)h * D * D;
      for (int i = tid; i < D * D; i += kThreads)
        dst[jb.transposed ? (i % D) * D + i / D : i] = jb.final_mul * W[i];
    }
  }
}

// State before each range that begins inside a head: s_in[j] = lambda^rows(j - 1)
// s_in[j - 1] + part[j - 1] along the head's ranges, from the state before the
// walk.  A thread owns kE elements and goes through the ranges.  Bound by the
// latency of its loads, which do not depend on one another: 8 or 16 are in
// flight.  Few heads take one element a thread, for more threads (four heads of
// 128 x 128 in 148 pieces each: 45 us with four, which suffice from some hundred
// threads an SM on).
template <int kE>
__global__ void __launch_bounds__(128) lin_scan(const __grid_constant__ LinStateParams p, int DD) {
  constexpr int kAhead = kE == 4 ? 8 : 16;
  const LinPlan& pl = p.pl;
  const LinWalk& wk = p.walk[blockIdx.y];
  pdl_release();
  const int per = (DD + kE * (int)blockDim.x - 1) / (kE * (int)blockDim.x);  // blocks of a head
  const int bh = blockIdx.x / per, b = bh / p.H, h = bh % p.H, sub = pl.sub, lg = sub == 4 ? 2 : sub - 1;
  const LinCuts cuts(pl, p.lengths, p.B, p.H, p.N, wk.reverse);
  const LinCuts::Head head = cuts.head(bh);
  const int j0 = head.first, j1 = head.last;
  if (j1 == j0) return;
  const int len = lin_length(p.lengths, b, p.N);
  const float log_decay = p.log_decay[h], l2 = lin_log2_decay(log_decay);
  // the head's ranges j0 .. j1 - 1: decay over each, and whether the pieces of its part have been written
  __shared__ float2 fall[kLinMaxGrid];
  __shared__ bool has[kLinMaxGrid * kLinMaxSub];
  const int n = (j1 - j0) * sub;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int j = j0 + (i >> lg);
    const int u0 = cuts.start_in(head, bh, j), u1 = cuts.start_in(head, bh, j + 1);
    const LinStretch st = lin_piece_of(lin_stretch(u0, u1, len, l2, pl, wk.reverse), i & (sub - 1), pl);
    has[i] = st.u0 < st.u1;
    if ((i & (sub - 1)) == 0) {
      const LinFall f(log_decay, lin_rows(u0, u1, len, pl, wk.reverse));
      fall[i >> lg] = make_float2(f.m, f.base);
    }
  }
  __syncthreads();
  pdl_wait();
  const int e = (blockIdx.x % per * blockDim.x + threadIdx.x) * kE;
  if (e >= DD) return;
  auto load = [](float (&f)[kE], const float* q) {
    if constexpr (kE == 4) {
      const float4 v = *reinterpret_cast<const float4*>(q);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
      f[0] = *q;
    }
  };
  auto store = [](float* q, const float (&f)[kE]) {
    if constexpr (kE == 4)
      *reinterpret_cast<float4*>(q) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *q = f[0];
  };
  float s[kE] = {};
  if (wk.init) {
    load(s, wk.init + b * wk.init_stride + (long long)h * DD + e);
#pragma unroll
    for (int x = 0; x < kE; ++x) s[x] *= wk.init_mul;
  }
  if (wk.s_head) store(wk.s_head + (long long)j0 * DD + e, s);
  for (int i0 = 0; i0 < n; i0 += kAhead) {
    float a[kAhead][kE] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < n && has[i0 + i]) load(a[i], wk.parts + ((long long)j0 * sub + i0 + i) * DD + e);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= n) continue;
      const int k = (i0 + i) >> lg, part = (i0 + i) & (sub - 1);
      const LinFall f(part == 0 ? fall[k] : make_float2(1.f, 0.f));
#pragma unroll
      for (int x = 0; x < kE; ++x) s[x] = f(s[x], a[i][x]);
      if (part == sub - 1) store(wk.s_in + (long long)(j0 + k + 1) * DD + e, s);
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

int lin_simt_ctas(int D) {
  return kLinSms * (D == 32 ? SimtLayout<32>::kCtas : D == 64 ? SimtLayout<64>::kCtas : SimtLayout<128>::kCtas);
}

cudaError_t launch_lin_scan(const LinStateParams& p, int D, cudaStream_t st) {
  const int DD = D * D, heads = p.B * p.H;
  if ((long long)DD / 4 * heads * p.n_walks >= kLinSms * 512)
    return launch_after(lin_scan<4>, dim3((DD + 511) / 512 * heads, p.n_walks), 128, 0, st, p, DD);
  return launch_after(lin_scan<1>, dim3((DD + 127) / 128 * heads, p.n_walks), 128, 0, st, p, DD);
}

}  // namespace vdn
