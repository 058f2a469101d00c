// linear.h - plan, parameter blocks and host launchers of the causal linear
// memory with a decay for each head (vdn_linear_attn_fwd / _bwd / _step).
//
// All four results of the forward and backward calls are one operation, a
// "job", with the tensors in other roles.  With rows taken in walk order (token
// order, or its reverse):
//
//   o_i = alpha sum_{j <= i} lambda^(i-j) (x_i . y_j) z_j + factor_i x_i W,
//
//   result   walk      x      y      z      state W before the walk
//   out      forward   q      k      v      state_in
//   dq       forward   d_out  v      k      state_in, transposed
//   dk       reverse   v      d_out  q      d_state_out / alpha, transposed
//   dv       reverse   k      q      d_out  d_state_out / alpha
//
// (alpha = scale).  Split at chunk ends: with n rows in the chunk, p = 0..n-1
// the row's place in walk order and W the state before it,
//
//   factor of row p on W:  alpha lambda^(p + e),       e = 1 forward, 0 reverse
//   W after the chunk:     lambda^n W + sum_p lambda^(n - p - e) y_p^T z_p
//
// which needs no division by lambda: the reverse walk carries lambda R instead
// of R, so that the gradient by state_in is alpha times the last W.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "plan.h"

namespace vdn {

constexpr int kLinSms = 148;          // CTAs a wave holds (one for each SM of a B200)
constexpr int kLinMaxGrid = 2 * kLinSms;  // most ranges of a split plan
constexpr int kLinMaxSub = 4;             // most pieces of a range's part
constexpr int kLinCutBatch = 32;          // most sequences that ranges are cut by the lengths of (LinCuts): a warp's lanes
constexpr int kLinSimtChunk = 64;     // rows of a chunk: fp32 kernels
constexpr int kLinTcChunk = 128;      // rows of a chunk: tensor-core kernels

struct LinView {
  void* p;
  long long sb, sn, sh;  // elements
};

// TMA view of a tensor; the coordinates of a broadcast dimension (or one of a single entry) are multiplied by 0.
struct LinMap {
  CUtensorMap map;
  int mh, mb;
};
struct LinTcMaps {
  LinMap m[7];  // the call's inputs, then its outputs
};

// The chunks of every (batch, head), (batch, head)-major and in walk order,
// form one list; CTA j takes [start(j), start(j + 1)): whole heads, as many as
// make one wave of CTAs, or equal parts (by cost where sequences have lengths:
// LinCuts).  Where a range begins
// inside a head, the state before it is the sum of what the earlier ranges of
// that head leave: each range's own share ("part") is formed by a first kernel,
// a scan over the ranges adds them up, and the walk starts from the result.
struct LinPlan {
  int chunk;        // rows of a chunk
  int nc;           // chunks of a head
  int grid;         // ranges
  int split;        // a range may begin inside a head
  int sub;          // pieces of a range's part, each formed by itself: 1, 2 or 4
  long long total;  // chunks of all heads

  VDN_HD long long start(int j) const { return split ? total * j / grid : total / nc * j / grid * nc; }
  // the range that holds chunk t of the list (equal parts)
  VDN_HD int range_of(long long t) const { return (int)(((t + 1) * grid + total - 1) / total - 1); }
};

// Real rows of the chunks [u0, u1) (walk order) of a head with n tokens.
VDN_HD int lin_rows(int u0, int u1, int n, const LinPlan& pl, int reverse) {
  const int lo = reverse ? pl.nc - u1 : u0, hi = reverse ? pl.nc - u0 : u1;
  const long long most = (long long)(hi - lo) * pl.chunk, have = (long long)n - (long long)lo * pl.chunk;
  return (int)(have < 0 ? 0 : have < most ? have : most);
}

// The chunks that carry the part of range j (walk order): the range's last stretch, if its head goes on behind it, from
// where a token's decay to the stretch's end is not 0 in fp32; piece i of it.  Empty: u0 == u1.
struct LinStretch {
  int u0, u1, end;
};

struct LinJob {
  LinView x, y, z, o;
  int mx, my, mz, mo;    // x, y, z, o among the call's maps
  int reverse;
  int transposed;        // the states in memory are [z][y] for this job
  const float* init;     // state before the walk or null; entries init_stride apart, [H, D, D] each
  long long init_stride;
  float init_mul;
  const float* s_in;     // [grid, D, D]: state before range j (natural orientation of its walk)
  const float* s_head;   // [grid, D, D] or null: copies of `init` for the head that range j begins and does not
                         // end (its last range may overwrite `init`: state_out may be state_in)
  float* final_out;      // state after the walk, or null
  long long final_stride;
  float final_mul;
};

struct LinOutParams {
  LinPlan pl;
  int B, N, H, d, n_jobs;
  float alpha;
  const float* log_decay;
  const int* lengths;
  int* status;
  int* record;
  int inject_timeout;
  LinJob job[3];
};

// One walk's states: parts of the ranges, then their scan.
struct LinWalk {
  LinView y, z;
  int my, mz;
  int reverse;
  float* parts;        // [grid, sub, D, D]; a piece without weight is not written
  float* s_in;         // [grid, D, D]
  float* s_head;       // [grid, D, D] or null (LinJob::s_head)
  const float* init;
  long long init_stride;
  float init_mul;
};

struct LinStateParams {
  LinPlan pl;
  int B, N, H, d, n_walks;
  const float* log_decay;
  const int* lengths;
  int* status;
  int* record;
  LinWalk walk[2];
};

struct LinStepParams {
  LinView q, k, v, o;
  int B, H;
  float scale;
  const float* log_decay;
  float* pool;
  long long slot_stride;
  const int* slots;
  int n_slots;
  int* status;
};

// Sets a kernel's shared memory once on each device (the attribute belongs to the device's copy of the kernel) and checks
// that it takes at least min_regs registers a thread there.
cudaError_t lin_prepare(const void* kernel, int smem_bytes, int min_regs, std::atomic<unsigned long long>& done);

// fp32: 1 for fp32 tensors, 0 for bf16
cudaError_t launch_lin_states_simt(const LinStateParams& p, int D, int fp32, cudaStream_t st);
cudaError_t launch_lin_states_tc(const LinTcMaps& m, const LinStateParams& p, cudaStream_t st);
cudaError_t launch_lin_out_tc(const LinTcMaps& m, const LinOutParams& p, cudaStream_t st);
bool make_lin_map(LinMap* m, const LinView& v, int B, int N, int H, int d, bool output);
int lin_simt_ctas(int D);  // CTAs of launch_lin_out_simt that run at once
cudaError_t launch_lin_scan(const LinStateParams& p, int D, cudaStream_t st);
cudaError_t launch_lin_out_simt(const LinOutParams& p, int D, int fp32, cudaStream_t st);
cudaError_t launch_lin_step(const LinStepParams& p, int D, int fp32, cudaStream_t st);

}  // namespace vdn
