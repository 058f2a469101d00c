// lin_api.cu - host side of the causal linear memory and of the residual
// RMSNorm: argument checks, the plan of ranges, workspace layout, launches
// (declared in include/vdnattn.h).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "linear.h"
#include "norm.h"
#include "vdnattn.h"

namespace vdn {
namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
vdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA; }

// `step`: cfg->tokens is not read.
vdn_status check_linear(const vdn_linear_cfg* c, bool step = false) {
  if (!c) return VDN_ERR_INVALID_ARG;
  const int tokens = step ? 1 : c->tokens;
  if (c->batch < 1 || tokens < 0 || c->heads < 1) return VDN_ERR_INVALID_ARG;
  if (!(c->scale <= 0.f) && !std::isnormal(c->scale)) return VDN_ERR_INVALID_ARG;
  if (c->debug_flags & ~(VDN_POISON_WS | VDN_INJECT_TIMEOUT)) return VDN_ERR_INVALID_ARG;
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return VDN_ERR_UNSUPPORTED;
  if (c->dtype != VDN_BF16 && c->dtype != VDN_FP32) return VDN_ERR_UNSUPPORTED;
  // row coordinates and counts of (batch, head) pairs are 32-bit
  if (c->heads > 4096 || (long long)c->batch * c->heads >= (1ll << 24) || tokens >= (1 << 30))
    return VDN_ERR_UNSUPPORTED;
  return VDN_OK;
}

long long state_size(const vdn_linear_cfg* c) { return (long long)c->heads * c->head_dim * c->head_dim; }

vdn_status check_state(const vdn_linear_cfg* c, const float* p, long long stride) {
  if (!p) return VDN_OK;
  if (!aligned(p, 16) || stride % 4) return VDN_ERR_ALIGNMENT;
  if (stride != 0 && stride < state_size(c)) return VDN_ERR_INVALID_ARG;
  return VDN_OK;
}

vdn_status check_common(const vdn_linear_cfg* c) {
  if (!c->log_decay) return VDN_ERR_INVALID_ARG;
  if (!aligned(c->log_decay, 4) || !aligned(c->lengths, 4) || !aligned(c->slots, 4) || !aligned(c->status_word, 4))
    return VDN_ERR_ALIGNMENT;
  return VDN_OK;
}

// An output that is an input (any other overlap is the caller's to avoid).
bool same_data(std::initializer_list<const vdn_view*> outputs, std::initializer_list<const vdn_view*> inputs) {
  for (const vdn_view* o : outputs)
    for (const vdn_view* x : inputs)
      if (o->data == x->data) return true;
  return false;
}

// A tensor's view: `step`: the token stride is not used.
vdn_status check_view(const vdn_linear_cfg* c, const vdn_view* v, bool output, bool step = false) {
  if (!v || !v->data) return VDN_ERR_INVALID_ARG;
  const long long e = c->dtype == VDN_FP32 ? 4 : 2;
  const long long s[3] = {v->batch_stride, step ? 0 : v->token_stride, v->head_stride};
  const long long n[3] = {c->batch, step ? 1 : c->tokens, c->heads};
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0 || s[i] >= (1ll << 36)) return VDN_ERR_INVALID_ARG;
    if (output && s[i] == 0 && n[i] > 1) return VDN_ERR_INVALID_ARG;
  }
  if (!aligned(v->data, 16)) return VDN_ERR_ALIGNMENT;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && s[i] * e % 16) return VDN_ERR_ALIGNMENT;
  return VDN_OK;
}

LinView view(const vdn_view* v) {
  return LinView{v->data, v->batch_stride, v->token_stride, v->head_stride};
}

// ---------------------------------------------------------------- plan and workspace

// bf16 goes to the tensor cores.  A tensor whose tokens are one broadcast row (token stride 0) has no TMA view: such a
// call, which has no use of its own, takes the kernels of fp32.
bool on_tensor_cores(const vdn_linear_cfg* c, std::initializer_list<const vdn_view*> inputs) {
  if (c->dtype != VDN_BF16) return false;
  for (const vdn_view* v : inputs)
    if (c->tokens > 1 && v->token_stride == 0) return false;
  return true;
}

// Ranges: whole heads, or equal parts of all heads' chunks, which cost a kernel for the parts' states (half of a job's work,
// for `walks` states), the scan and two launches.  Which is shorter, in chunks of a CTA:
//
// bf16: parts as if states were formed over all chunks, and 5 (6 at head_dim 128) for scan and launches (with 8, eight heads
// of 1000 tokens took 26.9 us instead of 17.6; with 4, 64 heads of 2048 took 56.8 instead of 45.8).
// fp32: states are formed over the stretches of ranges that end inside a head only, which is counted (20 x 2000 x 15 x 128:
// 1621 us in parts, 2092 in heads; the bf16 kernels, bound by memory and latency, took 1.05-1.25 times as long for
// 150 to 400 heads with it).  Where two CTAs share an SM, a chunk of one alone takes 0.65 to 0.75 of the time (9.5 us and
// 15 at head_dim 64).
//
// Sequences of a padded batch are taken to fill three quarters of it, which parts make use of (LinCuts) and whole heads do
// not: gradients at 4 x 3840 x 16 x 128 take 213 us in whole heads whatever the lengths, in parts 128 to 228 us.
LinPlan make_plan(const vdn_linear_cfg* c, int jobs, int walks, bool tc, bool padded) {
  LinPlan pl;
  pl.chunk = tc ? kLinTcChunk : kLinSimtChunk;
  pl.nc = std::max(1, (c->tokens + pl.chunk - 1) / pl.chunk);
  const long long heads = (long long)c->batch * c->heads;
  pl.total = heads * pl.nc;
  const int per_wave = tc ? kLinSms : lin_simt_ctas(c->head_dim);
  const int most = per_wave / jobs;
  const long long work = padded && c->batch <= kLinCutBatch ? pl.total - pl.total / 4 : pl.total;
  if (tc) {
    const long long whole = (heads + most - 1) / most * pl.nc;
    pl.split = (work * (2 * jobs + walks) + 2 * per_wave - 1) / (2 * per_wave) + (c->head_dim == 128 ? 6 : 5) < whole;
  } else {
    const double alone = per_wave == kLinSms ? 1.0 : c->head_dim == 64 ? 0.65 : 0.75;
    auto pace = [&](long long ctas) { return ctas * jobs <= kLinSms ? alone : 1.0; };
    const double nc = pl.nc, range = (double)((work + most - 1) / most);
    const double whole = nc * ((heads - 1) / most + pace((heads - 1) % most + 1));
    const double stretch = range < nc ? range * (1.0 - range / (2.0 * nc)) : 0.5 * nc;
    pl.split = (range + 0.5 * walks / jobs * stretch) * pace(std::min<long long>(most, pl.total)) + 1.6 < whole;
  }
  pl.grid = (int)std::min<long long>(most, pl.split ? pl.total : heads);
  // a range's part in one, two or four pieces, of eight chunks at least
  const long long eights = pl.split ? pl.total / pl.grid / 8 : 1;
  pl.sub = eights >= 4 ? kLinMaxSub : eights >= 2 ? 2 : 1;
  return pl;
}

struct LinLayout {
  size_t parts[2], s_in[2], s_head, total;
};

LinLayout make_layout(const vdn_linear_cfg* c, const LinPlan& pl, int walks, bool head_copies) {
  LinLayout l;
  size_t off = 256;  // status slot: word 0 the status, the timeout record at byte 64
  const size_t n = pl.split ? align_up((size_t)pl.grid * c->head_dim * c->head_dim * 4, 256) : 0;  // a state of each range
  for (int i = 0; i < walks; ++i) {
    l.parts[i] = off;
    off += n * pl.sub;
    l.s_in[i] = off;
    off += n;
  }
  l.s_head = off;
  if (head_copies) off += n;
  l.total = off;
  return l;
}

vdn_status check_ws(const vdn_linear_cfg* c, size_t need) {
  if (!c->workspace || c->workspace_bytes < need) return VDN_ERR_WORKSPACE;
  return aligned(c->workspace, 256) ? VDN_OK : VDN_ERR_ALIGNMENT;
}

template <typename T = float>
T* ws(const vdn_linear_cfg* c, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(c->workspace) + off);
}

float scale_of(const vdn_linear_cfg* c) {
  return c->scale > 0.f ? c->scale : 1.0f / std::sqrt((float)c->head_dim);
}

cudaError_t poison(const vdn_linear_cfg* c, size_t total, cudaStream_t st) {
  if (!(c->debug_flags & VDN_POISON_WS) || total <= 256) return cudaSuccess;
  return cudaMemsetAsync(ws<uint8_t>(c, 256), 0xFF, total - 256, st);
}

// dst = src (or 0) for whole states: sequences without tokens
cudaError_t copy_states(const vdn_linear_cfg* c, float* dst, long long dst_stride, const float* src,
                        long long src_stride, cudaStream_t st) {
  if (!dst) return cudaSuccess;
  if (src == dst) return cudaSuccess;
  const size_t row = (size_t)state_size(c) * 4;
  const long long most_pitch = INT32_MAX / 4;  // of the 2D calls, in elements
  if (dst_stride <= most_pitch && (!src || src_stride <= most_pitch))
    return src ? cudaMemcpy2DAsync(dst, (size_t)dst_stride * 4, src, (size_t)src_stride * 4, row, (size_t)c->batch,
                                   cudaMemcpyDeviceToDevice, st)
               : cudaMemset2DAsync(dst, (size_t)dst_stride * 4, 0, row, (size_t)c->batch, st);
  cudaError_t e = cudaSuccess;
  for (int b = 0; b < c->batch && e == cudaSuccess; ++b)
    e = src ? cudaMemcpyAsync(dst + b * dst_stride, src + b * src_stride, row, cudaMemcpyDeviceToDevice, st)
            : cudaMemsetAsync(dst + b * dst_stride, 0, row, st);
  return e;
}

// The launches of a call; the jobs and walks name its tensors by their place, inputs first.
cudaError_t run(const vdn_linear_cfg* c, bool tc, std::initializer_list<const vdn_view*> inputs,
                std::initializer_list<const vdn_view*> outputs, LinStateParams& sp, LinOutParams& op, cudaStream_t st) {
  const int fp32 = c->dtype == VDN_FP32, D = c->head_dim;
  LinTcMaps maps;
  if (tc) {
    int i = 0;
    for (const vdn_view* v : inputs)
      if (!make_lin_map(&maps.m[i++], view(v), c->batch, c->tokens, c->heads, D, false)) return cudaErrorInvalidValue;
    for (const vdn_view* v : outputs)
      if (!make_lin_map(&maps.m[i++], view(v), c->batch, c->tokens, c->heads, D, true)) return cudaErrorInvalidValue;
  }
  if (op.pl.split) {
    cudaError_t e = tc ? launch_lin_states_tc(maps, sp, st) : launch_lin_states_simt(sp, D, fp32, st);
    if (e == cudaSuccess) e = launch_lin_scan(sp, D, st);
    if (e != cudaSuccess) return e;
  }
  return tc ? launch_lin_out_tc(maps, op, st) : launch_lin_out_simt(op, D, fp32, st);
}

}  // namespace
}  // namespace vdn

using namespace vdn;

extern "C" {

vdn_status vdn_linear_validate(const vdn_linear_cfg* cfg) { return check_linear(cfg); }

size_t vdn_linear_workspace_bytes(const vdn_linear_cfg* cfg, int32_t backward) {
  if (check_linear(cfg) != VDN_OK) return 0;
  // either form of the kernels may serve a bf16 call; lengths may be set or not
  size_t most = 0;
  for (bool tc : {false, true})
    for (bool padded : {false, true}) {
      const LinPlan pl = backward ? make_plan(cfg, 3, 2, tc, padded) : make_plan(cfg, 1, 1, tc, padded);
      most = std::max(most, make_layout(cfg, pl, backward ? 2 : 1, !backward).total);
    }
  return most;
}

vdn_status vdn_linear_attn_fwd(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* out,
                               const vdn_linear_cfg* cfg, void* stream) {
  NvtxRange nvtx("vdn:linear_attn_fwd");
  vdn_status s = check_linear(cfg);
  if (s == VDN_OK) s = check_common(cfg);
  if (s == VDN_OK) s = check_state(cfg, cfg->state_in, cfg->state_in_stride);
  if (s == VDN_OK) s = check_state(cfg, cfg->state_out, cfg->state_out_stride);
  if (s != VDN_OK) return s;
  const long long full = state_size(cfg);
  const long long in_stride = cfg->state_in_stride ? cfg->state_in_stride : full;
  const long long out_stride = cfg->state_out_stride ? cfg->state_out_stride : full;
  if (cfg->state_in && cfg->state_in == cfg->state_out && in_stride != out_stride) return VDN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cfg->tokens > 0) {
    for (const vdn_view* x : {q, k, v})
      if ((s = check_view(cfg, x, false)) != VDN_OK) return s;
    if ((s = check_view(cfg, out, true)) != VDN_OK) return s;
  }
  const bool tc = cfg->tokens > 0 && on_tensor_cores(cfg, {q, k, v});
  const LinPlan pl = make_plan(cfg, 1, 1, tc, cfg->lengths);
  const LinLayout l = make_layout(cfg, pl, 1, true);
  if ((s = check_ws(cfg, l.total)) != VDN_OK) return s;
  if (cfg->tokens > 0 && same_data({out}, {q, k, v})) return VDN_ERR_INVALID_ARG;
  if (cfg->tokens == 0)
    return cuda_status(copy_states(cfg, cfg->state_out, out_stride, cfg->state_in, in_stride, st));
  if (poison(cfg, l.total, st) != cudaSuccess) return VDN_ERR_CUDA;

  LinStateParams sp;
  std::memset(&sp, 0, sizeof(sp));
  sp.pl = pl;
  sp.B = cfg->batch, sp.N = cfg->tokens, sp.H = cfg->heads, sp.d = cfg->head_dim, sp.n_walks = 1;
  sp.log_decay = cfg->log_decay;
  sp.lengths = cfg->lengths;
  sp.status = cfg->status_word ? cfg->status_word : ws<int>(cfg, 0);
  sp.record = ws<int>(cfg, 64);
  sp.walk[0] = LinWalk{view(k), view(v), 1, 2, 0, ws(cfg, l.parts[0]), ws(cfg, l.s_in[0]),
                       cfg->state_in && cfg->state_out ? ws(cfg, l.s_head) : nullptr, cfg->state_in, in_stride, 1.f};
  LinOutParams op;
  std::memset(&op, 0, sizeof(op));
  op.pl = pl;
  op.B = sp.B, op.N = sp.N, op.H = sp.H, op.d = sp.d, op.n_jobs = 1;
  op.alpha = scale_of(cfg);
  op.log_decay = sp.log_decay;
  op.lengths = sp.lengths;
  op.status = sp.status;
  op.record = sp.record;
  op.inject_timeout = (cfg->debug_flags & VDN_INJECT_TIMEOUT) != 0;
  op.job[0] = LinJob{view(q), view(k), view(v), view(out), 0, 1, 2, 3, 0, 0, cfg->state_in, in_stride, 1.f,
                     sp.walk[0].s_in, sp.walk[0].s_head, cfg->state_out, out_stride, 1.f};
  return cuda_status(run(cfg, tc, {q, k, v}, {out}, sp, op, st));
}

vdn_status vdn_linear_attn_bwd(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* d_out,
                               const vdn_view* dq, const vdn_view* dk, const vdn_view* dv, const vdn_linear_cfg* cfg,
                               void* stream) {
  NvtxRange nvtx("vdn:linear_attn_bwd");
  vdn_status s = check_linear(cfg);
  if (s == VDN_OK) s = check_common(cfg);
  if (s == VDN_OK) s = check_state(cfg, cfg->state_in, cfg->state_in_stride);
  if (s == VDN_OK) s = check_state(cfg, cfg->d_state_out, cfg->d_state_out_stride);
  if (s == VDN_OK) s = check_state(cfg, cfg->d_state_in, cfg->d_state_in_stride);
  if (s != VDN_OK) return s;
  if (cfg->d_state_in && (cfg->d_state_in == cfg->d_state_out || cfg->d_state_in == cfg->state_in))
    return VDN_ERR_INVALID_ARG;
  const long long full = state_size(cfg);
  const long long in_stride = cfg->state_in_stride ? cfg->state_in_stride : full;
  const long long dout_stride = cfg->d_state_out_stride ? cfg->d_state_out_stride : full;
  const long long din_stride = cfg->d_state_in_stride ? cfg->d_state_in_stride : full;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cfg->tokens > 0) {
    for (const vdn_view* x : {q, k, v, d_out})
      if ((s = check_view(cfg, x, false)) != VDN_OK) return s;
    for (const vdn_view* x : {dq, dk, dv})
      if ((s = check_view(cfg, x, true)) != VDN_OK) return s;
  }
  const bool tc = cfg->tokens > 0 && on_tensor_cores(cfg, {q, k, v, d_out});
  const LinPlan pl = make_plan(cfg, 3, 2, tc, cfg->lengths);
  const LinLayout l = make_layout(cfg, pl, 2, false);
  if ((s = check_ws(cfg, l.total)) != VDN_OK) return s;
  if (cfg->tokens > 0 &&
      (same_data({dq, dk, dv}, {q, k, v, d_out}) || same_data({dq}, {dk, dv}) || same_data({dk}, {dv})))
    return VDN_ERR_INVALID_ARG;
  if (cfg->tokens == 0)
    return cuda_status(copy_states(cfg, cfg->d_state_in, din_stride, cfg->d_state_out, dout_stride, st));
  if (poison(cfg, l.total, st) != cudaSuccess) return VDN_ERR_CUDA;

  const float alpha = scale_of(cfg);
  LinStateParams sp;
  std::memset(&sp, 0, sizeof(sp));
  sp.pl = pl;
  sp.B = cfg->batch, sp.N = cfg->tokens, sp.H = cfg->heads, sp.d = cfg->head_dim, sp.n_walks = 2;
  sp.log_decay = cfg->log_decay;
  sp.lengths = cfg->lengths;
  sp.status = cfg->status_word ? cfg->status_word : ws<int>(cfg, 0);
  sp.record = ws<int>(cfg, 64);
  sp.walk[0] = LinWalk{view(k), view(v), 1, 2, 0, ws(cfg, l.parts[0]), ws(cfg, l.s_in[0]), nullptr,
                       cfg->state_in, in_stride, 1.f};
  sp.walk[1] = LinWalk{view(q), view(d_out), 0, 3, 1, ws(cfg, l.parts[1]), ws(cfg, l.s_in[1]), nullptr,
                       cfg->d_state_out, dout_stride, 1.f / alpha};
  LinOutParams op;
  std::memset(&op, 0, sizeof(op));
  op.pl = pl;
  op.B = sp.B, op.N = sp.N, op.H = sp.H, op.d = sp.d, op.n_jobs = 3;
  op.alpha = alpha;
  op.log_decay = sp.log_decay;
  op.lengths = sp.lengths;
  op.status = sp.status;
  op.record = sp.record;
  op.inject_timeout = (cfg->debug_flags & VDN_INJECT_TIMEOUT) != 0;
  op.job[0] = LinJob{view(d_out), view(v), view(k), view(dq), 3, 2, 1, 4, 0, 1, cfg->state_in, in_stride, 1.f,
                     sp.walk[0].s_in, nullptr, nullptr, 0, 0.f};
  op.job[1] = LinJob{view(v), view(d_out), view(q), view(dk), 2, 3, 0, 5, 1, 1, cfg->d_state_out, dout_stride, 1.f / alpha,
                     sp.walk[1].s_in, nullptr, nullptr, 0, 0.f};
  op.job[2] = LinJob{view(k), view(q), view(d_out), view(dv), 1, 0, 3, 6, 1, 0, cfg->d_state_out, dout_stride, 1.f / alpha,
                     sp.walk[1].s_in, nullptr, cfg->d_state_in, din_stride, alpha};
  return cuda_status(run(cfg, tc, {q, k, v, d_out}, {dq, dk, dv}, sp, op, st));
}

vdn_status vdn_linear_attn_step(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* out,
                                const vdn_linear_cfg* cfg, void* stream) {
  NvtxRange nvtx("vdn:linear_attn_step");
  vdn_status s = check_linear(cfg, true);
  if (s == VDN_OK) s = check_common(cfg);
  if (s != VDN_OK) return s;
  if (!cfg->state_out || cfg->n_slots < 1) return VDN_ERR_INVALID_ARG;
  if (!cfg->slots && cfg->n_slots < cfg->batch) return VDN_ERR_INVALID_ARG;
  if ((s = check_state(cfg, cfg->state_out, cfg->state_out_stride)) != VDN_OK) return s;
  for (const vdn_view* x : {q, k, v})
    if ((s = check_view(cfg, x, false, true)) != VDN_OK) return s;
  if ((s = check_view(cfg, out, true, true)) != VDN_OK) return s;
  if (same_data({out}, {q, k, v})) return VDN_ERR_INVALID_ARG;
  LinStepParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = view(q), p.k = view(k), p.v = view(v), p.o = view(out);
  p.B = cfg->batch, p.H = cfg->heads;
  p.scale = scale_of(cfg);
  p.log_decay = cfg->log_decay;
  p.pool = cfg->state_out;
  p.slot_stride = cfg->state_out_stride ? cfg->state_out_stride : state_size(cfg);
  p.slots = cfg->slots;
  p.n_slots = cfg->n_slots;
  p.status = cfg->status_word;
  return cuda_status(launch_lin_step(p, cfg->head_dim, cfg->dtype == VDN_FP32, static_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- RMSNorm

vdn_status vdn_norm_validate(const vdn_norm_cfg* c) {
  if (!c) return VDN_ERR_INVALID_ARG;
  if (c->rows < 0 || c->width < 1) return VDN_ERR_INVALID_ARG;
  if (c->output < VDN_NORM_TENSOR || c->output > VDN_NORM_E4M3_GROUP) return VDN_ERR_INVALID_ARG;
  for (int64_t x : {c->x_stride, c->residual_stride, c->residual_out_stride, c->out_stride, c->dy_stride, c->dh_stride,
                    c->dx_stride})
    if (x != 0 && x < c->width) return VDN_ERR_INVALID_ARG;
  if (c->dtype != VDN_BF16 && c->dtype != VDN_FP32) return VDN_ERR_UNSUPPORTED;
  if (c->rows >= (1ll << 31) - 1 || c->width > (1 << 20)) return VDN_ERR_UNSUPPORTED;  // one block a row at most
  return VDN_OK;
}

size_t vdn_norm_workspace_bytes(const vdn_norm_cfg* c) {
  if (vdn_norm_validate(c) != VDN_OK) return 0;
  return align_up(std::max<size_t>(1, norm_workspace(c->rows, c->width)), 256);
}

}  // extern "C"

namespace {

int64_t stride_or(int64_t s, int32_t width) { return s ? s : width; }

// An output at an input's address whose later rows lie elsewhere: a row would be overwritten before it is read.
struct Rows {
  const void* p;
  int64_t stride;
};
bool shifted(const Rows& out, const Rows& in, int64_t rows) {
  return out.p && out.p == in.p && out.stride != in.stride && rows > 1;
}

// 16-byte rows of a tensor of `e`-byte elements
bool vec_rows(const void* p, int64_t stride, int e) {
  return !p || (aligned(p, 16) && stride * e % 16 == 0);
}

}  // namespace

extern "C" {

vdn_status vdn_add_rmsnorm_fwd(const void* x, const void* residual, void* residual_out, void* out, float* scales,
                               const vdn_norm_cfg* cfg, void* stream) {
  NvtxRange nvtx("vdn:add_rmsnorm_fwd");
  vdn_status s = vdn_norm_validate(cfg);
  if (s != VDN_OK) return s;
  const bool quant = cfg->output != VDN_NORM_TENSOR;
  if (cfg->rows == 0) return VDN_OK;
  if (!x || !out || (quant && !scales)) return VDN_ERR_INVALID_ARG;
  const int e = cfg->dtype == VDN_FP32 ? 4 : 2;
  for (const void* p : {x, residual, (const void*)residual_out, quant ? nullptr : (const void*)out})
    if (!aligned(p, e)) return VDN_ERR_ALIGNMENT;
  if (!aligned(cfg->weight, 4) || !aligned(scales, 4)) return VDN_ERR_ALIGNMENT;
  // out may be x or residual where a thread reads what it overwrites; residual_out may be either in every mode
  if (out == residual_out || (quant && (out == x || out == residual))) return VDN_ERR_INVALID_ARG;
  const int32_t W = cfg->width;
  for (auto o : {Rows{out, stride_or(cfg->out_stride, W)}, Rows{residual_out, stride_or(cfg->residual_out_stride, W)}})
    if (shifted(o, Rows{x, stride_or(cfg->x_stride, W)}, cfg->rows) ||
        shifted(o, Rows{residual, stride_or(cfg->residual_stride, W)}, cfg->rows))
      return VDN_ERR_INVALID_ARG;
  NormParams p;
  p.x = x, p.res = residual, p.res_out = residual_out, p.out = out, p.scales = scales, p.weight = cfg->weight;
  p.rows = cfg->rows, p.W = cfg->width;
  p.eps = cfg->eps < 0.f ? 1e-6f : cfg->eps;
  p.sx = stride_or(cfg->x_stride, cfg->width);
  p.sres = stride_or(cfg->residual_stride, cfg->width);
  p.sres_out = stride_or(cfg->residual_out_stride, cfg->width);
  p.sout = stride_or(cfg->out_stride, cfg->width);
  const int vec = cfg->width % 8 == 0 && vec_rows(x, p.sx, e) && vec_rows(residual, p.sres, e) &&
                  vec_rows(residual_out, p.sres_out, e) && aligned(cfg->weight, 16) &&
                  (quant ? aligned(out, 8) && p.sout % 8 == 0 : vec_rows(out, p.sout, e));
  return cuda_status(launch_norm_fwd(p, cfg->dtype == VDN_FP32, cfg->output, vec, static_cast<cudaStream_t>(stream)));
}

vdn_status vdn_add_rmsnorm_bwd(const void* h, const void* dy, const void* dh, void* dx, float* dweight,
                               const vdn_norm_cfg* cfg, void* stream) {
  NvtxRange nvtx("vdn:add_rmsnorm_bwd");
  vdn_status s = vdn_norm_validate(cfg);
  if (s != VDN_OK) return s;
  if (cfg->output != VDN_NORM_TENSOR) return VDN_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int e = cfg->dtype == VDN_FP32 ? 4 : 2;
  if (cfg->rows > 0 && (!h || !dy || !dx)) return VDN_ERR_INVALID_ARG;
  for (const void* p : {h, dy, dh, (const void*)dx})
    if (!aligned(p, e)) return VDN_ERR_ALIGNMENT;
  if (!aligned(cfg->weight, 4) || !aligned(dweight, 4)) return VDN_ERR_ALIGNMENT;
  if (dweight) {
    if (!cfg->workspace || cfg->workspace_bytes < vdn_norm_workspace_bytes(cfg)) return VDN_ERR_WORKSPACE;
    if (!aligned(cfg->workspace, 256)) return VDN_ERR_ALIGNMENT;
  }
  if (cfg->rows > 0 && (dx == h || dx == dy)) return VDN_ERR_INVALID_ARG;
  if (shifted(Rows{dx, stride_or(cfg->dx_stride, cfg->width)}, Rows{dh, stride_or(cfg->dh_stride, cfg->width)}, cfg->rows))
    return VDN_ERR_INVALID_ARG;
  if (cfg->rows == 0) return dweight ? cuda_status(cudaMemsetAsync(dweight, 0, (size_t)cfg->width * 4, st)) : VDN_OK;
  NormBwdParams p;
  p.h = h, p.dy = dy, p.dh = dh, p.dx = dx, p.dweight = dweight, p.weight = cfg->weight;
  p.parts = dweight ? static_cast<float*>(cfg->workspace) : nullptr;
  p.rows = cfg->rows, p.W = cfg->width;
  p.eps = cfg->eps < 0.f ? 1e-6f : cfg->eps;
  p.sh = stride_or(cfg->x_stride, cfg->width);
  p.sdy = stride_or(cfg->dy_stride, cfg->width);
  p.sdh = stride_or(cfg->dh_stride, cfg->width);
  p.sdx = stride_or(cfg->dx_stride, cfg->width);
  p.n_parts = norm_parts(cfg->rows, cfg->width);
  const int vec = cfg->width % 8 == 0 && vec_rows(h, p.sh, e) && vec_rows(dy, p.sdy, e) && vec_rows(dh, p.sdh, e) &&
                  vec_rows(dx, p.sdx, e) && aligned(cfg->weight, 16);
  return cuda_status(launch_norm_bwd(p, cfg->dtype == VDN_FP32, vec, st));
}

}  // extern "C"
