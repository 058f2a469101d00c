/*
 * vdnattn.h - C ABI of libvdnattn, the sm_100a (B200) implementation of the
 * VDN-H3 dual-branch hybrid attention.
 *
 * Source of the operation: the VDN-H3 article (tahou.com, article
 * 216474224916730885), section "技术核心设计 / 双分支混合注意力机制" (the
 * softmax branch over a chunk window plus boundary anchors plus text; the
 * bidirectional frame-wise linear memory with half-weight text; the frame-7
 * example) and section "自适应门控融合双分支输出" (RMSNorm on the linear
 * branch, one sigmoid gate per branch, sum of the two).
 *
 * The call computes, for every video query token i (batch b, head h):
 *
 *   o_s[i] = softmax over keys J(i) of (scale * q_i . k_j), applied to v_j,
 *            J(i) = tokens of the frames in the window of i's chunk (the chunk
 *            and its two neighbours, clipped at the ends) and of the first and
 *            last frame, each frame once, plus all text tokens;
 *   o_l[i] = phi(q_i)^T (S_F + S_B) / (phi(q_i) . (z_F + z_B)), phi = elu + 1,
 *            S_F/z_F summing phi(k) v^T / phi(k) over the chunks before the
 *            window, S_B/z_B over the chunks after it, both without the two
 *            anchor frames, each holding half of the text state; o_l = 0 when
 *            the states hold no token;
 *   r[i]   = o_l[i] / sqrt(mean_d(o_l[i]^2) + eps) * gamma[h];
 *   out[i] = sigmoid(gate_s[i]) * o_s[i] + sigmoid(gate_l[i]) * r[i].
 *
 * Two readings the article leaves open are selectable (vdn_cfg):
 *   anchor_query_mode = VDN_ANCHOR_LOCAL (default): the rule above for every
 *     query frame, the anchors included (the frame-7 example's rule);
 *     VDN_ANCHOR_GLOBAL: a query in frame 0 or F-1 attends by softmax to
 *     every video frame (plus text) and reads nothing through the states
 *     (o_l = 0 there, so out = sigmoid(gate_s) * o_s); other rows unchanged.
 *   output_mode = VDN_OUTPUT_MERGED (default): out as above;
 *     VDN_OUTPUT_SPLIT: out = sigmoid(gate_s) * o_s and
 *     cfg->out_linear = sigmoid(gate_l) * r, the two gated branch terms
 *     (section 自适应门控融合双分支输出: one output per branch), for callers
 *     that project each branch before summing.
 *
 * Where the linear read and the merge run is selectable too (same result up
 * to rounding):
 *   readout_mode = VDN_READOUT_SEPARATE (default): the softmax kernel stores
 *     sigmoid(gate_s) * o_s (bf16) and a readout kernel of its own reads it
 *     back with q, M_c and gate_l and writes out;
 *     VDN_READOUT_FUSED: the readout, the RMSNorm and the merge run in the
 *     softmax kernel's epilogue (the frame-7 paragraph combines the linear read
 *     with the local branch at the query's position): o_s stays in TMEM in
 *     fp32 and q is read once.  Needs bf16 tensors, head_dim 128,
 *     the BF16 softmax precision and VDN_OUTPUT_MERGED without the VDN_OUT_*
 *     debug outputs (VDN_ERR_UNSUPPORTED otherwise).
 *
 * Layouts (row-major, no padding between rows):
 *   q, k, v, gate_s, gate_l, out : [batch, frames*tokens_per_frame, heads, head_dim]
 *   text_k, text_v               : [batch, text_tokens, heads, head_dim]
 *   token n of a video tensor lies in latent frame n / tokens_per_frame.
 * All of these are DEVICE pointers in the dtype given by vdn_cfg.dtype, each
 * 16-byte aligned; the caller owns them.  Accumulation is always fp32; tensor
 * core operands are bf16 (fp32 inputs are rounded to bf16 before the
 * contractions, and the intermediate softmax output o_s is kept in bf16).
 *
 * Ownership and threading: the library allocates no device memory.  Scratch
 * space is the caller-owned workspace (vdn_workspace_bytes).  Every device
 * function enqueues its work on the given stream and returns without host
 * synchronisation; the caller keeps inputs, outputs and the workspace alive
 * until that work completes.  Two calls that share a workspace must be
 * ordered on the GPU.  Functions are thread-safe.
 *
 * Errors: every argument check happens before anything is enqueued; on an
 * error return nothing was launched.  VDN_ERR_CUDA reports a launch error
 * (cudaGetLastError).  A kernel whose bounded wait runs out (1 s of global
 * time) writes VDN_ERR_TIMEOUT into *status_word (when given) and returns
 * early; that is read by the caller after synchronising.  The first such wait
 * also describes itself in a timeout record, 16 int32 words at byte 64 of the
 * workspace (count of waits that ran out, kernel id, block, warp, barrier as
 * its byte distance to the CTA's abort flag, phase parity, nanoseconds waited
 * as two words, SM); the library never clears it, the caller may.
 */
#ifndef VDNATTN_H
#define VDNATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define VDN_API __attribute__((visibility("default")))
#else
#define VDN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  VDN_OK = 0,
  VDN_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, frames % chunk != 0 */
  VDN_ERR_UNSUPPORTED = 2, /* head_dim not 32/64/128, unknown dtype, too many chunks */
  VDN_ERR_ALIGNMENT = 3,   /* a pointer is not 16-byte aligned */
  VDN_ERR_WORKSPACE = 4,   /* workspace NULL or smaller than vdn_workspace_bytes */
  VDN_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed */
  VDN_ERR_TIMEOUT = 6      /* written to status_word by a kernel whose wait ran out */
} vdn_status;

typedef enum { VDN_BF16 = 0, VDN_FP32 = 1 } vdn_dtype;

typedef enum { VDN_ANCHOR_LOCAL = 0, VDN_ANCHOR_GLOBAL = 1 } vdn_anchor_query_mode;
typedef enum { VDN_OUTPUT_MERGED = 0, VDN_OUTPUT_SPLIT = 1 } vdn_output_mode;
typedef enum { VDN_READOUT_SEPARATE = 0, VDN_READOUT_FUSED = 1 } vdn_readout_mode;

/* Operand precision of the softmax branch's two contractions.  BF16 (default):
 * bf16 operands, fp32 accumulation.  FP8: q, k, v, text_k, text_v quantised
 * to e4m3 with one scale per (batch, head) for q, one for k and text_k, one for
 * v and text_v (scale = max |x| / 448); P in e4m3; fp32 accumulation; o_s and
 * everything after it as in BF16.  FP8 needs head_dim 128, bf16 tensors and
 * tokens_per_frame % 16 == 0 (VDN_ERR_UNSUPPORTED otherwise), and a larger
 * workspace (vdn_workspace_bytes accounts for it). */
typedef enum { VDN_PREC_BF16 = 0, VDN_PREC_FP8 = 1 } vdn_softmax_precision;

/* debug_flags: what vdn_readout_merge writes into out instead of the merge. */
enum {
  VDN_OUT_SOFTMAX_ONLY = 1, /* out = o_s (no gate) */
  VDN_OUT_LINEAR_ONLY = 2,  /* out = r, the RMS-normalised linear read (no gate) */
  VDN_OUT_LINEAR_RAW = 4,   /* out = o_l, the linear read before RMSNorm */
  VDN_EXPORT_STATES = 8,    /* the scan (vdn_state_scan, or the one inside vdn_softmax_and_scan and
                               the whole calls) also writes S_F/z_F and S_B/z_B (fp32) */
  VDN_INJECT_TIMEOUT = 16,  /* test of the failure path only: in the state build, the MMA thread of
                               CTA 0 first waits, with a 10-ms limit, for a barrier phase
                               that nothing completes; it gives up, the CTA's other warps follow, the
                               kernel writes VDN_ERR_TIMEOUT to status_word and returns.  The call's
                               outputs are then undefined; the context stays usable. */
  VDN_STALL_READOUT_MMA = 32, /* test of the readout's barrier protocol only: the readout's MMA thread
                               sleeps 50 microseconds whenever it moves to another readout operand
                               (batch, chunk, head), letting the other warps run as far ahead as the
                               protocol allows.  Outputs are unchanged. */
  VDN_POISON_WS = 64,         /* vdn_hybrid_attn_fwd, _host and _static first fill the workspace past its
                               256-byte status slot with 0xFF bytes (NaN in bf16 and fp32), so that a
                               read of scratch the call has not written would show in the output.
                               Outputs are unchanged. */
  VDN_INJECT_TIMEOUT_SCAN = 128 /* test of the failure path only: under VDN_READOUT_FUSED, the producer of
                               CTA 0 of the softmax kernel waits, with a 10-ms limit, for one scan unit
                               more than its (batch, head) has; it gives up, the CTA's other warps
                               follow, the kernel writes VDN_ERR_TIMEOUT to status_word and returns.
                               The call's outputs are then undefined; the context stays usable. */
};

typedef struct {
  int32_t batch;            /* B  >= 1 */
  int32_t frames;           /* F  >= 1, latent frames; anchors are frames 0 and F-1 */
  int32_t tokens_per_frame; /* P  >= 1 */
  int32_t heads;            /* H  >= 1 */
  int32_t head_dim;         /* d in {32, 64, 128} */
  int32_t text_tokens;      /* T  >= 0 */
  int32_t chunk_frames;     /* C  >= 1, F % C == 0 (5 in the article's chunking, 1 in its frame-7 example) */
  int32_t dtype;            /* vdn_dtype of q, k, v, text, gates and out */
  float softmax_scale;      /* <= 0 selects 1/sqrt(head_dim) */
  float rms_eps;            /* < 0 selects 1e-6 */
  const float* rms_weight;  /* device [heads, head_dim] fp32 gamma (16-byte aligned), or NULL for ones */
  int32_t debug_flags;      /* VDN_OUT_* / VDN_EXPORT_STATES, 0 in production */
  int32_t anchor_query_mode; /* vdn_anchor_query_mode; 0 = LOCAL */
  void* workspace;          /* device, 256-byte aligned, >= vdn_workspace_bytes(cfg) bytes */
  size_t workspace_bytes;
  int32_t* status_word;     /* optional device int32; set to VDN_ERR_TIMEOUT by a kernel that gave up */
  float* export_fwd;        /* VDN_EXPORT_STATES: device [B, F/C, H, d+1, d] fp32; row d holds z */
  float* export_bwd;        /* same layout, backward states */
  int32_t output_mode;      /* vdn_output_mode; 0 = MERGED.  SPLIT excludes the VDN_OUT_* debug flags */
  int32_t softmax_precision; /* vdn_softmax_precision; 0 = BF16 */
  void* out_linear;         /* SPLIT only: device [B, N, H, d] in dtype, 16-byte aligned; else ignored */
  int32_t readout_mode;     /* vdn_readout_mode; 0 = SEPARATE */
} vdn_cfg;

/* Library version, (major << 16) | minor. */
VDN_API int32_t vdn_version(void);

/* Human-readable name of a status code (static string). */
VDN_API const char* vdn_status_string(vdn_status s);

/* Host-only argument check of cfg (sizes, dtype, head_dim, chunking).  No CUDA call. */
VDN_API vdn_status vdn_validate(const vdn_cfg* cfg);

/* Bytes of workspace a call with this cfg needs; 0 if cfg is invalid.  No CUDA call. */
VDN_API size_t vdn_workspace_bytes(const vdn_cfg* cfg);

/* Host-only membership table of the frame-7 rule: table[f*F + g] = 1 when query
 * frame f reads key frame g through the softmax branch, 2 through the forward
 * state, 3 through the backward state (under VDN_ANCHOR_GLOBAL the rows of
 * frames 0 and F-1 are all 1).  table is HOST memory of F*F bytes. */
VDN_API vdn_status vdn_plan_membership(const vdn_cfg* cfg, uint8_t* table);

/* The same table produced on the GPU by the index logic the kernels use
 * (KV ranges of the softmax kernel, chunk membership of the scan).
 * table_dev is DEVICE memory of F*F bytes.  stream is a cudaStream_t. */
VDN_API vdn_status vdn_membership_device(const vdn_cfg* cfg, uint8_t* table_dev, void* stream);

/* Whole call: staging (fp32 or head_dim 32 only), state build, sparse
 * softmax with the forward/backward scan (and, for bf16 with head_dim 64 or
 * 128, the softmax branch's gate) in the same kernel, readout + merge, all on
 * stream; under VDN_READOUT_FUSED: state build, then the softmax kernel with
 * the scan inside and the readout and merge in its epilogue.  out: [B, N, H, d] in dtype (and cfg->out_linear under
 * VDN_OUTPUT_SPLIT). */
VDN_API vdn_status vdn_hybrid_attn_fwd(const void* q, const void* k, const void* v,
                               const void* text_k, const void* text_v,
                               const void* gate_s, const void* gate_l, void* out,
                               const vdn_cfg* cfg, void* stream);

/* The steps of vdn_hybrid_attn_fwd, for callers that schedule them
 * separately.  vdn_stage_inputs (required first when dtype is fp32 or
 * head_dim is 32; otherwise a no-op), then either
 *   vdn_state_build -> vdn_softmax_and_scan -> vdn_readout_merge
 * (the sequence of the whole call: the scan runs in otherwise idle warps of
 * the softmax kernel), or, with the linear steps independent of the softmax
 * branch (e.g. on a second stream),
 *   vdn_state_build -> vdn_state_scan, and vdn_sparse_softmax, in either
 *   order, then vdn_readout_merge.
 * Each reads what the earlier steps left in the workspace. */
VDN_API vdn_status vdn_stage_inputs(const void* q, const void* k, const void* v,
                            const void* text_k, const void* text_v,
                            const vdn_cfg* cfg, void* stream);
/* Partial states [S | z] = phi(K)^T [V | 1] (tensor cores): for every state
 * segment (the non-anchor frames of one chunk, or the text) of every (batch,
 * head), one partial per state-build CTA whose equal share of the tiles meets
 * the segment. */
VDN_API vdn_status vdn_state_build(const void* k, const void* v, const void* text_k,
                           const void* text_v, const vdn_cfg* cfg, void* stream);
/* Forward/backward chunk states and their sum M_c, fp32 scan. */
VDN_API vdn_status vdn_state_scan(const vdn_cfg* cfg, void* stream);
/* The forward and backward states S_F / z_F and S_B / z_B of every (batch,
 * chunk, head), as fp32 [B, F/C, H, d+1, d] (row n < d: value column n of S;
 * row d: z; column a: key feature a), recomputed by the scan on `stream`
 * from the state partials that the last vdn_hybrid_attn_fwd or
 * vdn_state_build on cfg->workspace left there; the readout operands are
 * rewritten with the values they had.  fwd, bwd: device, 16-byte aligned,
 * B*(F/C)*H*(d+1)*d floats each, caller-owned.  Same as calling
 * vdn_state_scan with VDN_EXPORT_STATES and cfg->export_fwd/export_bwd set. */
VDN_API vdn_status vdn_export_states(const vdn_cfg* cfg, float* fwd, float* bwd, void* stream);
/* Block-sparse softmax branch o_s (window + anchors + text) into the workspace. */
VDN_API vdn_status vdn_sparse_softmax(const void* q, const void* k, const void* v,
                              const void* text_k, const void* text_v,
                              const vdn_cfg* cfg, void* stream);
/* vdn_sparse_softmax and, in the same kernel, vdn_state_scan: must follow
 * vdn_state_build on the same workspace (stream order).  gate_s (the
 * softmax branch's gate logits, [B, N, H, d], or NULL): for bf16 tensors whose
 * head_dim is 64 or 128, and without VDN_OUT_SOFTMAX_ONLY, the kernel stores
 * sigmoid(gate_s) * o_s in place of o_s (the softmax branch's term of the
 * gated merge; one rounding to bf16 either way) and notes so in the
 * workspace, and vdn_readout_merge then takes that term as it is; otherwise
 * o_s is stored and the readout applies the gate.  Errors as
 * vdn_sparse_softmax, plus VDN_ERR_INVALID_ARG for VDN_EXPORT_STATES without
 * export buffers and VDN_ERR_ALIGNMENT for a misaligned gate_s. */
VDN_API vdn_status vdn_softmax_and_scan(const void* q, const void* k, const void* v,
                                        const void* text_k, const void* text_v, const void* gate_s,
                                        const vdn_cfg* cfg, void* stream);
/* phi(Q) M_c readout, RMSNorm, gates and merge into out. */
VDN_API vdn_status vdn_readout_merge(const void* q, const void* gate_s, const void* gate_l,
                             void* out, const vdn_cfg* cfg, void* stream);
/* The steps of a VDN_READOUT_FUSED call: vdn_state_build ->
 * vdn_sparse_softmax_merge, which runs the softmax branch, the
 * forward/backward scan (in otherwise idle warps, as vdn_softmax_and_scan) and,
 * in the kernel's item epilogue, the readout, RMSNorm, gates and merge into
 * out; it must follow vdn_state_build on the same workspace (stream order).
 * Requirements of VDN_READOUT_FUSED apply whatever cfg->readout_mode says
 * (VDN_ERR_UNSUPPORTED otherwise); VDN_ERR_ALIGNMENT for a misaligned
 * pointer; VDN_ERR_INVALID_ARG for VDN_EXPORT_STATES without export buffers. */
VDN_API vdn_status vdn_sparse_softmax_merge(const void* q, const void* k, const void* v,
                                            const void* text_k, const void* text_v,
                                            const void* gate_s, const void* gate_l, void* out,
                                            const vdn_cfg* cfg, void* stream);

/* For callers that cannot allocate device memory (code running inside another
 * runtime's plugin/operator interface that hands over tensors but no
 * allocator, or latency-critical loops where cudaMalloc is not acceptable).
 * There is no counterpart on the article's pages: this is an interface
 * addition, not part of the method.
 *
 * Same operation, arguments and layouts as vdn_hybrid_attn_fwd, but
 * cfg->workspace / workspace_bytes are ignored: the scratch is a static device
 * array of vdn_static_scratch_bytes() (32 MiB) inside the library, which every
 * GPU that loads the library holds until the process exits.  The first call on
 * a device (with that device current) looks up the array's device address
 * with cudaGetSymbolAddress; make that first call before any stream capture.
 * The address is cached with the id of the CUDA context it was looked up in
 * and is valid only there: after cudaDeviceReset (or any replacement of the
 * context) the next call looks it up again, and that call too should precede
 * any capture.  Nothing is allocated.  Returns VDN_ERR_WORKSPACE when
 * vdn_workspace_bytes(cfg) exceeds the static size (it fits, e.g., 15 frames
 * x 256 tokens x 8 heads x head_dim 64); every argument error (sizes,
 * missing or misaligned pointers, including cfg->status_word and
 * cfg->rms_weight) is returned before any CUDA call, with nothing queued.
 * All calls on a device share the one array: calls whose GPU work overlaps
 * race and must be ordered by the caller.  The status slot of the array is
 * cleared on every call. */
VDN_API vdn_status vdn_hybrid_attn_fwd_static(const void* q, const void* k, const void* v,
                                              const void* text_k, const void* text_v,
                                              const void* gate_s, const void* gate_l, void* out,
                                              const vdn_cfg* cfg, void* stream);
/* Size in bytes of the static scratch used by vdn_hybrid_attn_fwd_static. */
VDN_API size_t vdn_static_scratch_bytes(void);

/* The whole call on HOST tensors (same layouts and dtype as vdn_hybrid_attn_fwd;
 * out, and cfg->out_linear under VDN_OUTPUT_SPLIT, are HOST pointers too).
 * Not part of the method: an interface for callers whose tensors live in host
 * memory.  The inputs are copied into `staging`, a caller-owned DEVICE buffer
 * of at least vdn_host_staging_bytes(cfg) bytes (256-byte aligned), on a
 * library-owned copy stream in the order the kernels need them (text, k, v,
 * then q, then the gates), so the state build runs while q is in flight and
 * the softmax branch while the gates are; the output is copied back on
 * `stream`.  cfg->workspace is used as in vdn_hybrid_attn_fwd; the export
 * buffers, if any, are device memory.  Host buffers should be page-locked
 * (cudaHostAlloc / cudaHostRegister): from pageable memory the copies do
 * not overlap.  The call returns once everything is enqueued; the caller
 * synchronises `stream` before reading out and must keep the host and device
 * buffers alive until then.  Errors: as vdn_hybrid_attn_fwd, plus
 * VDN_ERR_WORKSPACE for a missing or small staging buffer and
 * VDN_ERR_ALIGNMENT for a misaligned one. */
VDN_API size_t vdn_host_staging_bytes(const vdn_cfg* cfg);
VDN_API vdn_status vdn_hybrid_attn_fwd_host(const void* q, const void* k, const void* v,
                                            const void* text_k, const void* text_v,
                                            const void* gate_s, const void* gate_l, void* out,
                                            void* staging, size_t staging_bytes,
                                            const vdn_cfg* cfg, void* stream);

/* ------------------------------------------------------------------------
 * Causal linear memory with a decay for each head.
 *
 * The hybrid call's linear branch sums phi(k) v^T over whole frame-chunks, in
 * both directions, and needs the whole clip.  A model that produces frame after
 * frame, or text token after token, reads the causal form of the same memory:
 *
 *   S_t = lambda_h S_{t-1} + k_t^T v_t     (d x d, fp32),   lambda_h = exp(log_decay[h])
 *   out_t = scale * q_t S_t                (token t itself included)
 *
 * per batch entry and head, S before the first token = state_in (or 0).  Any
 * feature map is the caller's, applied to q and k beforehand; the RMSNorm that
 * follows is vdn_add_rmsnorm_fwd.  There is no counterpart on the article's
 * pages: an interface addition, not part of the method.
 *
 *   vdn_linear_attn_fwd   whole sequences, state in and out;
 *   vdn_linear_attn_bwd   the gradients by q, k, v and state_in;
 *   vdn_linear_attn_step  one token of each of `batch` sequences, on a pool of
 *                         states that is updated in place.
 *
 * log_decay is finite or -infinity (lambda = 0, a token sees itself only), and
 * expected to be <= 0; larger values follow the formula.  It is a constant of
 * the model: no gradient by it is formed.
 *
 * Accumulation, states and decay factors are fp32.  fp32 tensors are computed
 * in fp32 throughout.  The contractions of bf16 tensors run on the tensor
 * cores: decayed scores and the state are rounded to bf16 as operands of the
 * read (not in the carried state), and decayed keys enter the state in two or
 * three bf16 parts (2^-16 of a term, 2^-24 of one whose decay to the end is
 * above 2^-4 where the last state is asked for: out and dv may differ in their
 * rounding with it).  A token's contribution may end where its decay has fallen below
 * 2^-150.  A NaN or an infinity in a real token's row may reach earlier rows of
 * its 128-row chunk too.
 *
 * Tensors are views: element (b, n, h, i) of a tensor lies at data + b *
 * batch_stride + n * token_stride + h * head_stride + i, strides in elements
 * (the head_dim elements of a row are contiguous), so that q, k and v may be
 * slices of one projection.  data is 16-byte aligned and every stride a
 * multiple of 16 bytes; an input's stride may be 0 (a broadcast), an output's
 * only where that dimension has one entry.  Outputs must not overlap each other
 * or an input (the same address is refused, other overlaps are not seen).
 *
 * lengths (optional, device, one int32 per batch entry, clamped to [0, tokens]):
 * batch entry b has lengths[b] tokens, and its later rows are padding.  Padding
 * rows are not used whatever they hold, and the rows of out, dq, dk and dv
 * there are written as zeros.  state_out is the state after the last real
 * token: state_in (or 0) for a sequence without one.
 *
 * States are [batch][heads][head_dim (of k)][head_dim (of v)] fp32, 16-byte
 * aligned, with the given distance between batch entries.  state_out may be
 * state_in itself (same pointer and stride); any other overlap is not allowed.
 * ---------------------------------------------------------------------- */

typedef struct {
  void* data;
  int64_t batch_stride, token_stride, head_stride; /* elements */
} vdn_view;

typedef struct {
  int32_t batch;          /* B >= 1 */
  int32_t tokens;         /* N >= 0 (vdn_linear_attn_step: not read) */
  int32_t heads;          /* 1 <= H <= 4096 */
  int32_t head_dim;       /* d in {32, 64, 128} */
  int32_t dtype;          /* vdn_dtype of q, k, v, out and their gradients */
  float scale;            /* <= 0 selects 1/sqrt(head_dim); else a normal number */
  const float* log_decay; /* device [heads] fp32, 4-byte aligned */
  const int32_t* lengths; /* device [batch] or NULL (all tokens); not read by the step */
  const float* state_in;  /* fwd, bwd: S before the first token, or NULL (0) */
  float* state_out;       /* fwd: S after the last token, or NULL; step: the pool of states */
  const float* d_state_out; /* bwd: gradient by state_out, or NULL (0) */
  float* d_state_in;      /* bwd: gradient by state_in, or NULL */
  int64_t state_in_stride, state_out_stride;     /* elements between batch entries (step: between */
  int64_t d_state_out_stride, d_state_in_stride; /* slots); 0 selects heads * head_dim^2 */
  const int32_t* slots;   /* step: device [batch], the pool entry of each row, or NULL (row b: entry b) */
  int32_t n_slots;        /* step: entries of the pool */
  int32_t debug_flags;    /* VDN_POISON_WS, VDN_INJECT_TIMEOUT (tests); 0 in production */
  void* workspace;        /* device, 256-byte aligned, >= vdn_linear_workspace_bytes; not used by the step */
  size_t workspace_bytes;
  int32_t* status_word;   /* optional device int32: VDN_ERR_TIMEOUT by a kernel that gave up,
                             VDN_ERR_INVALID_ARG by the step for a slot >= n_slots */
} vdn_linear_cfg;

/* Host-only check of cfg's sizes, types and flags.  No CUDA call. */
VDN_API vdn_status vdn_linear_validate(const vdn_linear_cfg* cfg);
/* Bytes of workspace of the forward (backward = 0) or backward (1) call; 0 if
 * cfg is invalid.  No CUDA call: the size holds for every device. */
VDN_API size_t vdn_linear_workspace_bytes(const vdn_linear_cfg* cfg, int32_t backward);
/* out and, where given, state_out, from q, k, v and state_in. */
VDN_API vdn_status vdn_linear_attn_fwd(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* out,
                                       const vdn_linear_cfg* cfg, void* stream);
/* dq, dk, dv and, where given, d_state_in, from q, k, v, state_in, the
 * gradient d_out by out and, where given, d_state_out. */
VDN_API vdn_status vdn_linear_attn_bwd(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* d_out,
                                       const vdn_view* dq, const vdn_view* dk, const vdn_view* dv,
                                       const vdn_linear_cfg* cfg, void* stream);
/* One token for each of cfg->batch rows (token_stride is not read): entry
 * slots[b] of the pool cfg->state_out becomes lambda S + k_b^T v_b, and out_b =
 * scale * q_b S of the new state.  A negative slot marks a padding row: no state
 * is touched and its out row is written as zeros; so does a slot >= n_slots,
 * which also writes VDN_ERR_INVALID_ARG to status_word.  Rows with the same slot
 * are successive tokens of one sequence, taken in the order of the rows.  To find
 * them the slots are read batch times: for batches of thousands of rows that costs
 * more than the states (NULL, for rows in the pool's order, does not). */
VDN_API vdn_status vdn_linear_attn_step(const vdn_view* q, const vdn_view* k, const vdn_view* v, const vdn_view* out,
                                        const vdn_linear_cfg* cfg, void* stream);

/* ------------------------------------------------------------------------
 * RMSNorm with the residual's addition, and an output in 8 bits with scales.
 *
 *   h = x + residual,   y = h / sqrt(mean_i(h_i^2) + eps) * weight        (rows of `width` elements)
 *
 * in fp32; residual_out receives h rounded once to the tensors' type (the norm
 * is taken of the unrounded sum).  The result is y in the tensors' type, or e4m3
 * values with fp32 scales, y ~ value * scale, scale = max|y| / 448 over the row
 * or over each 128 columns (the last group may be shorter), 1 where all are zero;
 * values are rounded to nearest even.  A row that holds a NaN or an infinity
 * gives what the formula gives: NaN values and, under a scale, a NaN scale
 * where a NaN is in its reach.  Squares beyond fp32's range (elements above
 * 1e16, or, with eps below 2^-80, below 1e-12) are summed of the row multiplied
 * by a power of two, so that every finite row is normed.  The gradients' 1 / rms
 * itself is fp32: it overflows for rows of denormal numbers.
 *
 * Backward (of the tensor output; h is the stored residual_out, or x): with
 * g = dy * weight, r = 1 / sqrt(mean(h^2) + eps):
 *   dx = dh + r g - h r^3 mean(g h)    (the gradient by x and by residual; dh, the
 *        gradient that reaches h from elsewhere, may be NULL)
 *   dweight = sum over rows of dy h r   (fp32, summed in a fixed order)
 *
 * Row strides in elements, any value >= width; pointers aligned to their
 * element.  Rows that are 16-byte aligned with a width divisible by 8 take
 * vector loads.  x or residual may be residual_out or, with VDN_NORM_TENSOR, out,
 * and dh may be dx, with the same strides; outputs must not overlap otherwise
 * (the same address with another stride, or where it is not allowed, is refused;
 * other overlaps are not seen).  There is no counterpart on the article's pages
 * (its RMSNorm of the linear read is part of vdn_hybrid_attn_fwd).
 * ---------------------------------------------------------------------- */

/* Form of the norm's result. */
typedef enum { VDN_NORM_TENSOR = 0, VDN_NORM_E4M3_ROW = 1, VDN_NORM_E4M3_GROUP = 2 } vdn_norm_output;

typedef struct {
  int64_t rows;        /* >= 0 */
  int32_t width;       /* 1 <= width <= 2^20 */
  int32_t dtype;       /* vdn_dtype of x, residual, residual_out, the tensor output, dy, dh, dx */
  int32_t output;      /* vdn_norm_output; the backward takes VDN_NORM_TENSOR only */
  float eps;           /* < 0 selects 1e-6 */
  const float* weight; /* device [width] fp32, 4-byte aligned, or NULL (ones) */
  int64_t x_stride, residual_stride, residual_out_stride, out_stride; /* elements; 0 selects width */
  int64_t dy_stride, dh_stride, dx_stride; /* backward (h: x_stride) */
  void* workspace;     /* backward with dweight: device, 256-byte aligned, >= vdn_norm_workspace_bytes */
  size_t workspace_bytes;
} vdn_norm_cfg;

VDN_API vdn_status vdn_norm_validate(const vdn_norm_cfg* cfg);
/* Bytes of workspace of vdn_add_rmsnorm_bwd with dweight; 0 if cfg is invalid. */
VDN_API size_t vdn_norm_workspace_bytes(const vdn_norm_cfg* cfg);
/* residual and residual_out may be NULL (h = x; h not stored).  scales: fp32
 * [rows] (E4M3_ROW) or [rows, ceil(width / 128)] (E4M3_GROUP); not used by
 * VDN_NORM_TENSOR. */
VDN_API vdn_status vdn_add_rmsnorm_fwd(const void* x, const void* residual, void* residual_out, void* out,
                                       float* scales, const vdn_norm_cfg* cfg, void* stream);
/* dx and, where given, dweight [width] fp32. */
VDN_API vdn_status vdn_add_rmsnorm_bwd(const void* h, const void* dy, const void* dh, void* dx, float* dweight,
                                       const vdn_norm_cfg* cfg, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VDNATTN_H */
