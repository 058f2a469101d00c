"""ctypes binding of libvdnattn (argument marshalling only).

Every step of the hybrid attention runs in the library's CUDA kernels; this
module only turns torch tensors into pointers, fills the ``vdn_cfg`` struct,
passes the current CUDA stream and maps status codes to exceptions.  It
raises if the library has not been built: there is no other path.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import warnings
from dataclasses import dataclass

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvdnattn.so")
_lib = None

VDN_BF16, VDN_FP32 = 0, 1
OUT_SOFTMAX_ONLY, OUT_LINEAR_ONLY, OUT_LINEAR_RAW, EXPORT_STATES, INJECT_TIMEOUT = 1, 2, 4, 8, 16
STALL_READOUT_MMA, POISON_WS, INJECT_TIMEOUT_SCAN = 32, 64, 128
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "pointer not aligned",
          4: "workspace missing or too small", 5: "CUDA error", 6: "device wait timed out"}

EXPORTED = ["vdn_version", "vdn_status_string", "vdn_validate", "vdn_workspace_bytes", "vdn_plan_membership",
            "vdn_membership_device", "vdn_hybrid_attn_fwd", "vdn_stage_inputs", "vdn_state_build",
            "vdn_state_scan", "vdn_sparse_softmax", "vdn_softmax_and_scan", "vdn_readout_merge",
            "vdn_sparse_softmax_merge",
            "vdn_hybrid_attn_fwd_static",
            "vdn_static_scratch_bytes", "vdn_host_staging_bytes", "vdn_hybrid_attn_fwd_host", "vdn_export_states",
            "vdn_linear_validate", "vdn_linear_workspace_bytes", "vdn_linear_attn_fwd", "vdn_linear_attn_bwd",
            "vdn_linear_attn_step", "vdn_norm_validate", "vdn_norm_workspace_bytes", "vdn_add_rmsnorm_fwd",
            "vdn_add_rmsnorm_bwd"]


class VdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, 'unknown')} (status {code})")
        self.code = code


class VdnCfg(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("frames", ctypes.c_int32), ("tokens_per_frame", ctypes.c_int32),
        ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("text_tokens", ctypes.c_int32),
        ("chunk_frames", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("rms_eps", ctypes.c_float),
        ("rms_weight", ctypes.c_void_p),
        ("debug_flags", ctypes.c_int32), ("anchor_query_mode", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("status_word", ctypes.c_void_p),
        ("export_fwd", ctypes.c_void_p), ("export_bwd", ctypes.c_void_p),
        ("output_mode", ctypes.c_int32), ("softmax_precision", ctypes.c_int32),
        ("out_linear", ctypes.c_void_p), ("readout_mode", ctypes.c_int32),
    ]


class VdnView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class VdnLinearCfg(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
        ("log_decay", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
        ("state_in", ctypes.c_void_p), ("state_out", ctypes.c_void_p),
        ("d_state_out", ctypes.c_void_p), ("d_state_in", ctypes.c_void_p),
        ("state_in_stride", ctypes.c_int64), ("state_out_stride", ctypes.c_int64),
        ("d_state_out_stride", ctypes.c_int64), ("d_state_in_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p), ("n_slots", ctypes.c_int32), ("debug_flags", ctypes.c_int32),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("status_word", ctypes.c_void_p),
    ]


class VdnNormCfg(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32), ("output", ctypes.c_int32),
        ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64), ("residual_out_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64), ("dh_stride", ctypes.c_int64),
        ("dx_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


def library() -> ctypes.CDLL:
    """Load libvdnattn.so from the package directory (raises if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m video_diffusion_hybrid_sparse_b200.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P = ctypes.c_void_p
        C = ctypes.POINTER(VdnCfg)
        lib.vdn_version.restype = ctypes.c_int32
        lib.vdn_status_string.restype = ctypes.c_char_p
        lib.vdn_status_string.argtypes = [ctypes.c_int]
        lib.vdn_validate.argtypes = [C]
        lib.vdn_workspace_bytes.restype = ctypes.c_size_t
        lib.vdn_workspace_bytes.argtypes = [C]
        lib.vdn_plan_membership.argtypes = [C, P]
        lib.vdn_membership_device.argtypes = [C, P, P]
        lib.vdn_hybrid_attn_fwd.argtypes = [P, P, P, P, P, P, P, P, C, P]
        lib.vdn_stage_inputs.argtypes = [P, P, P, P, P, C, P]
        lib.vdn_state_build.argtypes = [P, P, P, P, C, P]
        lib.vdn_state_scan.argtypes = [C, P]
        lib.vdn_export_states.argtypes = [C, P, P, P]
        lib.vdn_sparse_softmax.argtypes = [P, P, P, P, P, C, P]
        lib.vdn_softmax_and_scan.argtypes = [P, P, P, P, P, P, C, P]
        lib.vdn_readout_merge.argtypes = [P, P, P, P, C, P]
        lib.vdn_sparse_softmax_merge.argtypes = [P, P, P, P, P, P, P, P, C, P]
        lib.vdn_hybrid_attn_fwd_static.argtypes = [P, P, P, P, P, P, P, P, C, P]
        lib.vdn_static_scratch_bytes.restype = ctypes.c_size_t
        lib.vdn_host_staging_bytes.restype = ctypes.c_size_t
        lib.vdn_host_staging_bytes.argtypes = [C]
        lib.vdn_hybrid_attn_fwd_host.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_size_t, C, P]
        V, L, R = ctypes.POINTER(VdnView), ctypes.POINTER(VdnLinearCfg), ctypes.POINTER(VdnNormCfg)
        lib.vdn_linear_validate.argtypes = [L]
        lib.vdn_linear_workspace_bytes.restype = ctypes.c_size_t
        lib.vdn_linear_workspace_bytes.argtypes = [L, ctypes.c_int32]
        lib.vdn_linear_attn_fwd.argtypes = [V, V, V, V, L, P]
        lib.vdn_linear_attn_bwd.argtypes = [V, V, V, V, V, V, V, L, P]
        lib.vdn_linear_attn_step.argtypes = [V, V, V, V, L, P]
        lib.vdn_norm_validate.argtypes = [R]
        lib.vdn_norm_workspace_bytes.restype = ctypes.c_size_t
        lib.vdn_norm_workspace_bytes.argtypes = [R]
        lib.vdn_add_rmsnorm_fwd.argtypes = [P, P, P, P, P, R, P]
        lib.vdn_add_rmsnorm_bwd.argtypes = [P, P, P, P, P, R, P]
        for name in EXPORTED:
            if name not in ("vdn_version", "vdn_status_string", "vdn_workspace_bytes", "vdn_static_scratch_bytes",
                            "vdn_host_staging_bytes", "vdn_linear_workspace_bytes", "vdn_norm_workspace_bytes"):
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


@dataclass
class Shape:
    """Sizes of one call: batch, latent frames, tokens per frame, heads,
    head_dim, text tokens, frames per chunk."""
    B: int
    F: int
    P: int
    H: int
    d: int
    T: int
    C: int
    fp32: bool = False

    @property
    def N(self) -> int:
        return self.F * self.P


ANCHOR_LOCAL, ANCHOR_GLOBAL = 0, 1
OUTPUT_MERGED, OUTPUT_SPLIT = 0, 1
PREC_BF16, PREC_FP8 = 0, 1
READOUT_SEPARATE, READOUT_FUSED = 0, 1


def make_cfg(s: Shape, *, softmax_scale: float = 0.0, rms_eps: float = -1.0, rms_weight=None,
             debug_flags: int = 0, workspace=None, status=None, export=None,
             anchor_query_mode: int = ANCHOR_LOCAL, out_linear=None, softmax_precision: int = PREC_BF16,
             readout_mode: int = READOUT_SEPARATE) -> VdnCfg:
    cfg = VdnCfg()
    cfg.batch, cfg.frames, cfg.tokens_per_frame = s.B, s.F, s.P
    cfg.heads, cfg.head_dim, cfg.text_tokens, cfg.chunk_frames = s.H, s.d, s.T, s.C
    cfg.dtype = VDN_FP32 if s.fp32 else VDN_BF16
    cfg.softmax_scale = softmax_scale
    cfg.rms_eps = rms_eps
    cfg.rms_weight = _ptr(rms_weight)
    cfg.debug_flags = debug_flags
    cfg.anchor_query_mode = anchor_query_mode
    cfg.output_mode = OUTPUT_SPLIT if out_linear is not None else OUTPUT_MERGED
    cfg.softmax_precision = softmax_precision
    cfg.out_linear = _ptr(out_linear)
    cfg.readout_mode = readout_mode
    if workspace is not None:
        cfg.workspace = workspace.data_ptr()
        cfg.workspace_bytes = workspace.numel() * workspace.element_size()
    cfg.status_word = _ptr(status)
    if export is not None:
        cfg.export_fwd = export[0].data_ptr()
        cfg.export_bwd = export[1].data_ptr()
    return cfg


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(code: int, where: str):
    if code != 0:
        raise VdnError(code, where)


def _stream(stream=None) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def shape_of(q: torch.Tensor, text_k: torch.Tensor, frames: int, chunk_frames: int) -> Shape:
    B, N, H, d = q.shape
    if N % frames:
        raise ValueError("video tokens must be frames * tokens_per_frame")
    return Shape(B, frames, N // frames, H, d, text_k.shape[1], chunk_frames, q.dtype == torch.float32)


def workspace_bytes(s: Shape, softmax_precision: int = PREC_BF16) -> int:
    cfg = make_cfg(s, softmax_precision=softmax_precision)
    n = library().vdn_workspace_bytes(ctypes.byref(cfg))
    if n == 0:
        _check(library().vdn_validate(ctypes.byref(cfg)), "vdn_workspace_bytes")
    return n


_WS: dict = {}


def new_workspace(s: Shape, device, softmax_precision: int = PREC_BF16) -> torch.Tensor:
    """A fresh device workspace for shape s (one per call in flight)."""
    return torch.empty(workspace_bytes(s, softmax_precision), dtype=torch.uint8, device=torch.device(device))


def workspace_for(s: Shape, device, softmax_precision: int = PREC_BF16) -> torch.Tensor:
    """A cached device workspace large enough for shape s."""
    n = workspace_bytes(s, softmax_precision)
    dev = torch.device(device)
    key = (dev.index if dev.index is not None else torch.cuda.current_device())
    buf = _WS.get(key)
    if buf is None or buf.numel() < n:
        buf = torch.empty(n, dtype=torch.uint8, device=dev)
        _WS[key] = buf
    return buf


def hybrid_attn_fwd(q, k, v, text_k, text_v, gate_s, gate_l, *, frames: int, chunk_frames: int, out=None,
                    softmax_scale: float = 0.0, rms_eps: float = -1.0, rms_weight=None, debug_flags: int = 0,
                    workspace=None, status=None, export=None, stream=None,
                    anchor_query_mode: int = ANCHOR_LOCAL, out_linear=None,
                    softmax_precision: int = PREC_BF16, readout_mode: int = READOUT_SEPARATE) -> torch.Tensor:
    """The whole hybrid attention call on the current CUDA stream.

    q, k, v, gate_s, gate_l: [B, F*P, H, d]; text_k, text_v: [B, T, H, d];
    all contiguous CUDA tensors of one dtype (bf16 or fp32).  With
    ``out_linear`` (a tensor like q) the SPLIT output is written: ``out``
    gets sigmoid(gate_s) * o_s and ``out_linear`` sigmoid(gate_l) * r.
    ``readout_mode=READOUT_FUSED`` runs the readout and merge in the softmax
    kernel's epilogue (bf16, head_dim 128, merged output)."""
    s = shape_of(q, text_k, frames, chunk_frames)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = workspace_for(s, q.device, softmax_precision)
    cfg = make_cfg(s, softmax_scale=softmax_scale, rms_eps=rms_eps, rms_weight=rms_weight,
                   debug_flags=debug_flags, workspace=workspace, status=status, export=export,
                   anchor_query_mode=anchor_query_mode, out_linear=out_linear,
                   softmax_precision=softmax_precision, readout_mode=readout_mode)
    code = library().vdn_hybrid_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(text_k), _ptr(text_v),
                                         gate_s.data_ptr(), gate_l.data_ptr(), out.data_ptr(),
                                         ctypes.byref(cfg), _stream(stream))
    _check(code, "vdn_hybrid_attn_fwd")
    return out


def export_states(s: Shape, workspace: torch.Tensor, fwd: torch.Tensor, bwd: torch.Tensor, *, stream=None,
                  softmax_precision: int = PREC_BF16) -> None:
    """S_F / z_F and S_B / z_B ([B, F/C, H, d+1, d] fp32 each) recomputed from
    the state partials that the last call on `workspace` left there."""
    cfg = make_cfg(s, workspace=workspace, softmax_precision=softmax_precision)
    _check(library().vdn_export_states(ctypes.byref(cfg), fwd.data_ptr(), bwd.data_ptr(), _stream(stream)),
           "vdn_export_states")


_STAGING: dict = {}


_REC_FIELDS = ("timeouts", "kernel", "block", "warp", "bar_off", "parity")
# kernel ids in the record: 1 state build, 3 softmax (bf16), 31 softmax (fp8),
# 4 readout + merge (TMA-fed), 41 readout + merge (general), 20 causal linear
# memory (bf16), 21 the states of its ranges


def timeout_record(workspace: torch.Tensor) -> dict:
    """The kernels' timeout record: 16 int32 words at byte 64 of the
    workspace, describing the first bounded wait that ran out since the record
    was cleared (kernel id, block, warp, barrier as its byte distance to the
    CTA's abort flag, phase parity, global nanoseconds waited, SM)."""
    w = workspace[64:128].view(torch.int32).cpu().tolist()
    rec = dict(zip(_REC_FIELDS, w[:6]))
    rec["ns"] = (w[6] & 0xFFFFFFFF) | (w[7] << 32)
    rec["sm"] = w[8]
    return rec


def clear_timeout_record(workspace: torch.Tensor) -> None:
    workspace[64:128].zero_()


def staging_bytes(s: Shape, split: bool = False) -> int:
    """Bytes of the device staging buffer :func:`hybrid_attn_fwd_host` needs."""
    cfg = make_cfg(s)
    if split:
        cfg.output_mode = OUTPUT_SPLIT
    n = library().vdn_host_staging_bytes(ctypes.byref(cfg))
    if n == 0:
        _check(library().vdn_validate(ctypes.byref(cfg)), "vdn_host_staging_bytes")
    return n


def new_staging(s: Shape, device, split: bool = False) -> torch.Tensor:
    """A fresh device staging buffer (one per host call in flight)."""
    return torch.empty(staging_bytes(s, split), dtype=torch.uint8, device=torch.device(device))


def staging_for(s: Shape, device, split: bool = False) -> torch.Tensor:
    """A cached device staging buffer for :func:`hybrid_attn_fwd_host`."""
    n = staging_bytes(s, split)
    dev = torch.device(device)
    key = (dev.index if dev.index is not None else torch.cuda.current_device())
    buf = _STAGING.get(key)
    if buf is None or buf.numel() < n:
        buf = torch.empty(n, dtype=torch.uint8, device=dev)
        _STAGING[key] = buf
    return buf


def hybrid_attn_fwd_host(q, k, v, text_k, text_v, gate_s, gate_l, *, frames: int, chunk_frames: int, out=None,
                         softmax_scale: float = 0.0, rms_eps: float = -1.0, rms_weight=None, workspace=None,
                         staging=None, stream=None, anchor_query_mode: int = ANCHOR_LOCAL,
                         out_linear=None, device="cuda", softmax_precision: int = PREC_BF16,
                         readout_mode: int = READOUT_SEPARATE) -> torch.Tensor:
    """The whole call on HOST tensors (contiguous CPU tensors, ideally pinned),
    copies overlapped with the kernels inside the library.  Returns the host
    ``out``; synchronise ``stream`` (default: the current stream of
    ``device``) before reading it."""
    s = shape_of(q, text_k, frames, chunk_frames)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=q.is_pinned())
    if workspace is None:
        workspace = workspace_for(s, device, softmax_precision)
    if staging is None:
        staging = staging_for(s, device, out_linear is not None)
    cfg = make_cfg(s, softmax_scale=softmax_scale, rms_eps=rms_eps, rms_weight=rms_weight, workspace=workspace,
                   anchor_query_mode=anchor_query_mode, out_linear=out_linear, softmax_precision=softmax_precision,
                   readout_mode=readout_mode)
    code = library().vdn_hybrid_attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(text_k), _ptr(text_v),
                                              gate_s.data_ptr(), gate_l.data_ptr(), out.data_ptr(),
                                              staging.data_ptr(), staging.numel(), ctypes.byref(cfg),
                                              _stream(stream))
    _check(code, "vdn_hybrid_attn_fwd_host")
    return out


class Steps:
    """The separately scheduled steps of one call (same arguments as
    :func:`hybrid_attn_fwd`), for per-kernel timing and stream overlap."""

    def __init__(self, q, k, v, text_k, text_v, gate_s, gate_l, out, *, frames, chunk_frames, workspace=None,
                 debug_flags=0, rms_weight=None, export=None, status=None, anchor_query_mode=ANCHOR_LOCAL,
                 out_linear=None, softmax_precision=PREC_BF16, readout_mode=READOUT_SEPARATE):
        self.t = (q, k, v, text_k, text_v, gate_s, gate_l, out)
        self.s = shape_of(q, text_k, frames, chunk_frames)
        self.ws = workspace if workspace is not None else workspace_for(self.s, q.device, softmax_precision)
        self.cfg = make_cfg(self.s, workspace=self.ws, debug_flags=debug_flags, rms_weight=rms_weight,
                            export=export, status=status, anchor_query_mode=anchor_query_mode,
                            out_linear=out_linear, softmax_precision=softmax_precision,
                            readout_mode=readout_mode)
        self.lib = library()

    def stage(self, stream=None):
        q, k, v, tk, tv = self.t[:5]
        _check(self.lib.vdn_stage_inputs(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(tk), _ptr(tv),
                                         ctypes.byref(self.cfg), _stream(stream)), "vdn_stage_inputs")

    def state_build(self, stream=None):
        _, k, v, tk, tv = self.t[:5]
        _check(self.lib.vdn_state_build(k.data_ptr(), v.data_ptr(), _ptr(tk), _ptr(tv), ctypes.byref(self.cfg),
                                        _stream(stream)), "vdn_state_build")

    def state_scan(self, stream=None):
        _check(self.lib.vdn_state_scan(ctypes.byref(self.cfg), _stream(stream)), "vdn_state_scan")

    def sparse_softmax(self, stream=None):
        q, k, v, tk, tv = self.t[:5]
        _check(self.lib.vdn_sparse_softmax(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(tk), _ptr(tv),
                                           ctypes.byref(self.cfg), _stream(stream)), "vdn_sparse_softmax")

    def softmax_and_scan(self, stream=None, gate=True):
        """The softmax branch and the scan; with ``gate`` the kernel also
        applies the softmax branch's gate (as the whole call does)."""
        q, k, v, tk, tv, gs = self.t[:6]
        _check(self.lib.vdn_softmax_and_scan(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(tk), _ptr(tv),
                                             gs.data_ptr() if gate else None, ctypes.byref(self.cfg),
                                             _stream(stream)),
               "vdn_softmax_and_scan")

    def readout_merge(self, stream=None):
        q, gs, gl, out = self.t[0], self.t[5], self.t[6], self.t[7]
        _check(self.lib.vdn_readout_merge(q.data_ptr(), gs.data_ptr(), gl.data_ptr(), out.data_ptr(),
                                          ctypes.byref(self.cfg), _stream(stream)), "vdn_readout_merge")

    def softmax_merge(self, stream=None):
        """The softmax branch with the scan inside and the readout and merge
        in its epilogue (after state_build)."""
        q, k, v, tk, tv, gs, gl, out = self.t
        _check(self.lib.vdn_sparse_softmax_merge(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(tk), _ptr(tv),
                                                 gs.data_ptr(), gl.data_ptr(), out.data_ptr(),
                                                 ctypes.byref(self.cfg), _stream(stream)),
               "vdn_sparse_softmax_merge")

    def all_fused(self, stream=None):
        """The sequence of a call with the fused readout."""
        self.state_build(stream)
        self.softmax_merge(stream)

    def all(self, stream=None):
        """The whole call's sequence (the scan inside the softmax kernel)."""
        self.stage(stream)
        self.state_build(stream)
        self.softmax_and_scan(stream)
        self.readout_merge(stream)

    def all_separate(self, stream=None):
        """The same result with the scan as a kernel of its own."""
        self.stage(stream)
        self.state_build(stream)
        self.state_scan(stream)
        self.sparse_softmax(stream)
        self.readout_merge(stream)


def plan_membership(F: int, C: int, anchor_query_mode: int = ANCHOR_LOCAL) -> np.ndarray:
    """Host membership table from the library (1 softmax, 2 forward, 3 backward)."""
    s = Shape(1, F, 1, 1, 64, 0, C)
    table = np.zeros((F, F), dtype=np.uint8)
    cfg = make_cfg(s, anchor_query_mode=anchor_query_mode)
    _check(library().vdn_plan_membership(ctypes.byref(cfg), table.ctypes.data), "vdn_plan_membership")
    return table


def membership_device(F: int, C: int, P: int = 1, T: int = 0, device="cuda",
                      anchor_query_mode: int = ANCHOR_LOCAL) -> np.ndarray:
    """The membership table as the kernels' index logic produces it on the GPU."""
    s = Shape(1, F, P, 1, 64, T, C)
    table = torch.zeros((F, F), dtype=torch.uint8, device=device)
    cfg = make_cfg(s, anchor_query_mode=anchor_query_mode)
    _check(library().vdn_membership_device(ctypes.byref(cfg), table.data_ptr(), _stream()),
           "vdn_membership_device")
    torch.cuda.synchronize()
    return table.cpu().numpy()


def validate(s: Shape, **kw) -> int:
    """Status code of the host-side argument check (no CUDA call)."""
    return library().vdn_validate(ctypes.byref(make_cfg(s, **kw)))


# ---------------------------------------------------------------- causal linear memory and residual RMSNorm

# Like all calls here, these are outside autograd: an output carries no gradient and no forward-mode tangent, whatever its
# inputs require, and outputs and states written in place do not count as changes of their tensors.  A training program
# calls the forward and backward functions from a torch.autograd.Function of its own.

NORM_OUT_TENSOR, NORM_OUT_E4M3_ROW, NORM_OUT_E4M3_GROUP = 0, 1, 2
_DTYPES = {torch.bfloat16: VDN_BF16, torch.float32: VDN_FP32}
_HERE = contextlib.nullcontext()
_calls = None  # the extension module of csrc/py/calls.cpp


class _Checked:
    """Stands for the extension module where it cannot be used: every call is left to the code here."""

    linear_fwd = linear_bwd = linear_step = norm_fwd = norm_bwd = staticmethod(lambda *args: None)


def _direct():
    """The module that makes ordinary calls in one step (csrc/py/calls.cpp): each
    of its functions returns None for a call that it leaves to the code here.
    Without it, or with one of another torch, all calls are made here, on the same
    kernels, with some microseconds more on the host."""
    global _calls
    if _calls is None:
        library()
        try:
            from . import _calls as module

            if module.torch_version != str(torch.__version__):
                raise ImportError(f"built with torch {module.torch_version}, this is {torch.__version__}")
            _calls = module
        except ImportError as e:
            warnings.warn(f"the binding's extension module is not used ({e}); rebuild with python -m "
                          "video_diffusion_hybrid_sparse_b200.build", RuntimeWarning, stacklevel=3)
            _calls = _Checked
    return _calls


def _on(t: torch.Tensor, stream):
    """Context in which a call on ``t`` allocates and launches: its device, and
    ``stream`` (of that device) when one is given."""
    if not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    if stream is not None:
        if stream.device != t.device:
            raise ValueError("the stream and the tensors are on different devices")
        return torch.cuda.stream(stream)
    return _HERE if t.get_device() == torch.cuda.current_device() else torch.cuda.device(t.device)


def _here(t: torch.Tensor) -> int:
    """The current stream of the device of ``t``."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _as_stored(name, t):
    """The memory of ``t`` holds its values (torch negates some views lazily)."""
    if t.is_neg():
        raise ValueError(f"{name}: a lazily negated view; call resolve_neg() on it")


def _match(name, t, like):
    """``t`` has the shape, type and device of ``like``, and rows of contiguous elements."""
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name}: expected {tuple(like.shape)} {like.dtype} on {like.device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: the elements of the last dimension must be contiguous")


def _new(like):
    """A contiguous tensor of the shape, type and device of ``like``."""
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _view(name, t, like, shape, dtype, index) -> VdnView:
    """View of a [B, N, H, d] or (a step's) [B, H, d] tensor, checked against ``like``, whose shape, type and device
    number follow."""
    _as_stored(name, t)
    s = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or s[-1] != 1:
        _match(name, t, like)
    return VdnView(t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else VdnView(t.data_ptr(), s[0], 0, s[1])


def _state(name, t, B, H, d, device):
    """Pointer and batch stride of [B, H, d, d] fp32 states (the last three dimensions contiguous)."""
    if t is None:
        return 0, 0
    if t.shape != (B, H, d, d) or t.dtype != torch.float32 or t.device != device:
        raise ValueError(f"{name}: expected {(B, H, d, d)} torch.float32 on {device}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    _as_stored(name, t)
    s = t.stride()
    if s[1:] != (d * d, d, 1) and (H > 1 or s[2:] != (d, 1)):
        raise ValueError(f"{name}: the last three dimensions must be contiguous")
    if B > 1 and s[0] < H * d * d:
        raise ValueError(f"{name}: states must not overlap (an expanded state: copy it)")
    return t.data_ptr(), s[0] if B > 1 else 0


def _flat(name, t, n, dtype, device):
    """Pointer of a contiguous vector of n elements, or 0."""
    if t is None:
        return 0
    if t.shape != (n,) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous ({n},) {dtype} on {device}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    _as_stored(name, t)
    return t.data_ptr()


def _word(name, t, device):
    """Pointer of an int32 status word, or 0."""
    if t is None:
        return 0
    if t.numel() < 1 or t.dtype != torch.int32 or t.device != device:
        raise ValueError(f"{name}: expected an int32 word on {device}, got {tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _sizes(q, dims):
    if q.dim() != dims or q.dtype not in _DTYPES:
        raise ValueError(f"q: expected a {'[B, N, H, d]' if dims == 4 else '[B, H, d]'} bf16 or fp32 tensor, got "
                         f"{tuple(q.shape)} {q.dtype}")
    return q.shape


def linear_workspace_bytes(B: int, N: int, H: int, d: int, dtype=torch.bfloat16, backward: bool = False) -> int:
    """Bytes of workspace of :func:`linear_attn_fwd` (``backward``: :func:`linear_attn_bwd`)."""
    cfg = VdnLinearCfg()
    cfg.batch, cfg.tokens, cfg.heads, cfg.head_dim, cfg.dtype = B, N, H, d, _DTYPES[dtype]
    n = library().vdn_linear_workspace_bytes(ctypes.byref(cfg), int(backward))
    if n == 0:
        _check(library().vdn_linear_validate(ctypes.byref(cfg)), "vdn_linear_workspace_bytes")
    return n


# of sizes only: nothing of a call's tensors is kept
_linear_bytes = functools.lru_cache(maxsize=256)(linear_workspace_bytes)


def _made(r, where):
    """The outputs of a call made in one step, or its error."""
    if r.__class__ is int:
        _check(r, where)
    return r


def _scratch(workspace, n, device):
    """``workspace``, or a new one of ``n`` bytes from the caching allocator: it
    belongs to the current stream (and, during a capture, to that graph), so calls
    on several streams and captured graphs share none."""
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return workspace


def linear_attn_fwd(q, k, v, log_decay, *, scale: float = 0.0, state_in=None, state_out=None, lengths=None, out=None,
                    workspace=None, status=None, stream=None, debug_flags: int = 0) -> torch.Tensor:
    """The causal linear memory with a decay for each head, over whole sequences.

    out_t = scale * q_t S_t with S_t = exp(log_decay[h]) S_{t-1} + k_t^T v_t.

    q, k, v (and out): [B, N, H, d] of one dtype (bf16 or fp32), d in {32, 64,
    128}, any strides that are multiples of 16 bytes with contiguous rows (slices
    of one projection serve); log_decay: [H] fp32, a constant (no gradient);
    state_in, state_out: [B, H, d, d] fp32 or None, state_out is written and may
    be state_in; lengths: [B] int32 or None, the tokens of each padded sequence:
    rows behind them come out as zeros.  ``scale`` <= 0 selects d**-0.5.  A kernel
    whose wait runs out sets ``status`` (int32) to 6; its timeout record is in the
    ``workspace`` of the call (:func:`timeout_record`) where one was given.
    Outside autograd: the output requires no gradient; :func:`linear_attn_bwd`
    forms the gradients."""
    if stream is None and workspace is None:
        r = _direct().linear_fwd(q, k, v, log_decay, scale, state_in, state_out, lengths, out, status, debug_flags)
        if r is not None:
            return _made(r, "vdn_linear_attn_fwd")
    with _on(q, stream):
        B, N, H, d = _sizes(q, 4)
        dev = q.device
        if out is None:
            out = _new(q)
        like = (q, q.shape, q.dtype, q.get_device())
        a, b, c, o = _view("q", q, *like), _view("k", k, *like), _view("v", v, *like), _view("out", out, *like)
        s_in, s_in_stride = _state("state_in", state_in, B, H, d, dev)
        s_out, s_out_stride = _state("state_out", state_out, B, H, d, dev)
        ws = _scratch(workspace, _linear_bytes(B, N, H, d, q.dtype), dev)
        cfg = VdnLinearCfg(B, N, H, d, _DTYPES[q.dtype], scale, _flat("log_decay", log_decay, H, torch.float32, dev),
                      _flat("lengths", lengths, B, torch.int32, dev), s_in, s_out, 0, 0, s_in_stride, s_out_stride, 0, 0,
                      0, 0, debug_flags, ws.data_ptr(), ws.nbytes, _word("status", status, dev))
        _check(library().vdn_linear_attn_fwd(a, b, c, o, ctypes.byref(cfg), _here(q)), "vdn_linear_attn_fwd")
    return out


def linear_attn_bwd(q, k, v, log_decay, d_out, *, scale: float = 0.0, state_in=None, d_state_out=None,
                    d_state_in=None, lengths=None, dq=None, dk=None, dv=None, workspace=None, status=None, stream=None,
                    debug_flags: int = 0):
    """Gradients (dq, dk, dv) of :func:`linear_attn_fwd` by q, k and v, from the
    gradient ``d_out`` by its output and, where given, ``d_state_out`` by its last
    state ([B, H, d, d] fp32); ``d_state_in``, where given, receives the gradient
    by state_in.  Nothing of the forward call is kept: q, k, v and state_in are
    read again.  Rows behind ``lengths`` get zeros."""
    if stream is None and workspace is None:
        r = _direct().linear_bwd(q, k, v, log_decay, d_out, scale, state_in, d_state_out, d_state_in, lengths, dq, dk, dv,
                                 status, debug_flags)
        if r is not None:
            return _made(r, "vdn_linear_attn_bwd")
    with _on(q, stream):
        B, N, H, d = _sizes(q, 4)
        dev = q.device
        dq, dk, dv = (_new(q) if t is None else t for t in (dq, dk, dv))
        like = (q, q.shape, q.dtype, q.get_device())
        views = [_view(n, t, *like) for n, t in (("q", q), ("k", k), ("v", v), ("d_out", d_out), ("dq", dq), ("dk", dk),
                                                 ("dv", dv))]
        s_in, s_in_stride = _state("state_in", state_in, B, H, d, dev)
        ds_out, ds_out_stride = _state("d_state_out", d_state_out, B, H, d, dev)
        ds_in, ds_in_stride = _state("d_state_in", d_state_in, B, H, d, dev)
        ws = _scratch(workspace, _linear_bytes(B, N, H, d, q.dtype, True), dev)
        cfg = VdnLinearCfg(B, N, H, d, _DTYPES[q.dtype], scale, _flat("log_decay", log_decay, H, torch.float32, dev),
                      _flat("lengths", lengths, B, torch.int32, dev), s_in, 0, ds_out, ds_in, s_in_stride, 0,
                      ds_out_stride, ds_in_stride, 0, 0, debug_flags, ws.data_ptr(), ws.nbytes,
                      _word("status", status, dev))
        _check(library().vdn_linear_attn_bwd(*views, ctypes.byref(cfg), _here(q)), "vdn_linear_attn_bwd")
    return dq, dk, dv


def linear_attn_step(q, k, v, log_decay, state, *, slots=None, scale: float = 0.0, out=None, status=None,
                     stream=None) -> torch.Tensor:
    """One token for each of B sequences: the recurrent form of :func:`linear_attn_fwd`.

    q, k, v (and out): [B, H, d]; state: the pool [n, H, d, d] fp32, updated in
    place; slots: [B] int32, the pool entry of each row (None: row b has entry
    b).  A negative slot marks a padding row (out is zero there, no state is
    touched), and so does one past the pool, which also sets ``status`` (int32) to
    1.  Rows of the same slot are successive tokens, in the order of the rows; the
    search for them is quadratic in B (batches of thousands: order the pool and
    leave slots out).  For serving: it has no backward form."""
    if stream is None:
        r = _direct().linear_step(q, k, v, log_decay, state, slots, scale, out, status)
        if r is not None:
            return _made(r, "vdn_linear_attn_step")
    with _on(q, stream):
        B, H, d = _sizes(q, 3)
        dev = q.device
        if out is None:
            out = _new(q)
        like = (q, q.shape, q.dtype, q.get_device())
        a, b, c, o = _view("q", q, *like), _view("k", k, *like), _view("v", v, *like), _view("out", out, *like)
        n = state.shape[0]
        pool, slot_stride = _state("state", state, n, H, d, dev)
        cfg = VdnLinearCfg(B, 0, H, d, _DTYPES[q.dtype], scale, _flat("log_decay", log_decay, H, torch.float32, dev), 0, 0,
                      pool, 0, 0, 0, slot_stride, 0, 0, _flat("slots", slots, B, torch.int32, dev), n, 0, 0, 0,
                      _word("status", status, dev))
        _check(library().vdn_linear_attn_step(a, b, c, o, ctypes.byref(cfg), _here(q)), "vdn_linear_attn_step")
    return out


def _rows(name, t, like, dtype):
    """Pointer and row stride of a tensor of ``dtype`` with the [rows, W] shape and the device of ``like``; 0 for None."""
    if t is None:
        return 0, 0
    if t.shape != like.shape or t.dtype != dtype or t.device != like.device:
        raise ValueError(f"{name}: expected {tuple(like.shape)} {dtype} on {like.device}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    _as_stored(name, t)
    (rows, W), (s0, s1) = t.shape, t.stride()
    if s1 != 1 and W != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if rows <= 1:
        return t.data_ptr(), 0
    if s0 < W:
        raise ValueError(f"{name}: rows must not overlap")
    return t.data_ptr(), s0


def _matrix(x):
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError(f"expected a [rows, width] bf16 or fp32 tensor, got {tuple(x.shape)} {x.dtype}")
    return x.shape


@functools.lru_cache(maxsize=256)
def _norm_bytes(rows, W, dtype):
    cfg = VdnNormCfg()
    cfg.rows, cfg.width, cfg.dtype = rows, W, _DTYPES[dtype]
    n = library().vdn_norm_workspace_bytes(ctypes.byref(cfg))
    if n == 0:
        _check(library().vdn_norm_validate(ctypes.byref(cfg)), "vdn_norm_workspace_bytes")
    return n


def add_rmsnorm_fwd(x, weight=None, *, residual=None, residual_out=None, eps: float = -1.0,
                    out_mode: int = NORM_OUT_TENSOR, out=None, scales=None, stream=None):
    """RMSNorm of h = x + residual: y = h / sqrt(mean(h**2) + eps) * weight.

    x, residual, residual_out: [rows, W], bf16 or fp32, any row stride;
    residual_out, where given, receives h in the tensors' type (it may be x or
    residual, as may out in the tensors' type); weight: [W] fp32 or None (ones).  Returns y in the tensors' type,
    or, for NORM_OUT_E4M3_ROW / NORM_OUT_E4M3_GROUP, (values, scales): e4m3
    [rows, W] and fp32 scales [rows, 1] / [rows, ceil(W / 128)], y ~ value *
    scale.  Outside autograd: no output requires a gradient;
    :func:`add_rmsnorm_bwd` forms those of the tensor output."""
    if stream is None:
        r = _direct().norm_fwd(x, weight, residual, residual_out, eps, out_mode, out, scales)
        if r is not None:
            return _made(r, "vdn_add_rmsnorm_fwd")
    with _on(x, stream):
        rows, W = _matrix(x)
        dev = x.device
        kind, ps = x.dtype, 0
        if out_mode != NORM_OUT_TENSOR:
            if out_mode not in (NORM_OUT_E4M3_ROW, NORM_OUT_E4M3_GROUP):
                raise VdnError(1, "vdn_add_rmsnorm_fwd")
            kind = torch.float8_e4m3fn
            groups = 1 if out_mode == NORM_OUT_E4M3_ROW else (W + 127) // 128
            if scales is None:
                scales = torch.empty_strided((rows, groups), (groups, 1), dtype=torch.float32, device=dev)
            elif scales.shape != (rows, groups) or scales.dtype != torch.float32 or scales.device != dev \
                    or not scales.is_contiguous():
                raise ValueError(f"scales: expected a contiguous {(rows, groups)} torch.float32 on {dev}, got "
                                 f"{tuple(scales.shape)} {scales.dtype} on {scales.device}")
            _as_stored("scales", scales)
            ps = scales.data_ptr()
        if out is None:
            out = torch.empty_like(x, dtype=kind, memory_format=torch.contiguous_format)
        px, x_stride = _rows("x", x, x, x.dtype)
        pr, r_stride = _rows("residual", residual, x, x.dtype)
        ph, h_stride = _rows("residual_out", residual_out, x, x.dtype)
        po, o_stride = _rows("out", out, x, kind)
        cfg = VdnNormCfg(rows, W, _DTYPES[x.dtype], out_mode, eps, _flat("weight", weight, W, torch.float32, dev), x_stride,
                    r_stride, h_stride, o_stride, 0, 0, 0, 0, 0)
        _check(library().vdn_add_rmsnorm_fwd(px, pr, ph, po, ps, ctypes.byref(cfg), _here(x)), "vdn_add_rmsnorm_fwd")
    return out if ps == 0 and kind is x.dtype else (out, scales)


def add_rmsnorm_bwd(h, weight, dy, *, dh=None, eps: float = -1.0, dx=None, dweight=None, want_dweight: bool = True,
                    workspace=None, stream=None):
    """Gradients (dx, dweight) of :func:`add_rmsnorm_fwd` with the tensor output:
    dx, by x and equally by residual, in the tensors' type, and dweight [W] fp32
    (None unless ``want_dweight``).  h: the stored residual_out (or x); dh: the
    gradient that reaches h from elsewhere, or None (dx may be dh)."""
    if stream is None and workspace is None:
        r = _direct().norm_bwd(h, weight, dy, dh, eps, dx, dweight, want_dweight)
        if r is not None:
            return _made(r, "vdn_add_rmsnorm_bwd")
    with _on(h, stream):
        rows, W = _matrix(h)
        dev = h.device
        if dx is None:
            dx = _new(h)
        pw = ws_ptr = ws_bytes = 0
        if not want_dweight:
            dweight = None
        else:
            if dweight is None:
                dweight = torch.empty(W, dtype=torch.float32, device=dev)
            pw = _flat("dweight", dweight, W, torch.float32, dev)
            ws = _scratch(workspace, _norm_bytes(rows, W, h.dtype), dev)
            ws_ptr, ws_bytes = ws.data_ptr(), ws.nbytes
        ph, h_stride = _rows("h", h, h, h.dtype)
        pdy, dy_stride = _rows("dy", dy, h, h.dtype)
        pdh, dh_stride = _rows("dh", dh, h, h.dtype)
        pdx, dx_stride = _rows("dx", dx, h, h.dtype)
        cfg = VdnNormCfg(rows, W, _DTYPES[h.dtype], 0, eps, _flat("weight", weight, W, torch.float32, dev), h_stride, 0, 0, 0,
                    dy_stride, dh_stride, dx_stride, ws_ptr, ws_bytes)
        _check(library().vdn_add_rmsnorm_bwd(ph, pdy, pdh, pdx, pw, ctypes.byref(cfg), _here(h)), "vdn_add_rmsnorm_bwd")
    return dx, dweight
