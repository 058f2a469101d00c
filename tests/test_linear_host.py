"""Refusals of the causal linear memory and of the residual RMSNorm: status codes of the C entry points before any CUDA
call (the pointers are never used), and the binding's own checks."""
import ctypes
import os
import subprocess

import pytest
import torch

from video_diffusion_hybrid_sparse_b200 import binding as vb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # an aligned address that nothing reads


def cfg(**kw):
    c = vb.VdnLinearCfg()
    base = dict(batch=2, tokens=300, heads=4, head_dim=64, dtype=vb.VDN_BF16, log_decay=P, workspace=P,
                workspace_bytes=1 << 40)
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return c


def view(data=P, b=4 * 64 * 300, n=4 * 64, h=64):
    return vb.VdnView(data, b, n, h)


@pytest.mark.parametrize("struct,name", [(vb.VdnLinearCfg, "vdn_linear_cfg"), (vb.VdnNormCfg, "vdn_norm_cfg"),
                                         (vb.VdnView, "vdn_view")])
def test_struct_layouts_match_the_header(struct, name, tmp_path):
    fields = [f[0] for f in struct._fields_]
    src = tmp_path / "layout.c"
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "vdnattn.h"', "int main(void) {"]
    lines += [f'  printf("%zu\\n", offsetof({name}, {f}));' for f in fields]
    lines += [f'  printf("%zu\\n", sizeof({name}));', "  return 0;", "}"]
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(tokens=0), 0), (dict(batch=0), 1), (dict(tokens=-1), 1), (dict(heads=0), 1),
    (dict(head_dim=48), 2), (dict(head_dim=256), 2), (dict(dtype=2), 2), (dict(heads=5000), 2), (dict(tokens=1 << 30), 2),
    (dict(batch=1 << 23), 2), (dict(debug_flags=vb.EXPORT_STATES), 1), (dict(debug_flags=vb.POISON_WS), 0),
])
def test_linear_validate(kw, code):
    c = cfg(**kw)
    assert vb.library().vdn_linear_validate(ctypes.byref(c)) == code
    n = [vb.library().vdn_linear_workspace_bytes(ctypes.byref(c), b) for b in (0, 1)]
    assert all(x >= 256 for x in n) if code == 0 else n == [0, 0]


BAD = [  # (what is wrong, config, status)
    ("no decay", dict(log_decay=None), 1), ("decay misaligned", dict(log_decay=P + 2), 3),
    ("lengths misaligned", dict(lengths=P + 1), 3), ("status misaligned", dict(status_word=P + 2), 3),
    ("state misaligned", dict(state_in=P + 8), 3), ("state stride too small", dict(state_in=P, state_in_stride=64), 1),
    ("state stride misaligned", dict(state_in=P, state_in_stride=4 * 64 * 64 + 1), 3),
    ("no workspace", dict(workspace=None), 4), ("workspace too small", dict(workspace_bytes=255), 4),
    ("workspace misaligned", dict(workspace=P + 128), 3), ("unknown head_dim", dict(head_dim=96), 2),
]


@pytest.mark.parametrize("what,kw,code", BAD, ids=[b[0] for b in BAD])
def test_linear_calls_refuse_configs(what, kw, code):
    lib, c, v = vb.library(), cfg(**kw), view()
    assert lib.vdn_linear_attn_fwd(v, v, v, v, ctypes.byref(c), None) == code
    assert lib.vdn_linear_attn_bwd(v, v, v, v, v, v, v, ctypes.byref(c), None) == code


BAD_VIEWS = [
    ("null", vb.VdnView(None, 0, 0, 0), 1), ("misaligned", view(P + 8), 3), ("token stride misaligned", view(n=260), 3),
    ("negative stride", view(b=-64), 1),
]


@pytest.mark.parametrize("what,bad,code", BAD_VIEWS, ids=[b[0] for b in BAD_VIEWS])
def test_linear_calls_refuse_views(what, bad, code):
    lib, c, good = vb.library(), cfg(state_out=P, n_slots=2), view()
    for i in range(4):
        a = [good] * 4
        a[i] = bad
        assert lib.vdn_linear_attn_fwd(*a, ctypes.byref(c), None) == code
        if "token" not in what:  # the step has no token stride
            assert lib.vdn_linear_attn_step(*a, ctypes.byref(c), None) == code
    for i in range(7):
        a = [good] * 7
        a[i] = bad
        assert lib.vdn_linear_attn_bwd(*a, ctypes.byref(c), None) == code


def test_broadcast_outputs_and_aliases_are_refused():
    lib, good, flat = vb.library(), view(), view(h=0)
    c = cfg()
    assert lib.vdn_linear_attn_fwd(good, good, good, flat, ctypes.byref(c), None) == 1
    assert lib.vdn_linear_attn_bwd(good, good, good, good, good, flat, good, ctypes.byref(c), None) == 1
    c = cfg(state_in=P, state_out=P, state_out_stride=8 * 64 * 64)
    assert lib.vdn_linear_attn_fwd(good, good, good, good, ctypes.byref(c), None) == 1
    c = cfg(d_state_out=P, d_state_in=P)
    assert lib.vdn_linear_attn_bwd(good, good, good, good, good, good, good, ctypes.byref(c), None) == 1


def test_step_refusals():
    lib, v = vb.library(), view()
    for kw, code in ((dict(n_slots=2), 1), (dict(state_out=P), 1), (dict(state_out=P, n_slots=1), 1),
                     (dict(state_out=P + 4, n_slots=2), 3), (dict(state_out=P, n_slots=2, slots=P + 2), 3)):
        assert lib.vdn_linear_attn_step(v, v, v, v, ctypes.byref(cfg(**kw)), None) == code


def norm(**kw):
    c = vb.VdnNormCfg()
    for k, v in {**dict(rows=4, width=100, dtype=vb.VDN_BF16, eps=-1.0), **kw}.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(), 0), (dict(rows=0), 0), (dict(rows=-1), 1), (dict(width=0), 1), (dict(output=3), 1), (dict(output=-1), 1),
    (dict(dtype=5), 2), (dict(x_stride=99), 1), (dict(out_stride=100), 0), (dict(width=(1 << 20) + 1), 2),
    (dict(rows=1 << 31), 2),
])
def test_norm_validate(kw, code):
    lib, c = vb.library(), norm(**kw)
    assert lib.vdn_norm_validate(ctypes.byref(c)) == code
    assert (lib.vdn_norm_workspace_bytes(ctypes.byref(c)) > 0) == (code == 0)
    if code:
        assert lib.vdn_add_rmsnorm_fwd(P, P, P, P, P, ctypes.byref(c), None) == code
        assert lib.vdn_add_rmsnorm_bwd(P, P, P, P, None, ctypes.byref(c), None) == code


def test_norm_refusals():
    lib = vb.library()
    f, b = lib.vdn_add_rmsnorm_fwd, lib.vdn_add_rmsnorm_bwd
    c = norm()
    assert f(None, None, None, P, None, ctypes.byref(c), None) == 1
    assert f(P, None, None, None, None, ctypes.byref(c), None) == 1
    assert f(P + 1, None, None, P, None, ctypes.byref(c), None) == 3
    assert f(P, P + 1, None, P, None, ctypes.byref(c), None) == 3
    assert f(P, None, None, P, None, ctypes.byref(norm(weight=P + 2)), None) == 3
    q = norm(output=vb.NORM_OUT_E4M3_ROW)
    assert f(P, None, None, P, None, ctypes.byref(q), None) == 1
    assert f(P, None, None, P, P + 2, ctypes.byref(q), None) == 3
    assert b(P, P, None, P, None, ctypes.byref(q), None) == 2
    assert b(P, P, None, P, P, ctypes.byref(c), None) == 4
    assert b(P, P, None, P, P, ctypes.byref(norm(workspace=P + 16, workspace_bytes=1 << 30)), None) == 3
    assert b(None, P, None, P, None, ctypes.byref(c), None) == 1
    assert b(P, P, None, P + 1, None, ctypes.byref(c), None) == 3
    assert f(None, None, None, None, None, ctypes.byref(norm(rows=0)), None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    ld = torch.zeros(2)
    with pytest.raises(ValueError):
        vb.linear_attn_fwd(x, x, x, ld)
    with pytest.raises(ValueError):
        vb.linear_attn_bwd(x, x, x, ld, x)
    with pytest.raises(ValueError):
        vb.linear_attn_step(x[:, 0], x[:, 0], x[:, 0], ld, torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError):
        vb.add_rmsnorm_fwd(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        vb.add_rmsnorm_bwd(torch.zeros(2, 8), None, torch.zeros(2, 8))


def test_workspace_follows_the_split():
    """One long head is cut into ranges with states of their own; many heads are not."""
    long = vb.linear_workspace_bytes(1, 100_000, 1, 128)
    assert long > 256 + 64 * 128 * 128 * 4
    assert vb.linear_workspace_bytes(1, 100_000, 1, 128, backward=True) > 256 + 64 * 128 * 128 * 4
    assert vb.linear_workspace_bytes(64, 100_000, 16, 128) == 256
    with pytest.raises(vb.VdnError):
        vb.linear_workspace_bytes(1, 10, 1, 40)


def test_outputs_that_are_inputs_are_refused():
    lib, c = vb.library(), cfg(state_out=P, n_slots=2)
    t = [view((i + 1) << 24) for i in range(7)]
    for i in range(3):
        a = t[:3] + [t[i]]
        assert lib.vdn_linear_attn_fwd(*a, ctypes.byref(c), None) == 1
        assert lib.vdn_linear_attn_step(*a, ctypes.byref(c), None) == 1
    for o in (4, 5, 6):
        for i in [0, 1, 2, 3] + [x for x in (4, 5, 6) if x != o]:
            a = list(t)
            a[o] = t[i]
            assert lib.vdn_linear_attn_bwd(*a, ctypes.byref(c), None) == 1
    Q = 1 << 24
    assert lib.vdn_add_rmsnorm_fwd(P, None, Q, Q, None, ctypes.byref(norm()), None) == 1
    e4m3 = norm(output=vb.NORM_OUT_E4M3_GROUP)
    assert lib.vdn_add_rmsnorm_fwd(P, None, None, P, Q, ctypes.byref(e4m3), None) == 1
    assert lib.vdn_add_rmsnorm_fwd(P, Q, None, Q, P, ctypes.byref(e4m3), None) == 1
    for h, dy in ((Q, P), (P, Q)):
        assert lib.vdn_add_rmsnorm_bwd(h, dy, None, Q, None, ctypes.byref(norm()), None) == 1


def test_rows_in_place_keep_their_stride():
    """An output at an input's address has the input's stride."""
    lib, Q = vb.library(), 1 << 24
    f, b = lib.vdn_add_rmsnorm_fwd, lib.vdn_add_rmsnorm_bwd
    W = norm().width
    for name, args in (("x_stride", (P, None, P, Q)), ("residual_stride", (Q, P, P, 1 << 25)),
                       ("residual_out_stride", (P, None, P, Q)), ("out_stride", (P, Q, None, P)),
                       ("residual_stride", (Q, P, None, P))):
        assert f(*args, None, ctypes.byref(norm(rows=2, **{name: 2 * W})), None) == 1
    assert b(P, Q, 1 << 25, 1 << 25, None, ctypes.byref(norm(rows=2, dh_stride=2 * W)), None) == 1
