"""Refusals of the causal linear memory whose status code another check returns too: every tensor and state has an address
of its own here, so that only the check under test can refuse the call.  No pointer is read: each call ends in its checks."""
import ctypes

import pytest
import torch

from video_diffusion_hybrid_sparse_b200 import binding as vb

B, N, H, D = 2, 300, 4, 64
STATE = H * D * D
INVALID, ALIGNMENT = 1, 3


def at(i):
    return (i + 1) << 28


LOG_DECAY, STATE_IN, STATE_OUT, D_STATE_OUT, D_STATE_IN, WORKSPACE = (at(i) for i in range(20, 26))


def cfg(**kw):
    c = vb.VdnLinearCfg()
    base = dict(batch=B, tokens=N, heads=H, head_dim=D, dtype=vb.VDN_BF16, log_decay=LOG_DECAY, workspace=WORKSPACE,
                workspace_bytes=1 << 40)
    for k, v in {**base, **kw}.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def views(**bad):
    """Seven views at addresses of their own; `bad`: tN=(data, batch, token, head stride)."""
    t = [vb.VdnView(at(i), N * H * D, H * D, D) for i in range(7)]
    for name, (data, b, n, h) in bad.items():
        i = int(name[1:])
        t[i] = vb.VdnView(at(i) if data is None else data, b, n, h)
    return t


def fwd(c, **bad):
    return vb.library().vdn_linear_attn_fwd(*views(**bad)[:4], c, None)


def bwd(c, **bad):
    return vb.library().vdn_linear_attn_bwd(*views(**bad), c, None)


def step(c, **bad):
    return vb.library().vdn_linear_attn_step(*views(**bad)[:4], c, None)


@pytest.mark.parametrize("kw,code", [
    (dict(log_decay=None), INVALID), (dict(log_decay=LOG_DECAY + 2), ALIGNMENT),
    (dict(state_in=STATE_IN, state_in_stride=64), INVALID), (dict(state_in=STATE_IN, state_in_stride=STATE - 4), INVALID),
    (dict(state_in=STATE_IN, state_in_stride=-STATE), INVALID),
])
def test_configs(kw, code):
    assert fwd(cfg(**kw)) == code and bwd(cfg(**kw)) == code
    if "log_decay" in kw:
        assert step(cfg(state_out=STATE_OUT, n_slots=2, **kw)) == code


@pytest.mark.parametrize("kw", [dict(state_out=STATE_OUT, state_out_stride=64)])
def test_forward_states(kw):
    assert fwd(cfg(**kw)) == INVALID
    # in place with another distance between the batch entries
    assert fwd(cfg(state_in=STATE_IN, state_out=STATE_IN, state_out_stride=2 * STATE)) == INVALID
    assert fwd(cfg(state_in=STATE_IN, state_out=STATE_IN, state_in_stride=2 * STATE)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(d_state_out=D_STATE_OUT, d_state_out_stride=64), dict(d_state_in=D_STATE_IN, d_state_in_stride=64),
    dict(d_state_out=D_STATE_OUT, d_state_in=D_STATE_OUT), dict(state_in=STATE_IN, d_state_in=STATE_IN),
])
def test_backward_states(kw):
    assert bwd(cfg(**kw)) == INVALID


GOOD = (N * H * D, H * D, D)


@pytest.mark.parametrize("bad", [(0, *GOOD), (None, -64, H * D, D), (None, N * H * D, -64, D), (None, N * H * D, H * D, -64),
                                 (None, 1 << 36, H * D, D)],
                         ids=["null", "negative batch", "negative token", "negative head", "too large"])
def test_views(bad):
    for i in range(4):
        assert fwd(cfg(), **{f"t{i}": bad}) == INVALID
        if bad[2] > 0:  # the step has no token stride
            assert step(cfg(state_out=STATE_OUT, n_slots=2), **{f"t{i}": bad}) == INVALID
    for i in range(7):
        assert bwd(cfg(), **{f"t{i}": bad}) == INVALID


@pytest.mark.parametrize("flat", [(None, 0, H * D, D), (None, N * H * D, 0, D), (None, N * H * D, H * D, 0)],
                         ids=["batch", "token", "head"])
def test_broadcast_outputs(flat):
    assert fwd(cfg(), t3=flat) == INVALID
    for i in (4, 5, 6):
        assert bwd(cfg(), **{f"t{i}": flat}) == INVALID
    if flat[2]:
        assert step(cfg(state_out=STATE_OUT, n_slots=2), t3=flat) == INVALID


@pytest.mark.parametrize("kw", [dict(n_slots=2), dict(state_out=STATE_OUT), dict(state_out=STATE_OUT, n_slots=-1),
                                dict(state_out=STATE_OUT, n_slots=1), dict(state_out=STATE_OUT, n_slots=2, state_out_stride=64)],
                         ids=["no pool", "no entries", "negative entries", "fewer entries than rows", "entries overlap"])
def test_step(kw):
    assert step(cfg(**kw)) == INVALID


@pytest.mark.parametrize("tokens", [-7, 1 << 30, 0, 5])
def test_step_does_not_read_tokens(tokens):
    """Whatever cfg.tokens holds, the step goes on to its later checks (here: an output that is an input)."""
    same = (at(0), *GOOD)
    assert step(cfg(state_out=STATE_OUT, n_slots=2, tokens=tokens), t3=same) == INVALID
    assert step(cfg(state_out=STATE_OUT + 8, n_slots=2, tokens=tokens)) == ALIGNMENT
    assert step(cfg(state_out=STATE_OUT, n_slots=2, tokens=tokens), t1=(at(1) + 8, *GOOD)) == ALIGNMENT


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 1e-40])
def test_scales_that_are_not_numbers(scale):
    """A scale above 0 is a normal number (its inverse enters the backward call); a NaN does not select the default."""
    assert fwd(cfg(scale=scale)) == INVALID and bwd(cfg(scale=scale)) == INVALID
    assert step(cfg(scale=scale, state_out=STATE_OUT, n_slots=2)) == INVALID
    assert vb.library().vdn_linear_validate(cfg(scale=scale)) == INVALID


@pytest.mark.parametrize("scale", [0.0, -1.0, -float("inf"), 1.2e-38, 3.4e38])
def test_scales(scale):
    assert vb.library().vdn_linear_validate(cfg(scale=scale)) == 0


def test_negated_views_are_refused():
    """A lazily negated tensor's memory holds other values than the tensor: the binding refuses it wherever it goes."""
    t, neg = torch.ones(2, 3, 2, 32), torch._neg_view(torch.ones(2, 3, 2, 32))
    like = (t, t.shape, t.dtype, t.get_device())
    rows, states, vector = torch.ones(4, 8), torch.ones(2, 2, 32, 32), torch.ones(5)
    assert vb._view("k", t, *like).data == t.data_ptr() and vb._rows("x", rows, rows, rows.dtype)[0] == rows.data_ptr()
    for f in (lambda: vb._view("k", neg, *like), lambda: vb._rows("x", torch._neg_view(rows), rows, rows.dtype),
              lambda: vb._state("state_in", torch._neg_view(states), 2, 2, 32, states.device),
              lambda: vb._flat("weight", torch._neg_view(vector), 5, vector.dtype, vector.device)):
        with pytest.raises(ValueError, match="negat"):
            f()
