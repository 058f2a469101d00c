"""The causal linear memory with a decay for each head, and the RMSNorm around it: cases, plain forms and exact values.

Five operators, called through the package's binding where ``own`` is true and
computed from elementary torch operations in 32 bits otherwise:

* ``prefill``    out_t = scale * q_t S_t,  S_t = lambda_h S_{t-1} + k_t^T v_t, over whole prompts, with the state handed in
                 and out (``linear_attn_fwd``);
* ``step``       the same for one token of each of many sequences, on a pool of states (``linear_attn_step``);
* ``grad``       the gradients of ``prefill`` by q, k, v and the incoming state (``linear_attn_bwd``);
* ``norm``       RMSNorm of x + residual, the sum written back, the result as e4m3 values with one scale for a row or for
                 each 128 columns, or in the tensors' type (``add_rmsnorm_fwd``);
* ``norm_grad``  its gradients by x (the residual's is the same) and by the weight (``add_rmsnorm_bwd``).
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp32": 4}
_MODES = ("tensor", "row", "group")  # the norm's result: the tensors' type; e4m3, a scale a row; e4m3, a scale for 128 columns


def listed():
    return [
        # a short text prompt in a small model: launches and latency are all there is
        dict(name="prefill short", op="prefill", B=1, N=256, H=8, d=64, type="bf16", ragged=False, packed=False, state=False),
        # a padded batch of four streams that go on from their states, q, k, v as slices of one projection
        dict(name="prefill ragged batch", op="prefill", B=4, N=3840, H=16, d=128, type="bf16", ragged=True, packed=True, state=True),
        # one video of 60 latent frames of 4032 tokens: the longest sequence, few heads
        dict(name="prefill long video", op="prefill", B=1, N=241920, H=4, d=128, type="bf16", ragged=False, packed=False, state=False),
        # 32-bit tensors and an odd length: checks of a model against its 32-bit form
        dict(name="prefill fp32", op="prefill", B=2, N=1031, H=8, d=64, type="fp32", ragged=False, packed=False, state=True),
        # one sequence's next token: the smallest call
        dict(name="step one", op="step", B=1, slots=4, H=8, d=64, type="bf16"),
        # the next token of 192 sequences out of a pool of 256
        dict(name="step many", op="step", B=192, slots=256, H=16, d=128, type="bf16"),
        # a small training batch of odd length, with a state's gradient coming in
        dict(name="grad small", op="grad", B=2, N=1000, H=8, d=64, type="bf16", ragged=False, packed=True, state=True),
        # one training video of 45 latent frames of 1024 tokens
        dict(name="grad video", op="grad", B=1, N=46080, H=16, d=128, type="bf16", ragged=False, packed=False, state=False),
        # a decoding batch of 8 tokens before an 8-bit product
        dict(name="norm few rows", op="norm", rows=8, W=2048, type="bf16", mode="row", residual=True),
        # a whole 15-frame video latent before an 8-bit product with blocks of 128
        dict(name="norm video", op="norm", rows=60480, W=2048, type="bf16", mode="group", residual=True),
        # a small training batch in 32 bits, of a width that no vector divides
        dict(name="norm_grad small", op="norm_grad", rows=1000, W=517, type="fp32", residual=True),
        # the training video's tokens
        dict(name="norm_grad video", op="norm_grad", rows=46080, W=2048, type="bf16", residual=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "step", "grad", "norm", "norm_grad"))
    kind = "fp32" if rng.random() < 0.25 else "bf16"
    if op in ("prefill", "grad"):
        d, H = rng.choice((32, 64, 128)), rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
        B = rng.choice((1, 1, 2, 3, 5, 8))
        most = (300_000_000 if op == "prefill" else 130_000_000) // (_BYTES[kind] * B * H * d)
        return dict(op=op, B=B, N=_spread(rng, 1, min(most, 100_000)), H=H, d=d, type=kind, ragged=rng.random() < 0.4,
                    packed=rng.random() < 0.4, state=rng.random() < 0.5)
    if op == "step":
        d, H = rng.choice((32, 64, 128)), rng.choice((1, 2, 3, 4, 6, 8, 12, 16))
        B = _spread(rng, 1, min(700, 100_000_000 // (H * d * d)))
        return dict(op=op, B=B, slots=B + rng.choice((0, 1, 7, 64)), H=H, d=d, type=kind)
    W = rng.choice((64, 96, 128, 200, 256, 384, 500, 512, 768, 1000, 1024, 1536, 2000, 2048, 4096, 5120, 8192, 12345, 16384))
    rows = _spread(rng, 1, min(70_000, 120_000_000 // W))
    if op == "norm":
        return dict(op=op, rows=rows, W=W, type=kind, mode=rng.choice(_MODES), residual=rng.random() < 0.7)
    return dict(op=op, rows=rows, W=W, type=kind, residual=rng.random() < 0.5)


def _lengths(c):
    """Tokens of each sequence of a padded batch."""
    return [c["N"] - (c["N"] * b * 3) // (4 * c["B"]) if c["ragged"] else c["N"] for b in range(c["B"])]


def _unit(x):
    return x / x.square().mean(-1, keepdim=True).sqrt()


def _decay(H):
    """log lambda of each head: from a memory of two tokens to one of some hundreds, in equal ratios."""
    h = torch.arange(1, H + 1, device="cuda", dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / H)).float()


def prepare(case, seed):
    c, g = case, torch.Generator("cuda").manual_seed(seed)
    t = _TYPES[c["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] in ("prefill", "grad"):
        B, N, H, d = c["B"], c["N"], c["H"], c["d"]
        # q and k as a per-head norm leaves them, v as a projection does
        qkv = [_unit(normal(B, N, H, d)).to(t), _unit(normal(B, N, H, d)).to(t), normal(B, N, H, d).to(t)]
        if c["packed"]:
            qkv = torch.stack(qkv, dim=2).unbind(2)
        s = dict(case=c, q=qkv[0], k=qkv[1], v=qkv[2], log_decay=_decay(H), state_in=None, lengths=None)
        if c["ragged"]:
            s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        if c["state"]:
            s["state_in"] = normal(B, H, d, d)
        if c["op"] == "grad":
            s["d_out"] = normal(B, N, H, d).to(t)
            s["d_state"] = normal(B, H, d, d) if c["state"] else None
        return s
    if c["op"] == "step":
        B, H, d = c["B"], c["H"], c["d"]
        slots = torch.randperm(c["slots"], generator=g, device="cuda")[:B].to(torch.int32)
        return dict(case=c, q=_unit(normal(B, H, d)).to(t), k=_unit(normal(B, H, d)).to(t), v=normal(B, H, d).to(t),
                    log_decay=_decay(H), pool=normal(c["slots"], H, d, d), slots=slots)
    rows, W = c["rows"], c["W"]
    s = dict(case=c, x=normal(rows, W).to(t), gamma=1.0 + 0.1 * normal(W), residual=None)
    if c["op"] == "norm" and c["residual"]:
        s["residual"] = (2.0 * normal(rows, W)).to(t)
    if c["op"] == "norm_grad":
        s["dy"] = normal(rows, W).to(t)
        s["dh"] = normal(rows, W).to(t) if c["residual"] else None
    return s


# ---------------------------------------------------------------- the framework's calls

_EPS = 1e-6


def _own(s):
    from video_diffusion_hybrid_sparse_b200 import binding as vb

    c = s["case"]
    if c["op"] == "prefill":
        state = torch.empty((c["B"], c["H"], c["d"], c["d"]), device="cuda")
        out = vb.linear_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], state_in=s["state_in"], state_out=state,
                                 lengths=s["lengths"])
        return {"out": out, "state": state}
    if c["op"] == "grad":
        d_in = torch.empty((c["B"], c["H"], c["d"], c["d"]), device="cuda")
        dq, dk, dv = vb.linear_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["d_out"], state_in=s["state_in"],
                                        d_state_out=s["d_state"], d_state_in=d_in, lengths=s["lengths"])
        return {"dq": dq, "dk": dk, "dv": dv, "d_state": d_in}
    if c["op"] == "step":
        out = vb.linear_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], slots=s["slots"])
        return {"out": out, "pool": s["pool"]}
    if c["op"] == "norm":
        sum_out = torch.empty_like(s["x"]) if c["residual"] else None
        out = vb.add_rmsnorm_fwd(s["x"], s["gamma"], residual=s["residual"], residual_out=sum_out, eps=_EPS,
                                 out_mode=(vb.NORM_OUT_TENSOR, vb.NORM_OUT_E4M3_ROW, vb.NORM_OUT_E4M3_GROUP)[_MODES.index(c["mode"])])
        out = {"out": out} if c["mode"] == "tensor" else {"values": out[0], "scales": out[1]}
        return {"sum": sum_out, **out} if c["residual"] else out
    dx, dgamma = vb.add_rmsnorm_bwd(s["x"], s["gamma"], s["dy"], dh=s["dh"], eps=_EPS)
    return {"dx": dx, "dgamma": dgamma}


# ---------------------------------------------------------------- the plain forms

_C = 128  # tokens of a chunk of the plain form


def _power(log_decay, n):
    """lambda_h ** n for whole numbers n >= 0 ([..., H] from [...]), the angle in 64 bits; 0 where n < 0."""
    p = torch.exp(log_decay.double() * n.clamp(min=0).double().unsqueeze(-1))
    return torch.where(n.unsqueeze(-1) >= 0, p, torch.zeros_like(p)).float()


def _chunked(x, y, z, log_decay):
    """sum over s <= t of lambda^(t-s) (x_t . y_s) z_s for [B, N, H, d] in 32 bits: products inside chunks of 128 tokens, and
    the states before the chunks, which a matrix of decays over chunks sums from the chunks' own."""
    B, N, H, d = x.shape
    nc = -(-N // _C)
    x, y, z = (torch.nn.functional.pad(t, (0, 0, 0, 0, 0, nc * _C - N)).reshape(B, nc, _C, H, d).permute(0, 3, 1, 2, 4)
               for t in (x, y, z))  # [B, H, nc, C, d]
    i = torch.arange(_C, device=x.device)
    mask = _power(log_decay, i[:, None] - i[None, :]).permute(2, 0, 1)  # [H, C, C]
    out = torch.matmul(torch.matmul(x, y.transpose(-1, -2)) * mask[None, :, None], z)
    own_state = torch.matmul((y * _power(log_decay, _C - 1 - i).t()[None, :, None, :, None]).transpose(-1, -2), z)
    j = torch.arange(nc, device=x.device)
    across = _power(log_decay, torch.where(j[:, None] > j[None, :], (j[:, None] - 1 - j[None, :]) * _C, -1)).permute(2, 0, 1)
    before = torch.matmul(across, own_state.reshape(B, H, nc, d * d)).reshape(B, H, nc, d, d)
    out = out + torch.matmul(x * _power(log_decay, i + 1).t()[None, :, None, :, None], before)
    return out.permute(0, 2, 3, 1, 4).reshape(B, nc * _C, H, d)[:, :N]


def _plain_memory(s):
    c = s["case"]
    q, k, v = (s[n].float() for n in "qkv")
    B, N, H, d = q.shape
    ld, scale = s["log_decay"], d ** -0.5
    t = torch.arange(N, device=q.device)
    n = torch.full((B,), N, device=q.device) if s["lengths"] is None else s["lengths"].long()
    real = (t[None] < n[:, None])[:, :, None, None]
    zero = torch.zeros((), device=q.device)
    q, k, v = (torch.where(real, a, zero) for a in (q, k, v))
    start, tail = _power(ld, t + 1)[None], _power(ld, n[:, None] - 1 - t[None])  # lambda^(t+1); lambda^(n-1-t), 0 from n on
    whole = _power(ld, n)[:, :, None, None]  # lambda^n: [B, H, 1, 1]
    s0 = s["state_in"]
    if c["op"] == "prefill":
        out = _chunked(q, k, v, ld)
        state = torch.matmul((k * tail[..., None]).permute(0, 2, 3, 1), v.permute(0, 2, 1, 3))
        if s0 is not None:
            out = out + start[..., None] * torch.einsum("bnhi,bhij->bnhj", q, s0)
            state = state + whole * s0
        return {"out": (out * scale).to(s["q"].dtype), "state": state}
    do, ds = torch.where(real, s["d_out"].float(), zero), s["d_state"]
    dq = _chunked(do, v, k, ld) * scale
    dk = _chunked(v.flip(1), do.flip(1), q.flip(1), ld).flip(1) * scale
    dv = _chunked(k.flip(1), q.flip(1), do.flip(1), ld).flip(1) * scale
    d_in = scale * torch.matmul((q * start[..., None]).permute(0, 2, 3, 1), do.permute(0, 2, 1, 3))
    if s0 is not None:
        dq = dq + scale * start[..., None] * torch.einsum("bnhj,bhij->bnhi", do, s0)
    if ds is not None:
        dk = dk + tail[..., None] * torch.einsum("bnhj,bhij->bnhi", v, ds)
        dv = dv + tail[..., None] * torch.einsum("bnhi,bhij->bnhj", k, ds)
        d_in = d_in + whole * ds
    return {**{n: a.to(s["q"].dtype) for n, a in (("dq", dq), ("dk", dk), ("dv", dv))}, "d_state": d_in}


def _plain_step(s):
    q, k, v = (s[n].float() for n in "qkv")
    at = s["slots"].long()
    state = torch.exp(s["log_decay"])[None, :, None, None] * s["pool"][at] + k[..., :, None] * v[..., None, :]
    s["pool"][at] = state
    out = (q[..., :, None] * state).sum(-2) * q.shape[-1] ** -0.5
    return {"out": out.to(s["q"].dtype), "pool": s["pool"]}


def _plain_norm(s):
    c = s["case"]
    x, gamma = s["x"].float(), s["gamma"]
    if c["op"] == "norm":
        h = x + s["residual"].float() if c["residual"] else x
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS) * gamma
        out = {"sum": h.to(s["x"].dtype)} if c["residual"] else {}
        if c["mode"] == "tensor":
            return {**out, "out": y.to(s["x"].dtype)}
        rows, W = y.shape
        size = W if c["mode"] == "row" else 128
        groups = -(-W // size)
        y = torch.nn.functional.pad(y, (0, groups * size - W)).reshape(rows, groups, size)
        most = y.abs().amax(-1, keepdim=True)
        scale = torch.where(most > 0, most / 448.0, torch.ones_like(most))
        values = (y / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return {**out, "values": values.reshape(rows, groups * size)[:, :W], "scales": scale.reshape(rows, groups)}
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    dy, xn = s["dy"].float(), x * r
    g = dy * gamma
    dx = r * (g - xn * (g * xn).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xn).sum(0)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_memory(state) if op in ("prefill", "grad") else _plain_step(state) if op == "step" else _plain_norm(state)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    c = case
    e = _BYTES[c["type"]]
    if c["op"] in ("prefill", "grad"):
        H, d = c["H"], c["d"]
        tokens = sum(_lengths(c)) * H
        states = c["B"] * H * d * d * 4
        grad = c["op"] == "grad"
        # q, k, v (and the output's gradient) in, the output (or three gradients) out; a padded row is only written
        rows = tokens * (4 if grad else 3) + c["B"] * c["N"] * H * (3 if grad else 1)
        n_states = (3 if c["state"] else 1) if grad else (2 if c["state"] else 1)
        return {"bytes": rows * d * e + states * n_states + H * 4, "flops": tokens * d * d * (12 if grad else 4)}
    if c["op"] == "step":
        H, d = c["H"], c["d"]
        return {"bytes": c["B"] * H * (2 * d * d * 4 + 4 * d * e) + c["B"] * 4, "flops": c["B"] * H * d * d * 5}
    n, W = c["rows"] * c["W"], c["W"]
    if c["op"] == "norm":
        size = {"tensor": 0, "row": W, "group": 128}[c["mode"]]
        out = n * e if not size else n + c["rows"] * -(-W // size) * 4
        return {"bytes": n * e * (3 if c["residual"] else 1) + out + W * 4, "flops": n * 5}
    return {"bytes": n * e * (4 if c["residual"] else 3) + W * 8, "flops": n * 10}


# ---------------------------------------------------------------- exact values, in 64 bits


def _walk(x, y, z, log_decay, lengths, start, first):
    """Token by token in blocks: out_i = sum over j <= i of lambda^(i-j) (x_i . y_j) z_j + lambda^(i+first) x_i start, with the
    state after the last token, for sequences [H, n, d] in 64 bits. `first`: the power that the first row's start has."""
    outs, states = [], []
    ld = log_decay.double()[:, None, None]
    for b, n in enumerate(lengths):
        S = torch.zeros(x.shape[2], x.shape[3], x.shape[3], dtype=torch.float64, device=x.device) if start is None else start[b].double()
        out = torch.zeros(x.shape[1:], dtype=torch.float64, device=x.device)
        for at in range(0, n, 256):
            m = min(256, n - at)
            X, Y, Z = (t[b, at:at + m].double().transpose(0, 1) for t in (x, y, z))
            i = torch.arange(m, dtype=torch.float64, device=x.device)
            gap = i[:, None] - i[None, :]
            near = torch.einsum("hid,hjd->hij", X, Y) * torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), 0.0)
            out[at:at + m] = (near @ Z + torch.exp(ld[:, 0] * (i + first)[None])[..., None] * (X @ S)).transpose(0, 1)
            fall = torch.exp(ld[:, 0] * (m - first - i)[None])[..., None]
            S = torch.exp(ld * m) * S + (Y * fall).transpose(1, 2) @ Z
        outs.append(out)
        states.append(S)
    return torch.stack(outs), torch.stack(states)


def _back(t, lengths):
    """Each sequence's rows in the other order, the padding behind them."""
    return torch.stack([torch.cat((t[b, :n].flip(0), t[b, n:])) for b, n in enumerate(lengths)])


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("prefill", "grad"):
        n, ld, scale = _lengths(c), s["log_decay"], c["d"] ** -0.5
        if c["op"] == "prefill":
            out, state = _walk(s["q"], s["k"], s["v"], ld, n, s["state_in"], 1)
            return {"out": out * scale, "state": state}
        dq, _ = _walk(s["d_out"], s["v"], s["k"], ld, n, None if s["state_in"] is None else s["state_in"].transpose(-1, -2), 1)
        q, k, v, do = (_back(s[a], n) for a in ("q", "k", "v", "d_out"))
        ds = None if s["d_state"] is None else s["d_state"].double() / scale
        dk, _ = _walk(v, do, q, ld, n, None if ds is None else ds.transpose(-1, -2), 0)
        dv, d_in = _walk(k, q, do, ld, n, ds, 0)
        return {"dq": dq * scale, "dk": _back(dk, n) * scale, "dv": _back(dv, n) * scale, "d_state": d_in * scale}
    if c["op"] == "step":
        q, k, v, pool = (s[a].double() for a in ("q", "k", "v", "pool"))
        at = s["slots"].long()
        S = torch.einsum("h,bhij->bhij", torch.exp(s["log_decay"].double()), pool[at]) + torch.einsum("bhi,bhj->bhij", k, v)
        pool[at] = S
        return {"out": torch.einsum("bhi,bhij->bhj", q, S) / math.sqrt(c["d"]), "pool": pool}
    x, gamma = s["x"].double(), s["gamma"].double()
    if c["op"] == "norm":
        h = x if s["residual"] is None else x + s["residual"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / c["W"] + _EPS) * gamma
        out = {"sum": h} if c["residual"] else {}
        if c["mode"] == "tensor":
            return {**out, "out": y}
        edges = list(range(0, c["W"], c["W"] if c["mode"] == "row" else 128))
        parts = [y[:, a:a + (c["W"] if c["mode"] == "row" else 128)] for a in edges]
        scales = torch.stack([p.abs().max(1).values / 448 for p in parts], 1)
        return {**out, "values": torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], 1), "scales": scales}
    dy = s["dy"].double()
    root = torch.sqrt((x * x).sum(1, keepdim=True) / c["W"] + _EPS)
    # d/dx_j of x_i g_i / root: g_j dy_j / root - x_j (sum_i dy_i g_i x_i) / (W root^3)
    dx = gamma * dy / root - x * (dy * gamma * x).sum(1, keepdim=True) / (c["W"] * root ** 3)
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("rw,rw->w", dy, x / root)}

