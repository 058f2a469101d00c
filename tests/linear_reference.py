"""The causal linear memory with a decay for each head in 64 bits, from its
definition (a sum over all earlier tokens), with the sums of absolute values
that the error bounds of the tests are made of."""
import torch


def walk(x, y, z, log_decay, lengths, init, reverse):
    """out_i = sum_j lambda^|i-j| (x_i . y_j) z_j + f_i x_i init over j <= i (reverse: j >= i), f_i = lambda^(i+1)
    (reverse: lambda^(n-1-i)), and the state sum_j w_j y_j^T z_j + lambda^n init, w_j = lambda^(n-1-j) (reverse:
    lambda^(j+1)); rows behind a sequence's n tokens are zeros.  Returns out, state and both with absolute values."""
    x, y, z = (t.double() for t in (x, y, z))
    B, N, H, d = x.shape
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    state = torch.zeros(B, H, d, d, dtype=torch.float64, device=x.device)
    state_mag = torch.zeros_like(state)

    def power(l, n):  # lambda^n with lambda^0 = 1 even for lambda = 0
        return torch.where(n == 0, torch.ones_like(n), torch.exp(l * n.clamp(min=1e-300)))

    for b in range(B):
        n = N if lengths is None else min(max(int(lengths[b]), 0), N)
        i = torch.arange(n, dtype=torch.float64, device=x.device)
        gap = (i[None, :] - i[:, None]) if reverse else (i[:, None] - i[None, :])
        for h in range(H):
            l = log_decay[h].double()
            X, Y, Z = x[b, :n, h], y[b, :n, h], z[b, :n, h]
            S0 = torch.zeros(d, d, dtype=torch.float64, device=x.device) if init is None else init[b, h].double()
            D = torch.where(gap >= 0, power(l, gap.clamp(min=0)), 0.0)
            f = power(l, (n - 1 - i) if reverse else i + 1)[:, None]
            w = power(l, i + 1 if reverse else n - 1 - i)[:, None]
            whole = power(l, torch.tensor(float(n), dtype=torch.float64, device=x.device))
            out[b, :n, h] = (X @ Y.T * D) @ Z + f * (X @ S0)
            mag[b, :n, h] = (X.abs() @ Y.abs().T * D) @ Z.abs() + f * (X.abs() @ S0.abs())
            state[b, h] = (w * Y).T @ Z + whole * S0
            state_mag[b, h] = (w * Y.abs()).T @ Z.abs() + whole * S0.abs()
    return out, state, mag, state_mag


def forward(q, k, v, log_decay, scale, state_in=None, lengths=None):
    out, state, mag, state_mag = walk(q, k, v, log_decay, lengths, state_in, False)
    return {"out": (scale * out, scale * mag), "state": (state, state_mag)}


def backward(q, k, v, log_decay, scale, d_out, state_in=None, d_state=None, lengths=None):
    t = lambda s: None if s is None else s.transpose(-1, -2)  # noqa: E731
    ds = None if d_state is None else d_state.double() / scale
    dq, _, dq_m, _ = walk(d_out, v, k, log_decay, lengths, t(state_in), False)
    dk, _, dk_m, _ = walk(v, d_out, q, log_decay, lengths, t(ds), True)
    dv, din, dv_m, din_m = walk(k, q, d_out, log_decay, lengths, ds, True)
    return {n: (scale * a, scale * m) for n, a, m in (("dq", dq, dq_m), ("dk", dk, dk_m), ("dv", dv, dv_m),
                                                      ("d_state_in", din, din_m))}


def check(got, ref, what, dtype, d, n):
    """|got - ref| within what the arithmetic can lose, value by value.  `mag`
    is the value's sum with every term's absolute value.

    fp32 results (fp32 tensors, all states): a value is a chain of at most d + n +
    64 roundings of 2^-24 (dot products, sums over tokens, the decay's own
    error), each relative to a partial sum that mag bounds.  States of bf16
    tensors: a decayed key is kept in three bf16 parts (2^-24 of it), or in two
    (2^-16) where its weight in the state is below 2^-4 of the largest.
    bf16 results: a term's decayed score, or the state it is read from, is
    rounded to bf16 once (2^-8 of mag), the result once (2^-8 of itself)."""
    a, (r, mag) = got.double(), ref
    tol = mag * ((d + n + 64) * 2.0 ** -24)
    if dtype == torch.bfloat16:
        tol = tol + mag * (2.0 ** -16 if got.dtype == torch.float32 else 2.0 ** -8)
    if got.dtype == torch.bfloat16:
        tol = tol + (r.abs() + tol) * 2.0 ** -8
    assert torch.isfinite(a).all(), what
    over = (a - r).abs() - tol
    assert (over <= 1e-37).all(), f"{what}: {float(over.max()):.3e} past the bound, at {int(over.argmax())}"
    if r.norm() > 0 and got.dtype == torch.bfloat16:
        # two independent roundings of at most 2^-8, uniform: 2^-8 / sqrt(3) each in the root mean square of a term
        m = (a - r).norm() / max(float(r.norm()), float(mag.norm()) * 1e-3)
        assert m <= 2.0 ** -7, f"{what}: rel {float(m):.2e}"
