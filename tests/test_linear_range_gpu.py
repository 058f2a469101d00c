"""The causal linear memory at the ends of its decays' range, and the record of its waits that run out."""
import pytest
import torch

import linear_reference as R
from video_diffusion_hybrid_sparse_b200 import binding as vb

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def tensors(B, N, H, d, dtype, seed):
    g = torch.Generator("cuda").manual_seed(1000 * seed + 7 * N + d)
    return [torch.randn(B, N, H, d, device="cuda", generator=g).to(dtype) for _ in range(4)]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N,lengths,log_decay", [
    (1, None, (1.0, 0.5)), (10, None, (1.0, 2.0)), (40, None, (1.0, 0.7)), (127, None, (0.6, 0.1)),
    (300, [10, 0, 25], (1.0, 0.9)), (300, [300, 129, 1], (0.2, 0.01)), (3000, [3000, 2050, 40], (0.02, -0.01)),
])
def test_growing_memory_of_short_sequences(N, lengths, log_decay, d, dtype):
    """Decays above 1 whose power over a whole chunk has no fp32, in sequences that end before: all results are finite, those
    of the formula."""
    B, H = 3, 2
    ld = torch.tensor(log_decay, device="cuda")
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q, k, v, do = tensors(B, N, H, d, dtype, 1)
    g = torch.Generator("cuda").manual_seed(5)
    s0, ds = (torch.randn(B, H, d, d, device="cuda", generator=g) for _ in range(2))
    for init, dlast in ((None, None), (s0, ds)):
        ref = R.forward(q, k, v, ld, d ** -0.5, init, n)
        state, din = torch.empty_like(s0), torch.empty_like(s0)
        out = vb.linear_attn_fwd(q, k, v, ld, state_in=init, state_out=state, lengths=n)
        R.check(out, ref["out"], "out", dtype, d, N)
        R.check(state, ref["state"], "state", dtype, d, N)
        ref = R.backward(q, k, v, ld, d ** -0.5, do, init, dlast, n)
        grads = vb.linear_attn_bwd(q, k, v, ld, do, state_in=init, d_state_out=dlast, d_state_in=din, lengths=n)
        for name, got in zip(("dq", "dk", "dv", "d_state_in"), (*grads, din)):
            R.check(got, ref[name], name, dtype, d, N)


@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("N,d", [(500, 64), (500, 128), (9000, 128)])
def test_timeout_record(N, d, backward):
    """The wait that the injected timeout lets run out is the one in the record: kernel 20, block 0, the warp that issues the
    scores, 88 bytes before the flag, after 10 ms and before the limit of the other waits."""
    q, k, v, do = tensors(1, N, 2, d, BF16, 2)
    ld, status = torch.tensor([-0.01, -0.1], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(vb.linear_workspace_bytes(1, N, 2, d, BF16, backward), dtype=torch.uint8, device="cuda")

    def call(**kw):
        if backward:
            return vb.linear_attn_bwd(q, k, v, ld, do, workspace=ws, status=status, **kw)
        return vb.linear_attn_fwd(q, k, v, ld, workspace=ws, status=status, **kw)

    vb.clear_timeout_record(ws)
    call(debug_flags=vb.INJECT_TIMEOUT)
    assert int(status) == 6
    rec = vb.timeout_record(ws)
    assert {x: rec[x] for x in ("timeouts", "kernel", "block", "warp", "bar_off", "parity")} == {
        "timeouts": 1, "kernel": 20, "block": 0, "warp": 1, "bar_off": 88, "parity": 0}, rec
    assert 10_000_000 <= rec["ns"] < 1_000_000_000 and 0 <= rec["sm"] < 148
    vb.clear_timeout_record(ws)
    status.zero_()
    call()
    assert int(status) == 0 and vb.timeout_record(ws)["timeouts"] == 0


def test_outside_autograd():
    """No output requires a gradient; a function of the user's own carries the gradients of the two calls."""
    B, N, H, d = 2, 70, 2, 64
    q, k, v, do = (t.requires_grad_() for t in tensors(B, N, H, d, FP32, 3))
    ld = torch.tensor([-0.01, -0.1], device="cuda")
    assert not vb.linear_attn_fwd(q, k, v, ld).requires_grad
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    assert not vb.add_rmsnorm_fwd(x).requires_grad

    class Memory(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_decay):
            ctx.save_for_backward(q, k, v, log_decay)
            return vb.linear_attn_fwd(q, k, v, log_decay)

        @staticmethod
        def backward(ctx, d_out):
            return (*vb.linear_attn_bwd(*ctx.saved_tensors, d_out.contiguous()), None)

    Memory.apply(q, k, v, ld).backward(do.detach())
    ref = R.backward(q.detach(), k.detach(), v.detach(), ld, d ** -0.5, do.detach())
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        R.check(t.grad, ref[name], name, FP32, d, N)


def many_chunks(B, N, H, d, dtype):
    """Decays whose memory spans some thousand chunks: the states, which are fp32, are those of the formula in norm, though
    lambda^128 (or lambda^64) is a factor of every chunk.  A state's chain has N / 64 roundings of at most 2^-24 in no order:
    their root mean square is below sqrt(N / 64) / sqrt(3) * 2^-24; the sums inside a chunk and (bf16) the third part's 2^-24
    and the second's 2^-20 of a term below 2^-4 come to less than 1e-6."""
    ld = torch.tensor([-1e-6, -3.3e-5, -1e-4, -1e-5], device="cuda")
    g = torch.Generator("cuda").manual_seed(N)
    # values of one sign as a state's mean: errors that all have one direction do not cancel
    q, k, v, do = (torch.randn(B, N, H, d, device="cuda", generator=g).abs().to(dtype) for _ in range(4))
    w = torch.exp(ld.double()[None, :] * torch.arange(N, device="cuda").double()[:, None])  # lambda^i
    limit = (N / 64) ** 0.5 / 3 ** 0.5 * 2.0 ** -24 + 1e-6
    state, din = (torch.empty(B, H, d, d, device="cuda") for _ in range(2))
    vb.linear_attn_fwd(q, k, v, ld, scale=1.0, state_out=state)
    vb.linear_attn_bwd(q, k, v, ld, do, scale=1.0, d_state_in=din)
    for b in range(B):
        for h in range(H):
            s = (k[b, :, h].double() * w[:, h].flip(0)[:, None]).T @ v[b, :, h].double()
            r = (q[b, :, h].double() * (w[:, h] * torch.exp(ld[h].double()))[:, None]).T @ do[b, :, h].double()
            for name, got, want in (("state", state[b, h], s), ("d_state_in", din[b, h], r)):
                e = float((got.double() - want).norm() / want.norm())
                assert e <= limit, (name, b, h, e, limit)


@pytest.mark.parametrize("dtype,B,N,H,d", [(FP32, 1, 100_000, 4, 64), (FP32, 2, 60_000, 4, 128), (FP32, 40, 20_000, 4, 32),
                                           (BF16, 36, 10_000, 4, 128)])
def test_memory_over_many_chunks(dtype, B, N, H, d):
    """Heads in ranges and (bf16) whole ones."""
    many_chunks(B, N, H, d, dtype)


def test_memory_over_many_single_tokens():
    """20000 single tokens: the state is that of the formula in norm, though it is multiplied by lambda once a token.  Each
    of a state's n products is rounded by at most 2^-24 of it, in no order (new keys move it by many roundings): their root
    mean square is below sqrt(n / 3) 2^-24 of the last state's, whose predecessors are not larger.  expm1 is good to 2^-23
    of log_decay, which is 2^-23 n |log_decay| of the oldest term."""
    n, d = 20000, 64
    ld = torch.tensor([-1e-6, -3e-6, -3.3e-5, -2e-4], device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(n, 1, 4, d, device="cuda", generator=g) for _ in range(3))
    pool, out = torch.zeros(1, 4, d, d, device="cuda"), torch.empty(1, 4, d, device="cuda")
    for i in range(n):
        vb.linear_attn_step(q[i], k[i], v[i], ld, pool, out=out)
    for h in range(4):
        w = torch.exp(ld[h].double() * torch.arange(n - 1, -1, -1, device="cuda").double())
        want = (k[:, 0, h].double() * w[:, None]).T @ v[:, 0, h].double()
        e = float((pool[0, h].double() - want).norm() / want.norm())
        limit = (n / 3) ** 0.5 * 2.0 ** -24 + 2.0 ** -23 * n * abs(float(ld[h]))
        assert e <= limit, (h, e, limit)


@pytest.mark.parametrize("B,N,d", [(1, 100_000, 64), (2, 60_000, 128), (40, 20_000, 32), (8, 60_000, 64), (1, 241_920, 128)])
def test_sums_over_many_chunks(B, N, d):
    """bf16 heads in ranges, whose states are summed over dozens of chunks on the tensor cores."""
    many_chunks(B, N, 4, d, BF16)


def test_sums_without_decay():
    """The same without a decay, where the keys' first part is all of them."""
    B, N, H, d = 8, 60_000, 4, 64
    ld, g = torch.zeros(H, device="cuda"), torch.Generator("cuda").manual_seed(N)
    q, k, v, do = (torch.randn(B, N, H, d, device="cuda", generator=g).abs().to(BF16) for _ in range(4))
    state, din = (torch.empty(B, H, d, d, device="cuda") for _ in range(2))
    vb.linear_attn_fwd(q, k, v, ld, scale=1.0, state_out=state)
    vb.linear_attn_bwd(q, k, v, ld, do, scale=1.0, d_state_in=din)
    for got, y, z in ((state, k, v), (din, q, do)):
        want = torch.einsum("nhi,nhj->hij", y[0].double(), z[0].double())
        assert float((got[0].double() - want).norm() / want.norm()) <= (N / 64) ** 0.5 / 3 ** 0.5 * 2.0 ** -24 + 1e-6


@pytest.mark.parametrize("log_decay", [0.0, -1e-6, -0.004, -0.3, -0.7, 0.001])
def test_infinite_state_elements_stay(log_decay):
    """lambda S of an infinite element is that element, at a token, at a chunk and over a range; its neighbours are finite."""
    ld = torch.full((2,), log_decay, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)

    def with_infinities(B, d):
        s = torch.randn(B, 2, d, d, device="cuda", generator=g)
        s[0, 0, 3, 5], s[-1, 1, 0, d - 1] = float("inf"), -float("inf")
        return s

    for d in (32, 64, 128):
        pool = with_infinities(3, d)
        keep = pool.clone()
        q, k, v = (torch.randn(3, 2, d, device="cuda", generator=g) for _ in range(3))
        vb.linear_attn_step(q, k, v, ld, pool)
        assert torch.equal(pool.isinf(), keep.isinf()) and torch.equal(pool[pool.isinf()], keep[keep.isinf()])
        assert not pool.isnan().any()
    for dtype, B, N, d in ((FP32, 1, 300, 64), (FP32, 1, 9000, 64), (FP32, 2, 9000, 128), (BF16, 1, 300, 64),
                           (BF16, 1, 9000, 128), (BF16, 1, 40000, 32)):
        if N * abs(log_decay) > 80:
            continue  # the power itself is 0
        s0 = with_infinities(B, d)
        q, k, v, _ = tensors(B, N, 2, d, dtype, 4)
        last = torch.empty_like(s0)
        vb.linear_attn_fwd(q, k, v, ld, state_in=s0, state_out=last)
        assert torch.equal(last.isinf(), s0.isinf()) and torch.equal(last[last.isinf()], s0[s0.isinf()]), (dtype, N, d)
        assert not last.isnan().any()
