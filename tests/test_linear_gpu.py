"""vdn_linear_attn_fwd, _bwd and _step against the definition in 64 bits."""
import math

import pytest
import torch

import linear_reference as R
from video_diffusion_hybrid_sparse_b200 import binding as vb

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def decays(H):
    """No decay, ordinary ones, one that forgets at once (lambda = 0), one that nearly does."""
    return torch.tensor([(0.0, -0.004, -0.7, -math.inf, -0.06, -25.0)[h % 6] for h in range(H)], device="cuda")


def tensors(B, N, H, d, dtype, seed=0, packed=False, names="qkv"):
    g = torch.Generator("cuda").manual_seed(1000 * seed + 7 * N + d)
    t = [torch.randn(B, N, H, d, device="cuda", generator=g).to(dtype) for _ in names]
    if packed:
        return torch.stack(t, 2).unbind(2)
    return t


def states(B, H, d, seed):
    return torch.randn(B, H, d, d, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


SHAPES = [
    (1, 1, 1, 32), (1, 1, 2, 64), (2, 1, 3, 128), (1, 2, 2, 128), (2, 31, 2, 32), (1, 32, 1, 64), (2, 33, 3, 32),
    (1, 63, 2, 128), (2, 64, 2, 64), (1, 65, 1, 128), (1, 127, 2, 64), (3, 128, 2, 128), (2, 129, 3, 64),
    (1, 255, 2, 32), (2, 257, 2, 128), (1, 300, 5, 128), (1, 1000, 3, 64), (1, 1100, 2, 128), (2, 1300, 1, 32),
]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
def test_forward(B, N, H, d, dtype):
    q, k, v = tensors(B, N, H, d, dtype, packed=N % 2 == 1)
    ld, s0 = decays(H), states(B, H, d, 5)
    for init in (None, s0):
        ref = R.forward(q, k, v, ld, d ** -0.5, init)
        state = torch.full((B, H, d, d), float("nan"), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = vb.linear_attn_fwd(q, k, v, ld, state_in=init, state_out=state, status=status, debug_flags=vb.POISON_WS)
        assert int(status) == 0
        R.check(out, ref["out"], "out", dtype, d, N)
        R.check(state, ref["state"], "state", dtype, d, N)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,N,H,d", SHAPES)
def test_backward(B, N, H, d, dtype):
    q, k, v, do = tensors(B, N, H, d, dtype, packed=N % 2 == 1, names="qkvo")
    ld, s0, ds = decays(H), states(B, H, d, 5), states(B, H, d, 6)
    for init, dlast in ((None, None), (s0, ds)):
        ref = R.backward(q, k, v, ld, d ** -0.5, do, init, dlast)
        din = torch.full((B, H, d, d), float("nan"), device="cuda")
        dq, dk, dv = vb.linear_attn_bwd(q, k, v, ld, do, state_in=init, d_state_out=dlast, d_state_in=din,
                                        debug_flags=vb.POISON_WS)
        for name, got in (("dq", dq), ("dk", dk), ("dv", dv), ("d_state_in", din)):
            R.check(got, ref[name], name, dtype, d, N)


@pytest.mark.parametrize("B,N,H,d", [(1, 4000, 2, 128), (2, 3001, 1, 64), (1, 2500, 3, 32), (150, 400, 1, 64), (1, 1300, 160, 32)])
def test_ranges(B, N, H, d):
    """Heads cut into ranges whose states are formed first: few long heads, more heads than a wave holds; state handed in
    and out in place; the state in fp32 as near as fp32 sums are, in norm."""
    q, k, v, do = tensors(B, N, H, d, BF16, names="qkvo")
    ld, s0, ds = decays(H)[torch.arange(H) * 5 % min(H, 6)], states(B, H, d, 5), states(B, H, d, 6)
    ref = R.forward(q, k, v, ld, d ** -0.5, s0)
    state = s0.clone()
    out = vb.linear_attn_fwd(q, k, v, ld, state_in=state, state_out=state, debug_flags=vb.POISON_WS)
    R.check(out, ref["out"], "out", BF16, d, N)
    R.check(state, ref["state"], "state", BF16, d, N)
    assert (state.double() - ref["state"][0]).norm() <= 1e-6 * ref["state"][0].norm()
    ref = R.backward(q, k, v, ld, d ** -0.5, do, s0, ds)
    din = torch.empty_like(s0)
    grads = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=ds, d_state_in=din, debug_flags=vb.POISON_WS)
    for name, got in zip(("dq", "dk", "dv", "d_state_in"), (*grads, din)):
        R.check(got, ref[name], name, BF16, d, N)


def test_decay_beyond_the_ranges():
    """Decays that end inside a chunk, a range or never, in one long head each; keys only in the far past."""
    N, H, d = 9000, 6, 64
    q, k, v = tensors(1, N, H, d, BF16)
    ld = torch.tensor([0.0, -1e-4, -0.004, -0.03, -0.5, -3.0], device="cuda")
    for lo in (0, N - 300):
        k2 = k.clone()
        k2[:, :lo] = 0
        if lo:
            k2[:, lo + 40:] = 0
        ref = R.forward(q, k2, v, ld, 0.2)
        state = torch.empty(1, H, d, d, device="cuda")
        out = vb.linear_attn_fwd(q, k2, v, ld, scale=0.2, state_out=state)
        R.check(out, ref["out"], "out", BF16, d, N)
        R.check(state, ref["state"], "state", BF16, d, N)


def test_one_row_for_all_tokens():
    """A tensor whose token stride is 0 has no TMA view: the other kernels serve it."""
    B, N, H, d = 2, 300, 2, 64
    q, _, v = tensors(B, N, H, d, BF16)
    k = tensors(B, 1, H, d, BF16)[0].expand(B, N, H, d)
    ld = decays(H)
    ref = R.forward(q, k, v, ld, d ** -0.5)
    R.check(vb.linear_attn_fwd(q, k, v, ld), ref["out"], "out", BF16, d, N)


@pytest.mark.parametrize("d", [64, 128])
def test_injected_timeout(d):
    """A wait that runs out ends the call with VDN_ERR_TIMEOUT in the status word; the context stays usable."""
    q, k, v = tensors(1, 500, 2, d, BF16)
    ld = decays(2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vb.linear_attn_fwd(q, k, v, ld, status=status, debug_flags=vb.INJECT_TIMEOUT)
    assert int(status) == 6
    status.zero_()
    ref = R.forward(q, k, v, ld, d ** -0.5)
    R.check(vb.linear_attn_fwd(q, k, v, ld, status=status), ref["out"], "out", BF16, d, 500)
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,d", [(70, 32), (300, 64), (600, 128)])
def test_padded_batch(N, d, dtype):
    """Rows behind a sequence are not used, whatever they hold, and come out as zeros; a sequence without a token hands
    its state on."""
    H = 2
    lengths = torch.tensor([N, 0, 1, N // 2, N - 1, 129, -3, N + 5], dtype=torch.int32, device="cuda")
    B = len(lengths)
    n = lengths.clamp(0, N)
    q, k, v, do = tensors(B, N, H, d, dtype, names="qkvo")
    ld, s0, ds = decays(H)[[1, 4 % H]], states(B, H, d, 5), states(B, H, d, 6)
    ref_f = R.forward(q, k, v, ld, d ** -0.5, s0, n)
    ref_b = R.backward(q, k, v, ld, d ** -0.5, do, s0, ds, n)
    pad = torch.arange(N, device="cuda")[None, :] >= n[:, None]
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max], device="cuda", dtype=dtype)
    for t in (q, k, v, do):
        t[pad] = bad[torch.arange(int(pad.sum()), device="cuda") % 4][:, None, None]
    state, din = torch.empty_like(s0), torch.empty_like(s0)
    out = vb.linear_attn_fwd(q, k, v, ld, state_in=s0, state_out=state, lengths=lengths, debug_flags=vb.POISON_WS)
    grads = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=ds, d_state_in=din, lengths=lengths,
                               debug_flags=vb.POISON_WS)
    R.check(out, ref_f["out"], "out", dtype, d, N)
    R.check(state, ref_f["state"], "state", dtype, d, N)
    for name, got in zip(("dq", "dk", "dv"), grads):
        R.check(got, ref_b[name], name, dtype, d, N)
        assert (got[pad] == 0).all()
    R.check(din, ref_b["d_state_in"], "d_state_in", dtype, d, N)
    assert (out[pad] == 0).all()
    assert torch.equal(state[1], s0[1]) and torch.equal(state[6], s0[6])


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (FP32, 64), (FP32, 32)])
@pytest.mark.parametrize("lengths", [
    [4000, 0, 1, 2500, 3999, 3000],       # cut by cost, ends inside heads
    [0, 0, 4000, 4000, 4000, 0, 4000],    # sequences without tokens at both ends
    [4000, 300, 0, 0, 0, 0],              # too few tokens for that: equal parts
    [0, 0, 0, 0, 0, 0],
    [4000 - 97 * i for i in range(40)],   # more sequences than are cut so
], ids=["mixed", "ends", "few", "none", "many"])
def test_ragged_ranges(lengths, dtype, d):
    """Padded sequences long enough to be cut into ranges."""
    B, N, H = len(lengths), 4000, 2 if len(lengths) < 10 else 1
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    q, k, v, do = tensors(B, N, H, d, dtype, names="qkvo")
    ld, s0, ds = decays(H), states(B, H, d, 5), states(B, H, d, 6)
    ref_f = R.forward(q, k, v, ld, d ** -0.5, s0, n)
    ref_b = R.backward(q, k, v, ld, d ** -0.5, do, s0, ds, n)
    pad = torch.arange(N, device="cuda")[None, :] >= n[:, None]
    for t in (q, k, v, do):
        t[pad] = float("nan")
    state, din = s0.clone(), torch.empty_like(s0)
    out = vb.linear_attn_fwd(q, k, v, ld, state_in=state, state_out=state, lengths=n, debug_flags=vb.POISON_WS)
    grads = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=ds, d_state_in=din, lengths=n,
                               debug_flags=vb.POISON_WS)
    R.check(out, ref_f["out"], "out", dtype, d, N)
    R.check(state, ref_f["state"], "state", dtype, d, N)
    for name, got in zip(("dq", "dk", "dv"), grads):
        R.check(got, ref_b[name], name, dtype, d, N)
        assert (got[pad] == 0).all()
    R.check(din, ref_b["d_state_in"], "d_state_in", dtype, d, N)
    assert (out[pad] == 0).all()


@pytest.mark.parametrize("dtype,N,d", [(BF16, 700, 128), (BF16, 1500, 64), (FP32, 400, 64), (BF16, 400, 32)])
def test_views_in_place_state_and_guard_rows(dtype, N, d):
    """Slices of a wider tensor in another order of dimensions, a broadcast key, an output inside a larger one (what lies
    around it stays), the state updated in place."""
    B, H = 2, 3
    g = torch.Generator("cuda").manual_seed(3)
    wide = torch.randn(H, B, N + 3, 3 * d, device="cuda", generator=g).to(dtype)
    q = wide[..., :d].permute(1, 2, 0, 3)[:, 1:N + 1]
    v = wide[..., 2 * d:].permute(1, 2, 0, 3)[:, 3:]
    k = torch.randn(B, N, 1, d, device="cuda", generator=g).to(dtype).expand(B, N, H, d)
    box = torch.full((B, N + 2, H + 1, d), 7.0, device="cuda", dtype=dtype)
    pool = torch.randn(5, H, d, d, device="cuda", generator=g)
    keep = pool.clone()
    ld = decays(H)
    ref = R.forward(q, k, v, ld, 0.3, pool[1:5:2][:B])
    state = pool[1:5:2][:B]
    out = vb.linear_attn_fwd(q, k, v, ld, scale=0.3, state_in=state, state_out=state, out=box[:, 1:N + 1, :H])
    R.check(out, ref["out"], "out", dtype, d, N)
    R.check(state, ref["state"], "state", dtype, d, N)
    assert (box[:, 0] == 7).all() and (box[:, -1] == 7).all() and (box[:, :, H] == 7).all()
    assert torch.equal(pool[0::2], keep[0::2])


@pytest.mark.parametrize("dtype,N,d", [(BF16, 5000, 128), (BF16, 6000, 64), (FP32, 1500, 32)])
def test_prompt_in_pieces_then_tokens(dtype, N, d):
    """A prompt in two calls and then token by token through the pool is the prompt in one call."""
    B, H = 2, 2
    q, k, v = tensors(B, N, H, d, dtype)
    ld = torch.tensor([-0.01, -0.2], device="cuda")
    whole = vb.linear_attn_fwd(q, k, v, ld)
    pool = torch.zeros(6, H, d, d, device="cuda")
    cut, tail = N // 3, 5
    state = pool[2:4]
    first = vb.linear_attn_fwd(q[:, :cut], k[:, :cut], v[:, :cut], ld, state_out=state)
    second = vb.linear_attn_fwd(q[:, cut:N - tail], k[:, cut:N - tail], v[:, cut:N - tail], ld, state_in=state,
                                state_out=state)
    slots = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    steps = [vb.linear_attn_step(q[:, i], k[:, i], v[:, i], ld, pool, slots=slots) for i in range(N - tail, N)]
    got = torch.cat([first, second, torch.stack(steps, 1)], 1)
    # both sides are roundings of the same values: twice a bf16 result's bound against the other's magnitude, in the mean
    tol = 2.0 ** -7 if dtype == BF16 else 2e-5
    assert (got.double() - whole.double()).norm() / whole.double().norm() <= tol
    assert (pool[[0, 1, 4, 5]] == 0).all()


@pytest.mark.parametrize("d", [32, 64, 128])
def test_gradient_against_differences(d):
    """The call is linear in q, in (v, state) and in (k, state): central differences with steps as large as the values are
    exact but for rounding."""
    B, N, H = 2, 200, 2
    q, k, v, do, e = tensors(B, N, H, d, FP32, names="qkvoe")
    ld, s0, ds, es = torch.tensor([-0.02, -0.3], device="cuda"), states(B, H, d, 1), states(B, H, d, 2), states(B, H, d, 3)
    din = torch.empty_like(s0)
    dq, dk, dv = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=ds, d_state_in=din)

    def loss(q, k, v, s):
        last = torch.empty_like(s0)
        out = vb.linear_attn_fwd(q, k, v, ld, state_in=s, state_out=last)
        return (out.double() * do.double()).sum() + (last.double() * ds.double()).sum()

    for grad, step, at in ((dq, e, lambda s: (q + s * e, k, v, s0)), (dk, e, lambda s: (q, k + s * e, v, s0)),
                           (dv, e, lambda s: (q, k, v + s * e, s0)), (din, es, lambda s: (q, k, v, s0 + s * es))):
        num = (loss(*at(1.0)) - loss(*at(-1.0))) / 2
        ana = (grad.double() * step.double()).sum()
        # sums of B N H d products of independent values: rounding of 2^-24 of about their root mean square each
        size = (grad.double() * step.double()).norm() * 1e-4 + 1e-3
        assert abs(num - ana) <= size, (float(num), float(ana), float(size))


def step_reference(q, k, v, ld, pool, slots, scale):
    pool, out = pool.double().clone(), torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    for b in range(q.shape[0]):
        s = b if slots is None else int(slots[b])
        if 0 <= s < pool.shape[0]:
            S = torch.exp(ld.double())[:, None, None] * pool[s] + k[b].double()[:, :, None] * v[b].double()[:, None, :]
            pool[s] = S
            out[b] = scale * (q[b].double()[:, :, None] * S).sum(1)
            mag[b] = scale * (q[b].double().abs()[:, :, None] * S.abs()).sum(1)
    return out, mag, pool


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,d,slots", [
    (1, 1, 32, None), (3, 2, 64, None), (2, 3, 128, [4, 1]), (6, 2, 128, [0, -1, 3, 9, 2, -7]),
    (7, 1, 64, [2, 2, 0, 2, -1, 0, 1]), (150, 2, 32, "many"), (1, 5, 64, [5]), (300, 1, 128, "same"),
])
def test_step(B, H, d, slots, dtype):
    """Ordinary rows, padding, slots past the pool, rows that share a slot (successive tokens)."""
    n = 6
    if slots == "many":
        n, slots = 200, torch.randperm(200)[:B].tolist()
    elif slots == "same":
        slots = [3] * B
    q, k, v = (t[:, 0] for t in tensors(B, 3, H, d, dtype, packed=True))
    ld = decays(H)
    pool = states(max(n, B if slots is None else 0), H, d, 8)
    ix = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    out_ref, mag, pool_ref = step_reference(q, k, v, ld, pool, ix, d ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = vb.linear_attn_step(q, k, v, ld, pool, slots=ix, status=status)
    many = 1 if slots is None or len(set(slots)) == len(slots) else B
    # a state element: a product and a sum for each of its tokens; an output: d more
    assert ((pool.double() - pool_ref).abs() <= (3 * many + 2) * 2.0 ** -24 * (pool_ref.abs() + 60)).all()
    tol = (d + 3 * many + 8) * 2.0 ** -24 * (mag + 60) + (out_ref.abs() * 2.0 ** -8 if dtype == BF16 else 0)
    assert ((out.double() - out_ref).abs() <= tol).all()
    assert int(status) == (1 if slots is not None and max(slots) >= n else 0)


def test_step_beyond_32_bit_offsets():
    """The last slot of a pool of more than 2^31 elements, and a slot stride wider than the state."""
    H, d = 1, 128
    n = 2 ** 31 // (d * d) + 2
    base = torch.empty(n * d * d + 64 * d * d, device="cuda")
    pool = base.as_strided((n, H, d, d), (d * d, d * d, d, 1))
    pool[-1].normal_()
    pool[0].zero_()
    keep = pool[-1].clone()
    q, k, v = (t[:, 0] for t in tensors(1, 1, H, d, FP32))
    ld = torch.tensor([-0.5], device="cuda")
    ref, mag, _ = step_reference(q, k, v, ld, keep[None], None, d ** -0.5)
    out = vb.linear_attn_step(q, k, v, ld, pool, slots=torch.tensor([n - 1], dtype=torch.int32, device="cuda"))
    assert ((out.double() - ref).abs() <= (d + 8) * 2.0 ** -24 * mag).all()
    assert (pool[0] == 0).all()
    two = base.as_strided((3, H, d, d), (5 * d * d, d * d, d, 1))
    two.zero_()
    base[d * d:5 * d * d] = 3
    vb.linear_attn_step(q, k, v, ld, two, slots=torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert (base[d * d:5 * d * d] == 3).all() and (two[1] != 0).any() and (two[2] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_forward_beyond_32_bit_offsets(dtype):
    B, N, H, d = 2, 40, 1, 64
    far = 2 ** 31
    flat = torch.empty(far + N * d, device="cuda", dtype=dtype)
    q = flat.as_strided((B, N, H, d), (far, d, d, 1))
    q[0].normal_()
    q[1].normal_()
    ld = decays(H)
    ref = R.forward(q, q, q, ld, 0.1)
    R.check(vb.linear_attn_fwd(q, q, q, ld, scale=0.1), ref["out"], "out", dtype, d, N)


@pytest.mark.parametrize("dtype,N,d", [(BF16, 2000, 128), (FP32, 500, 64)])
def test_streams_graphs_and_repeats(dtype, N, d):
    """Calls on two streams at once and captured ones replayed together share nothing; every run gives the same bits."""
    B, H = 1, 2
    ld = torch.tensor([-0.01, -0.1], device="cuda")
    sets = [tensors(B, N, H, d, dtype, seed=i, names="qkvo") for i in range(3)]

    def call(t, **kw):
        last = torch.empty(B, H, d, d, device="cuda")
        out = vb.linear_attn_fwd(*t[:3], ld, state_out=last, **kw)
        return (out, last) + vb.linear_attn_bwd(*t[:3], ld, t[3], d_state_out=last, **kw)

    want = [call(t) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        for s, t in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(call(t))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3]))
    other = vb.linear_attn_fwd(*sets[0][:3], ld, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(other, want[0][0])
    graphs, outs = [], []
    for t in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(t))
        graphs.append(g)
    for _ in range(2):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_captured_call_with_new_lengths(dtype):
    """A captured call follows the lengths that its tensor holds at the replay."""
    B, N, H, d = 4, 3000, 3, 64
    q, k, v, do = tensors(B, N, H, d, dtype, names="qkvo")
    ld, s0 = decays(H), states(B, H, d, 5)
    lengths = torch.tensor([N, N, N, N], dtype=torch.int32, device="cuda")

    def call(n):
        last, din = torch.empty_like(s0), torch.empty_like(s0)
        out = vb.linear_attn_fwd(q, k, v, ld, state_in=s0, state_out=last, lengths=n)
        return (out, last, din) + vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=last, d_state_in=din, lengths=n)

    call(lengths)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call(lengths)
    for new in ([N, 0, 5, 2000], [0, 0, 0, 0], [100, 100, 100, 2999], [N, N, N, N]):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        want = call(lengths.clone())
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens():
    B, H, d = 2, 2, 64
    q = torch.empty(B, 0, H, d, device="cuda", dtype=BF16)
    s0, s1 = states(B, H, d, 1), torch.full((B, H, d, d), 5.0, device="cuda")
    ld = decays(H)
    assert vb.linear_attn_fwd(q, q, q, ld, state_in=s0, state_out=s1).shape == (B, 0, H, d)
    assert torch.equal(s0, s1)
    vb.linear_attn_fwd(q, q, q, ld, state_out=s1)
    assert (s1 == 0).all()
    vb.linear_attn_bwd(q, q, q, ld, q, d_state_out=s0, d_state_in=s1)
    assert torch.equal(s0, s1)


def test_no_tokens_and_states_far_apart():
    """Batch entries of the states 2 GB apart, which no pitched copy takes."""
    B, H, d, gap = 2, 1, 32, 1 << 29
    q = torch.empty(B, 0, H, d, device="cuda", dtype=BF16)
    far = torch.full((gap + d * d,), 5.0, device="cuda").as_strided((B, H, d, d), (gap, d * d, d, 1))
    s0, ld = states(B, H, d, 1), decays(H)
    vb.linear_attn_fwd(q, q, q, ld, state_in=s0, state_out=far)
    assert torch.equal(far, s0)
    back = torch.zeros_like(s0)
    vb.linear_attn_fwd(q, q, q, ld, state_in=far, state_out=back)
    assert torch.equal(back, s0)
    vb.linear_attn_fwd(q, q, q, ld, state_out=far)
    assert (far == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,N,H,d", [(400, 3, 2, 64), (90, 200, 4, 128), (1, 130, 301, 32), (37, 129, 8, 64)])
def test_many_short_heads(B, N, H, d, dtype):
    """More heads than CTAs: a CTA goes through several, padded and empty ones among them."""
    q, k, v, do = tensors(B, N, H, d, dtype, names="qkvo")
    ld, s0, ds = decays(H), states(B, H, d, 5), states(B, H, d, 6)
    n = torch.arange(B, device="cuda", dtype=torch.int32) * 7919 % (N + 1)
    ref = R.forward(q, k, v, ld, d ** -0.5, s0, n)
    state, din = s0.clone(), torch.empty_like(s0)
    out = vb.linear_attn_fwd(q, k, v, ld, state_in=state, state_out=state, lengths=n, debug_flags=vb.POISON_WS)
    R.check(out, ref["out"], "out", dtype, d, N)
    R.check(state, ref["state"], "state", dtype, d, N)
    ref = R.backward(q, k, v, ld, d ** -0.5, do, s0, ds, n)
    grads = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=ds, d_state_in=din, lengths=n)
    for name, got in zip(("dq", "dk", "dv", "d_state_in"), (*grads, din)):
        R.check(got, ref[name], name, dtype, d, N)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_broadcast_inputs(dtype):
    """One query for all batch entries, one value for all heads; states that share memory are refused."""
    B, N, H, d = 3, 200, 2, 64
    q = tensors(1, N, H, d, dtype)[0].expand(B, N, H, d)
    k = tensors(B, N, H, d, dtype, seed=1)[0]
    v = tensors(B, N, 1, d, dtype, seed=2)[0].expand(B, N, H, d)
    ld = decays(H)
    ref = R.forward(q, k, v, ld, 0.5)
    R.check(vb.linear_attn_fwd(q, k, v, ld, scale=0.5), ref["out"], "out", dtype, d, N)
    one = states(1, H, d, 1).expand(B, H, d, d)
    for kw in (dict(state_in=one), dict(state_out=one)):
        with pytest.raises(ValueError):
            vb.linear_attn_fwd(q, k, v, ld, **kw)
    with pytest.raises(ValueError):
        vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, one)
    with pytest.raises(ValueError):
        vb.linear_attn_bwd(q, k, v, ld, k, d_state_in=one)


def test_growing_memory():
    """log_decay > 0 follows the formula."""
    B, N, H, d = 1, 300, 2, 64
    ld = torch.tensor([0.01, 0.1], device="cuda")
    for dtype in (BF16, FP32):
        q, k, v = tensors(B, N, H, d, dtype)
        ref = R.forward(q, k, v, ld, 0.1)
        state = torch.empty(B, H, d, d, device="cuda")
        R.check(vb.linear_attn_fwd(q, k, v, ld, scale=0.1, state_out=state), ref["out"], "out", dtype, d, N)
        R.check(state, ref["state"], "state", dtype, d, N)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_both_ways_of_a_call(dtype):
    """Calls made in one step and those that go through the binding's own checks (here: with a stream or a workspace given)
    are the same calls."""
    B, N, H, d = 2, 300, 2, 64
    q, k, v, do = tensors(B, N, H, d, dtype, packed=True, names="qkvo")
    ld, s0, n = decays(H), states(B, H, d, 1), torch.tensor([300, 17], dtype=torch.int32, device="cuda")
    here = torch.cuda.current_stream()
    last = [torch.empty_like(s0) for _ in range(2)]
    a = vb.linear_attn_fwd(q, k, v, ld, state_in=s0, state_out=last[0], lengths=n, scale=0.2)
    b = vb.linear_attn_fwd(q, k, v, ld, state_in=s0, state_out=last[1], lengths=n, scale=0.2, stream=here)
    assert torch.equal(a, b) and torch.equal(*last) and a.is_contiguous() and a.stride() == b.stride()
    ws = torch.empty(vb.linear_workspace_bytes(B, N, H, d, dtype, True), dtype=torch.uint8, device="cuda")
    a = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=s0, d_state_in=last[0], lengths=n)
    b = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=s0, d_state_in=last[1], lengths=n, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(*last)
    into = [torch.empty(B, N, H, d, device="cuda", dtype=dtype) for _ in range(3)]
    c = vb.linear_attn_bwd(q, k, v, ld, do, state_in=s0, d_state_out=s0, d_state_in=last[1], lengths=n, dq=into[0],
                           dk=into[1], dv=into[2])
    assert all(x.data_ptr() == y.data_ptr() and torch.equal(x, z) for x, y, z in zip(c, into, a))
    pools = [states(5, H, d, 2), states(5, H, d, 2)]
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    a = vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, pools[0], slots=slots)
    b = vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, pools[1], slots=slots, stream=here)
    assert torch.equal(a, b) and torch.equal(*pools)


def test_binding_refuses_what_does_not_fit():
    B, N, H, d = 2, 40, 2, 64
    q, k, v = tensors(B, N, H, d, BF16)
    ld, s0 = decays(H), states(B, H, d, 1)
    for args, kw in (((q, k[:, :-1], v, ld), {}), ((q, k.float(), v, ld), {}), ((q, k, v, ld.double()), {}),
                     ((q, k, v, ld[:1]), {}), ((q, k, v, ld.cpu()), {}), ((q, k, v, ld), dict(state_in=s0[:1])),
                     ((q, k, v, ld), dict(state_in=s0.transpose(2, 3))), ((q, k, v, ld), dict(state_out=s0.bfloat16())),
                     ((q, k, v, ld), dict(lengths=torch.tensor([1, 2], device="cuda"))),
                     ((q, k, v, ld), dict(out=torch.empty_like(q, dtype=FP32))), ((q[0], k[0], v[0], ld), {}),
                     ((q, k, v.transpose(1, 3).contiguous().transpose(1, 3), ld), {})):
        with pytest.raises(ValueError):
            vb.linear_attn_fwd(*args, **kw)
    with pytest.raises(vb.VdnError):
        vb.linear_attn_fwd(*(t[..., :48] for t in (q, k, v)), ld)
    with pytest.raises(vb.VdnError):  # the output is an input
        vb.linear_attn_fwd(q, k, v, ld, out=k)
    with pytest.raises(vb.VdnError):
        wide = torch.empty(B, N, H, d + 1, device="cuda", dtype=BF16)[..., :d]
        vb.linear_attn_fwd(wide, k, v, ld)
    with pytest.raises(ValueError):
        vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, s0, slots=torch.tensor([0], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, s0[:, :1])
    with pytest.raises(vb.VdnError):  # fewer entries than rows
        vb.linear_attn_step(q[:, 0], k[:, 0], v[:, 0], ld, s0[:1])
