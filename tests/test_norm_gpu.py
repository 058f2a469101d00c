"""vdn_add_rmsnorm_fwd and _bwd against the definition in 64 bits."""
import pytest
import torch

from video_diffusion_hybrid_sparse_b200 import binding as vb

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
EPS = 1e-6
SHAPES = [(1, 1), (3, 7), (2, 8), (70, 24), (5, 64), (40, 63), (33, 72), (17, 100), (9, 128), (4, 129), (33, 256), (1, 264), (6, 500), (300, 512),
          (3, 520), (7, 1000), (64, 1024), (5, 2048), (2, 2056), (3, 4096), (2, 5001), (4, 8192), (2, 12345), (3, 16384),
          (2, 16392), (2, 32768), (2, 32776), (1, 50001)]


def rows_of(n, W, dtype, seed, scale=1.0):
    return (scale * torch.randn(n, W, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + W))).to(dtype)


def reference(x, res, gamma):
    h = x.double() if res is None else x.double() + res.double()
    r = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    return h, r, h * r * (1.0 if gamma is None else gamma.double())


def y_error(y, W):
    """Of y in 32 bits, relative: the mean's sum of W squares (at most W / 2 of the root), and a few products."""
    return y.abs() * (W / 2 + 8) * 2.0 ** -24


def check_e4m3(values, scales, y, size, W):
    """Each group's scale is max / 448, and each value its element rounded to e4m3: within 2^-4 of it, or half of the
    smallest step, 2^-10, near zero."""
    n = y.shape[0]
    groups = -(-W // size)
    pad = torch.nn.functional.pad(y, (0, groups * size - W)).reshape(n, groups, size)
    most = pad.abs().amax(2)
    want = torch.where(most > 0, most / 448, torch.ones_like(most))
    err = (W / 2 + 10) * 2.0 ** -24
    assert scales.shape == (n, groups)
    assert ((scales.double() - want).abs() <= want * err).all()
    s = scales.double().repeat_interleave(size, 1)[:, :W]
    v = values.float().double()
    assert ((v - y / s).abs() <= (y / s).abs() * (2.0 ** -4 + 3 * err) + 2.0 ** -10).all()
    top = torch.nn.functional.pad(v, (0, groups * size - W)).reshape(n, groups, size).abs().amax(2)
    assert (top[most > 0] == 448).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,W", SHAPES)
def test_forward(n, W, dtype):
    x, res = rows_of(n, W, dtype, 1), rows_of(n, W, dtype, 2, 3.0)
    gamma = 1.0 + 0.2 * rows_of(1, W, FP32, 3)[0]
    for residual, w in ((None, None), (None, gamma), (res, gamma)):
        h, _, y = reference(x, residual, w)
        stored = torch.full_like(x, float("nan")) if residual is not None else None
        out = vb.add_rmsnorm_fwd(x, w, residual=residual, residual_out=stored, eps=EPS)
        assert ((out.double() - y).abs() <= y_error(y, W) + (y.abs() * HALF[dtype] if dtype == BF16 else 0)).all()
        if stored is not None:
            assert torch.equal(stored, (x.float() + res.float()).to(dtype))
        for mode, size in ((vb.NORM_OUT_E4M3_ROW, W), (vb.NORM_OUT_E4M3_GROUP, 128)):
            values, scales = vb.add_rmsnorm_fwd(x, w, residual=residual, eps=EPS, out_mode=mode)
            check_e4m3(values, scales, y, size, W)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,W", SHAPES + [(1500, 512), (700, 2048), (2000, 40)])
def test_backward(n, W, dtype):
    h, dy, dh = rows_of(n, W, dtype, 1, 2.0), rows_of(n, W, dtype, 2), rows_of(n, W, dtype, 4)
    gamma = 1.0 + 0.2 * rows_of(1, W, FP32, 3)[0]
    H, DY = h.double(), dy.double()
    for w, extra in ((None, None), (gamma, dh)):
        g = DY if w is None else DY * w.double()
        r = 1.0 / torch.sqrt(H.square().mean(1, keepdim=True) + EPS)
        dx = r * g - H * r ** 3 * (g * H).mean(1, keepdim=True)
        size = (r * g).abs() + (H * r ** 3).abs() * (g * H).abs().mean(1, keepdim=True)
        if extra is not None:
            dx, size = dx + extra.double(), size + extra.double().abs()
        dw, dw_size = (DY * H * r).sum(0), (DY * H * r).abs().sum(0)
        got, got_w = vb.add_rmsnorm_bwd(h, w, dy, dh=extra, eps=EPS)
        # sums over W (and, for the weight, over the rows) of 2^-24 each, against the absolute sums
        assert ((got.double() - dx).abs() <= size * (1.5 * W + 16) * 2.0 ** -24
                + (dx.abs() * 1.001 * HALF[dtype] if dtype == BF16 else 0)).all()
        assert ((got_w.double() - dw).abs() <= dw_size * (n + W + 16) * 2.0 ** -24).all()
        only, none = vb.add_rmsnorm_bwd(h, w, dy, dh=extra, eps=EPS, want_dweight=False)
        assert none is None and torch.equal(only, got)


def test_backward_against_differences():
    n, W = 6, 96
    x, dy, e = (rows_of(n, W, FP32, s) for s in (1, 2, 3))
    gamma, eg = 1.0 + 0.2 * rows_of(1, W, FP32, 4)[0], rows_of(1, W, FP32, 5)[0]
    dx, dw = vb.add_rmsnorm_bwd(x, gamma, dy, eps=EPS)
    f = lambda a, w: (vb.add_rmsnorm_fwd(a, w, eps=EPS).double() * dy.double()).sum()  # noqa: E731
    t = 2.0 ** -7  # central difference: t^2 / 6 of the third derivative (order 1 for rows of size 1), 2^-24 / t of rounding
    num = (f(x + t * e, gamma) - f(x - t * e, gamma)) / (2 * t)
    ana = (dx.double() * e.double()).sum()
    assert abs(num - ana) <= 1e-3 * (dx.double() * e.double()).abs().sum()
    num = (f(x, gamma + eg) - f(x, gamma - eg)) / 2
    assert abs(num - (dw.double() * eg.double()).sum()) <= 1e-4 * (dw.double() * eg.double()).abs().sum()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("W,pitch,shift", [(256, 264, 0), (256, 259, 0), (256, 256, 1), (100, 128, 3), (2048, 2050, 2),
                                           (33000, 33001, 1)])
def test_strides_alignment_and_guards(W, pitch, shift, dtype):
    """Rows inside wider ones at any element: what lies around the outputs stays."""
    n = 5
    gamma = 1.0 + 0.2 * rows_of(1, W + shift, FP32, 3)[0][shift:]

    def inside(seed, fill=None):
        t = rows_of(1, n * pitch + 16, dtype, seed)[0] if fill is None else torch.full((n * pitch + 16,), fill, device="cuda", dtype=dtype)
        return t, t[shift:shift + n * pitch].as_strided((n, W), (pitch, 1), shift)

    (_, x), (_, res) = inside(1), inside(2)
    (box, out), (sbox, stored) = inside(0, 7.0), inside(0, 7.0)
    _, _, y = reference(x, res, gamma)
    vb.add_rmsnorm_fwd(x, gamma, residual=res, residual_out=stored, eps=EPS, out=out)
    assert ((out.double() - y).abs() <= y_error(y, W) + (y.abs() * HALF[dtype] if dtype == BF16 else 0)).all()
    assert torch.equal(stored, (x.float() + res.float()).to(dtype))
    for b, o in ((box, out), (sbox, stored)):
        o.fill_(7.0)
        assert (b == 7).all()
    for mode, size in ((vb.NORM_OUT_E4M3_ROW, W), (vb.NORM_OUT_E4M3_GROUP, 128)):
        values, scales = vb.add_rmsnorm_fwd(x, gamma, residual=res, eps=EPS, out_mode=mode)
        check_e4m3(values, scales, y, size, W)
    _, dx = inside(0, 7.0)
    vb.add_rmsnorm_bwd(x, gamma, res, eps=EPS, dx=dx)
    X, g = x.double(), res.double() * gamma.double()
    r = 1.0 / torch.sqrt(X.square().mean(1, keepdim=True) + EPS)
    want = r * g - X * r ** 3 * (g * X).mean(1, keepdim=True)
    size = (r * g).abs() + (X * r ** 3).abs() * (g * X).abs().mean(1, keepdim=True)
    assert ((dx.double() - want).abs() <= size * (1.5 * W + 16) * 2.0 ** -24
            + (want.abs() * 1.001 * HALF[dtype] if dtype == BF16 else 0)).all()


@pytest.mark.parametrize("W", [64, 2048, 40000])
def test_in_place(W):
    x, res = rows_of(4, W, BF16, 1), rows_of(4, W, BF16, 2)
    want_h, want = torch.empty_like(x), None
    want = vb.add_rmsnorm_fwd(x, None, residual=res, residual_out=want_h)
    a = x.clone()
    assert torch.equal(vb.add_rmsnorm_fwd(a, None, residual=res, residual_out=a), want) and torch.equal(a, want_h)
    b = res.clone()
    assert torch.equal(vb.add_rmsnorm_fwd(x, None, residual=b, residual_out=b), want) and torch.equal(b, want_h)
    c = x.clone()
    vb.add_rmsnorm_fwd(c, None, residual=res, out=c)
    assert torch.equal(c, want)
    want, dw = vb.add_rmsnorm_bwd(x, None, res, dh=b)
    dx, dw2 = vb.add_rmsnorm_bwd(x, None, res, dh=b, dx=b)
    assert dx is b and torch.equal(dx, want) and torch.equal(dw, dw2)


@pytest.mark.parametrize("W", [100, 256, 2048, 40000])
def test_special_rows(W):
    """Zeros, tiny and huge values, an infinity, a NaN: each row is its own affair."""
    x = rows_of(7, W, FP32, 1)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e18
    x[4, W // 2] = float("inf")
    x[5, 3] = float("nan")
    values, scales = vb.add_rmsnorm_fwd(x, None, eps=EPS, out_mode=vb.NORM_OUT_E4M3_GROUP)
    row_values, row_scales = vb.add_rmsnorm_fwd(x, None, eps=EPS, out_mode=vb.NORM_OUT_E4M3_ROW)
    _, _, y = reference(x, None, None)
    ok = [0, 1, 2, 3, 6]
    check_e4m3(values[ok], scales[ok], y[ok], 128, W)
    check_e4m3(row_values[ok], row_scales[ok], y[ok], W, W)
    assert (values[1].float() == 0).all() and (scales[1] == 1).all() and float(row_scales[1]) == 1
    # an infinity: 1 / rms = 0, so the others are 0 and it is a NaN; a NaN takes its row
    assert row_values[4].float().isnan().all() and row_scales[4].isnan().all()
    g = W // 2 // 128
    assert scales[4, g].isnan() and (torch.cat([scales[4, :g], scales[4, g + 1:]]) == 1).all()
    assert row_values[5].float().isnan().all() and scales[5].isnan().all()
    out = vb.add_rmsnorm_fwd(x, None, eps=EPS)
    assert torch.isfinite(out[ok]).all() and out[5].isnan().all() and int(out[4].isnan().sum()) == 1


@pytest.mark.parametrize("W", [40, 100, 500, 1000, 2048, 16384, 40000])
def test_squares_outside_the_range(W):
    """Rows whose squares 32 bits do not hold, beside ordinary ones: too large, and (eps = 0) too small."""
    n = 9
    x, dy = rows_of(n, W, FP32, 1), rows_of(n, W, FP32, 2)
    gamma = 1.0 + 0.2 * rows_of(1, W, FP32, 3)[0]
    x[1] *= 1e19
    x[4] *= 1e30
    x[7] *= 1e-25
    r = 1.0 / torch.sqrt(x.double().square().mean(1, keepdim=True))
    xn = x.double() * r
    y = xn * gamma.double()
    out = vb.add_rmsnorm_fwd(x, gamma, eps=0.0)
    assert ((out.double() - y).abs() <= y_error(y, W)).all()
    check_e4m3(*vb.add_rmsnorm_fwd(x, gamma, eps=0.0, out_mode=vb.NORM_OUT_E4M3_ROW), y, W, W)
    check_e4m3(*vb.add_rmsnorm_fwd(x, gamma, eps=0.0, out_mode=vb.NORM_OUT_E4M3_GROUP), y, 128, W)
    dx, dw = vb.add_rmsnorm_bwd(x, gamma, dy, eps=0.0)
    g = dy.double() * gamma.double()
    want = r * (g - xn * (g * xn).mean(1, keepdim=True))
    size = r * (g.abs() + xn.abs() * (g * xn).abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= size * (1.5 * W + 16) * 2.0 ** -24).all()
    assert ((dw.double() - (dy.double() * xn).sum(0)).abs() <= (dy.double() * xn).abs().sum(0) * (n + W + 16) * 2.0 ** -24).all()


def test_tiny_scales_and_empty():
    x = torch.zeros(2, 128, device="cuda")
    x[0, 0] = 1e-44
    values, scales = vb.add_rmsnorm_fwd(x, torch.full((128,), 1e-3, device="cuda"), eps=1.0, out_mode=vb.NORM_OUT_E4M3_ROW)
    assert torch.isfinite(values.float()).all() and (scales > 0).all()
    assert vb.add_rmsnorm_fwd(x[:0], None).shape == (0, 128)
    dx, dw = vb.add_rmsnorm_bwd(x[:0], None, x[:0])
    assert dx.shape == (0, 128) and (dw == 0).all()


def test_both_ways_of_a_call_and_refusals():
    """Calls made in one step and those that go through the binding's own checks (a stream given) are the same calls."""
    x, res, dy = (rows_of(6, 300, BF16, i) for i in (1, 2, 3))
    gamma, here = 1.0 + 0.2 * rows_of(1, 300, FP32, 3)[0], torch.cuda.current_stream()
    for mode in (vb.NORM_OUT_TENSOR, vb.NORM_OUT_E4M3_ROW, vb.NORM_OUT_E4M3_GROUP):
        a, b = (vb.add_rmsnorm_fwd(x, gamma, residual=res, out_mode=mode, **kw) for kw in ({}, dict(stream=here)))
        for s, t in zip(*((r if isinstance(r, tuple) else (r,)) for r in (a, b))):
            assert s.dtype == t.dtype and torch.equal(s.float(), t.float())
    a, b = (vb.add_rmsnorm_bwd(x, gamma, dy, dh=res, **kw) for kw in ({}, dict(stream=here)))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    for f in (lambda: vb.add_rmsnorm_fwd(x, gamma[:-1]), lambda: vb.add_rmsnorm_fwd(x, gamma.bfloat16()),
              lambda: vb.add_rmsnorm_fwd(x, residual=res[:, 1:]), lambda: vb.add_rmsnorm_fwd(x, residual=res.float()),
              lambda: vb.add_rmsnorm_fwd(x[0]), lambda: vb.add_rmsnorm_fwd(x.half()), lambda: vb.add_rmsnorm_fwd(x.t()),
              lambda: vb.add_rmsnorm_fwd(x, out=torch.empty_like(x, dtype=FP32)),
              lambda: vb.add_rmsnorm_fwd(x, residual_out=x[:1].expand(6, 300)),
              lambda: vb.add_rmsnorm_fwd(x, out_mode=1, scales=torch.empty(6, device="cuda")),
              lambda: vb.add_rmsnorm_bwd(x, gamma, dy[:-1]), lambda: vb.add_rmsnorm_bwd(x, gamma, dy, dweight=gamma[1:])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: vb.add_rmsnorm_fwd(x, out_mode=3), lambda: vb.add_rmsnorm_bwd(x, gamma, dy, dx=dy)):
        with pytest.raises(vb.VdnError):
            f()


def test_streams_graphs_and_repeats():
    x, dy = rows_of(3000, 2048, BF16, 1), rows_of(3000, 2048, BF16, 2)
    gamma = 1.0 + 0.2 * rows_of(1, 2048, FP32, 3)[0]
    want = vb.add_rmsnorm_bwd(x, gamma, dy)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            got.append(vb.add_rmsnorm_bwd(x, gamma, dy, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = vb.add_rmsnorm_bwd(x, gamma, dy)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_block_of_a_streaming_model():
    """The operators as a layer uses them: residual norm, projection, linear memory (prompt, then one token), residual
    norm with 8-bit output; the prompt's last token through the single-token form gives the same."""
    B, N, H, d = 2, 37, 2, 64
    W = H * d
    x, res = rows_of(B * N, W, BF16, 1), rows_of(B * N, W, BF16, 2)
    gamma = 1.0 + 0.2 * rows_of(1, W, FP32, 3)[0]
    proj = rows_of(W, 3 * W, BF16, 4, W ** -0.5)
    ld = torch.tensor([-0.05, -0.3], device="cuda")

    def front(x, res):
        h = torch.empty_like(x)
        return h, vb.add_rmsnorm_fwd(x, gamma, residual=res, residual_out=h) @ proj

    h, qkv = front(x, res)
    q, k, v = qkv.view(B, N, 3, H, d).unbind(2)
    pool = torch.zeros(4, H, d, d, device="cuda")
    full = vb.linear_attn_fwd(q, k, v, ld)
    vb.linear_attn_fwd(q[:, :-1], k[:, :-1], v[:, :-1], ld, state_out=pool[1:3])
    last = vb.linear_attn_step(q[:, -1], k[:, -1], v[:, -1], ld, pool, slots=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    # two roundings to bf16 of one value (and, in the prompt's form, of the state or the score)
    assert (last.double() - full[:, -1].double()).norm() <= 2.0 ** -7 * full[:, -1].double().norm()
    a, sa = vb.add_rmsnorm_fwd(full.view(B * N, W), gamma, residual=h, out_mode=vb.NORM_OUT_E4M3_GROUP)
    y = reference(full.view(B * N, W), h, gamma)[2]
    check_e4m3(a, sa, y, 128, W)
