"""The residual RMSNorm where 32 bits do not hold a row's squares: the choice to look again (csrc/norm_range.h, compiled
for the host) and, on the GPU, rows of such values in blocks that are not full."""
import itertools
import os
import subprocess

import numpy as np
import pytest
import torch

from video_diffusion_hybrid_sparse_b200 import binding as vb

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "video_diffusion_hybrid_sparse_b200", "csrc")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    """Reads lines `real eps s0 s1 s2 s3` and prints the choice of a block of four rows of two warps each (s_r: a warp's
    sum; the other's is 0), then the row's own factors."""
    at = tmp_path_factory.mktemp("range")
    src, exe = at / "range.cpp", at / "range"
    src.write_text('#include <cstdio>\n#include "norm_range.h"\nint main() {\n  int real; float eps, s[8] = {};\n'
                   '  while (scanf("%d %f %f %f %f %f", &real, &eps, s, s + 2, s + 4, s + 6) == 6)\n'
                   '    printf("%d %a\\n", (int)vdn::norm_look_again<4, 2>(s, real, eps), vdn::norm_rescue(s[0], eps));\n}\n')
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(cases):
        text = "\n".join(" ".join(repr(float(x)) if i else str(x) for i, x in enumerate(c)) for c in cases)
        lines = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        return [(bool(int(a)), float.fromhex(b)) for a, b in (line.split() for line in lines)]

    return ask


def test_missing_rows_do_not_enter_the_choice(host):
    """All threads of a block pass the barriers of a second look or none does: the choice is that of the real rows, and
    rows behind the last one, whose sums are 0, change nothing, whatever eps."""
    values = (0.0, 1e-30, 1.0, float("inf"), float("nan"))
    cases = [(real, eps, *(s if r < real else 0.0 for r, s in enumerate(sums)))
             for real in (1, 2, 3, 4) for eps in (0.0, 1e-30, 1e-6) for sums in itertools.product(values, repeat=4)]
    got = host(cases)
    own = {(eps, repr(s)): f != 1.0 for (_, f), (eps, s) in
           zip(host([(4, e, s, 1, 1, 1) for e in (0.0, 1e-30, 1e-6) for s in values]), itertools.product((0.0, 1e-30, 1e-6), values))}
    for (again, _), (real, eps, *sums) in zip(got, cases):
        assert again == any(own[eps, repr(s)] for s in sums[:real]), (real, eps, sums)


@pytest.mark.parametrize("W", [1, 2, 64, 2048, 16384, 32768, 40000, 1 << 20])
def test_factors_bring_every_row_into_range(host, W):
    """Rows of W equal elements from the smallest number to the largest, and of one such element among zeros: the squares'
    sum, of the row times its factor, is a normal number."""
    a = np.concatenate([np.float32(2.0) ** np.arange(-149, 128, dtype=np.float32), [np.finfo(np.float32).max]]).astype(np.float32)
    with np.errstate(over="ignore", under="ignore"):
        for n in (W, 1):
            sums = a * a * np.float32(n)
            f = np.array([x for _, x in host([(1, 0.0, s, 1, 1, 1) for s in sums])], dtype=np.float32)
            scaled = a * f
            again = scaled * scaled * np.float32(n)
            assert np.isfinite(again).all() and (again >= np.finfo(np.float32).tiny).all(), a[~np.isfinite(again)]


def normed(x, gamma, dy):
    """y, dx, dgamma with eps = 0, and the magnitudes of the last two, in 64 bits."""
    X, G, DY = x.double(), gamma.double(), dy.double()
    r = 1.0 / torch.sqrt(X.square().mean(1, keepdim=True))
    xn, g = X * r, DY * G
    c = (g * xn).mean(1, keepdim=True)
    size = r * (g.abs() + xn.abs() * (g * xn).abs().mean(1, keepdim=True))
    return xn * G, r * (g - xn * c), size, (DY * xn).sum(0), (DY * xn).abs().sum(0)


def check_rows(x, gamma, dy):
    """Forward (three forms) and backward of x with eps = 0: a row's mean of W squares costs W / 2 roundings of 2^-24 of its
    root, products a few more, the result one of its type; an e4m3 value is its element rounded (2^-4, or half of the
    smallest step) under a scale of max / 448."""
    n, W = x.shape
    half, err = HALF[x.dtype], (W / 2 + 12) * 2.0 ** -24
    y, dx, size, dw, dw_size = normed(x, gamma, dy)
    for _ in range(2):
        out = vb.add_rmsnorm_fwd(x, gamma, eps=0.0)
        assert ((out.double() - y).abs() <= y.abs() * (err + half * 1.001)).all()
        for mode, group in ((vb.NORM_OUT_E4M3_ROW, W), (vb.NORM_OUT_E4M3_GROUP, 128)):
            values, scales = vb.add_rmsnorm_fwd(x, gamma, eps=0.0, out_mode=mode)
            s = scales.double().repeat_interleave(group, 1)[:, :W]
            most = torch.nn.functional.pad(y, (0, -W % group)).reshape(n, -1, group).abs().amax(2)
            assert ((scales.double() - most / 448).abs() <= most / 448 * err).all()
            assert ((values.float().double() - y / s).abs() <= (y / s).abs() * (2.0 ** -4 + 3 * err) + 2.0 ** -10).all()
        got, got_w = vb.add_rmsnorm_bwd(x, gamma, dy, eps=0.0)
        assert ((got.double() - dx).abs() <= size * (1.5 * W + 16) * 2.0 ** -24 + dx.abs() * half * 1.001).all()
        assert ((got_w.double() - dw).abs() <= dw_size * (n + W + 16) * 2.0 ** -24).all()


def rows_of(n, W, dtype, seed):
    return torch.randn(n, W, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + W)).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("W", [48, 100, 400, 520, 600, 1000, 1024, 1100, 2000, 2048, 4000])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 1201])
def test_blocks_that_are_not_full(n, W, dtype):
    """eps = 0, a number of rows that no block divides, with and without a row that is looked at again."""
    x, dy, gamma = rows_of(n, W, dtype, 1), rows_of(n, W, dtype, 2), 1.0 + 0.2 * rows_of(1, W, torch.float32, 3)[0]
    check_rows(x, gamma, dy)
    x[n // 2] *= 1e-25
    x[-1] *= 1e20
    check_rows(x, gamma, dy)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("W", [1, 2, 48, 100, 500, 520, 1000, 2048, 4096, 16384, 32768, 40000])
def test_rows_at_the_ends_of_the_range(W, dtype):
    """Rows whose elements are near the type's largest number or among its smallest (denormal ones forward only, where
    1 / rms has no fp32)."""
    x, dy = rows_of(7, W, dtype, 1), rows_of(7, W, dtype, 2)
    gamma = 1.0 + 0.2 * rows_of(1, W, torch.float32, 3)[0]
    sign = torch.where(x > 0, 1.0, -1.0)
    some = 0.5 + 0.5 * x.float().abs().clamp(max=1.0)
    for i, size in ((0, 3.3e38), (2, 1e38), (3, 1e37), (5, 2e-37)):
        x[i] = (sign[i] * some[i] * size).to(dtype)
    err, half = (W / 2 + 12) * 2.0 ** -24, HALF[dtype]
    y, dx, size, dw, dw_size = normed(x, gamma, dy)
    out = vb.add_rmsnorm_fwd(x, gamma, eps=0.0)
    assert ((out.double() - y).abs() <= y.abs() * (err + half * 1.001)).all()
    got, got_w = vb.add_rmsnorm_bwd(x, gamma, dy, eps=0.0)
    # dx of the largest rows, and their 1 / rms, are denormal: half a step of 2^-149 (of the type) each
    steps = 2.0 ** -150 * (1 + size * x.double().square().mean(1, keepdim=True).sqrt()) + (2.0 ** -134 if half else 0)
    assert ((got.double() - dx).abs() <= size * (1.5 * W + 16) * 2.0 ** -24 + dx.abs() * half * 1.001 + steps).all()
    assert ((got_w.double() - dw).abs() <= dw_size * (7 + W + 16) * 2.0 ** -24).all()
    x[1], x[6] = (sign[1] * some[1] * 1e-39).to(dtype), 2.0 ** -133  # bf16's smallest number
    y = normed(x, gamma, dy)[0]
    out = vb.add_rmsnorm_fwd(x, gamma, eps=0.0)
    assert ((out.double() - y).abs() <= y.abs() * (err + half * 1.001)).all()
    for mode, group in ((vb.NORM_OUT_E4M3_ROW, W), (vb.NORM_OUT_E4M3_GROUP, 128)):
        values, scales = vb.add_rmsnorm_fwd(x, gamma, eps=0.0, out_mode=mode)
        s = scales.double().repeat_interleave(group, 1)[:, :W]
        assert ((values.float().double() - y / s).abs() <= (y / s).abs() * (2.0 ** -4 + 3 * err) + 2.0 ** -10).all()
