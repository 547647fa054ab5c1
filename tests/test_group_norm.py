"""Group norm of ragged scans and its backward pass against plain 64-bit forms.

Tolerances, from the arithmetic: a bf16 output is one rounding of an fp32 value
(relative 2^-8).  In fp32 the mean and the deviation are sums of few terms per
thread, added up in a tree: about 16 roundings of 2^-24 relative to the values'
size (where the mean is within a few deviations of zero), so outputs are within
2^-19 of theirs in the 2-norm, sums of products over rows within 2^-18.
"""
import math

import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import ACTS, BF, act64, gen, normal, rel, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def borders(n, kind):
    """Offsets of ``n`` rows, or None."""
    if kind == "one":
        return None
    if kind == "ragged":      # scans of any length, some empty, all rows in one
        cuts = [0, 0, n // 7, n // 7, n // 3, n - n // 5, n, n]
    elif kind == "inside":    # rows before the first scan and behind the last
        cuts = [n // 9, n // 2, n - n // 8]
    elif kind == "none":      # no scan has a row
        cuts = [n // 2] * 3
    else:                     # a scan per row
        cuts = list(range(n + 1))
    return torch.tensor(cuts, dtype=torch.int32, device="cuda")


def runs(n, offsets):
    at = [0, n] if offsets is None else offsets.tolist()
    return list(zip(at, at[1:]))


def forward64(x, w, b, groups, offsets, act, eps):
    """y, statistics"""
    n, c = x.shape
    y = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    rr = runs(n, offsets)
    st = torch.zeros(len(rr), groups, 2, dtype=torch.float64, device="cuda")
    st[:, :, 1] = eps ** -0.5
    for i, (lo, hi) in enumerate(rr):
        if lo == hi:
            continue
        v = x[lo:hi].double().view(hi - lo, groups, -1)
        m = v.mean((0, 2), keepdim=True)
        r = 1 / torch.sqrt(((v - m) ** 2).mean((0, 2), keepdim=True) + eps)
        st[i] = torch.stack((m.flatten(), r.flatten()), 1)
        y[lo:hi] = act64(act, ((v - m) * r).view(hi - lo, c) * w.double() + (0 if b is None else b.double()))[0]
    return y, st


def check(got, ref, what, slack=2.0 ** -19):
    """One rounding of a bf16 output, and ``slack`` in the 2-norm and of each value's size and the outputs'."""
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    size = ref.norm() / max(1.0, math.sqrt(ref.numel()))
    bound = 1.01 * step * ref.abs() + 16 * slack * (ref.abs() + size) + 1e-37
    worst = ((got.double() - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"
    if got.numel():
        assert rel(got, ref) <= step + slack, f"{what}: {rel(got, ref):.3g}"


SIZES = [(1, 1, 1), (1, 64, 8), (2, 6, 3), (37, 35, 5), (300, 64, 8), (513, 128, 32), (1000, 96, 96), (777, 60, 12),
         (40, 1000, 8), (65, 2048, 32), (9, 8192, 64), (20, 8192, 1), (33, 4099, 1), (5000, 130, 10), (20011, 128, 32)]


def inputs(n, c, dtype, seed):
    g = gen(seed)
    x = normal(g, n, c) * torch.exp(normal(g, c, std=0.5)) + normal(g, c)
    return x.to(dtype), 1 + normal(g, c, std=0.3), normal(g, c, std=0.3), (normal(g, n, c, std=1e-2)).to(dtype)


@pytest.mark.parametrize("n,c,groups", SIZES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kind", ["one", "ragged", "inside", "none"])
def test_forward(n, c, groups, dtype, kind):
    x, w, b, _ = inputs(n, c, dtype, n + 13 * c)
    off = borders(n, kind)
    act = ACTS[(n + c) % 5]
    y, st = sc.group_norm(x, w, b, groups, offsets=off, activation=act, stats=True)
    ref, st64 = forward64(x, w, b, groups, off, act, 1e-5)
    # a single value has no deviation: r is 1 / sqrt(eps) and u what the mean's rounding leaves
    check(y, ref, "y")
    check(st, st64, "stats")
    assert torch.equal(sc.group_norm(x, w, b, groups, offsets=off, activation=act), y)
    assert sc.rows_status() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,c,groups,scans", [(700, 48, 6, 700), (3000, 24, 3, 3000), (5000, 64, 64, 40)])
def test_many_scans_without_bias(n, c, groups, scans, act):
    x, w, _, _ = inputs(n, c, torch.float32, n)
    off = borders(n, "rows") if scans == n else (torch.arange(scans + 1, device="cuda") * (n // scans)).int()
    y = sc.group_norm(x, w, None, groups, offsets=off, activation=act)
    check(y, forward64(x, w, None, groups, off, act, 1e-5)[0], "y")


def test_strided_and_unaligned():
    for dtype in (BF, torch.float32):
        for n, c, extra in ((300, 64, 8), (300, 64, 4), (200, 60, 3), (129, 33, 1)):
            x, w, b, dy = inputs(n, c, dtype, 5 * n + c)
            off = borders(n, "ragged")
            want, st = sc.group_norm(x, w, b, 3 if c % 3 == 0 else 1 if c % 4 else 4, offsets=off, stats=True, activation="gelu")
            groups = st.shape[1]
            got = sc.group_norm(strided(x, extra), w, b, groups, offsets=off, activation="gelu")
            assert rel(got, want.double()) <= (2.0 ** -8 if dtype == BF else 2.0 ** -19)
            dx, dw, db = sc.group_norm_backward(dy, x, w, b, groups, st, offsets=off, activation="gelu")
            dx2, dw2, db2 = sc.group_norm_backward(strided(dy, extra), strided(x, extra), w, b, groups, st, offsets=off,
                                                   activation="gelu")
            assert rel(dx2, dx.double()) <= (2.0 ** -8 if dtype == BF else 2.0 ** -18)
            assert rel(dw2, dw.double()) <= 2.0 ** -18 and rel(db2, db.double()) <= 2.0 ** -18


def test_far_mean_and_constant():
    """A mean a thousand deviations from zero costs the digits that the inputs have, no more; without any
    deviation the output is act(bias)."""
    g = gen(3)
    x = 1000 + normal(g, 4000, 32)
    w, b = 1 + normal(g, 32, std=0.1), normal(g, 32, std=0.1)
    ref, _ = forward64(x, w, b, 4, None, "none", 1e-5)
    y = sc.group_norm(x, w, b, 4)
    # the mean is held in fp32: off by 2^-24 of 1000, and as much again for its sum
    assert (y.double() - ref).abs().max() <= 4 * 1000 * 2.0 ** -24 * w.abs().max()
    first = x.clone()
    first[0] = 1e4   # a first row far from the rest
    ref, _ = forward64(first, w, b, 4, None, "none", 1e-5)
    assert rel(sc.group_norm(first, w, b, 4), ref) <= 2.0 ** -16
    for value in (0.0, 7.25):
        y = sc.group_norm(torch.full((500, 32), value, device="cuda"), w, b, 4, activation="silu")
        check(y, act64("silu", b.double())[0].expand(500, 32), "constant")


def test_not_finite():
    """NaN and infinities stay within their scan's group."""
    x, w, b, _ = inputs(100, 16, torch.float32, 1)
    off = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    want = sc.group_norm(x, w, b, 4, offsets=off)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[50, 5] = bad
        got = sc.group_norm(y, w, b, 4, offsets=off)
        assert torch.isnan(got[40:, 4:8]).all()
        assert torch.equal(got[:40], want[:40]) and torch.equal(got[40:, :4], want[40:, :4]) and torch.equal(got[40:, 8:], want[40:, 8:])


def backward64(dy, x, w, b, groups, st, offsets, act):
    n, c = x.shape
    dx = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros(c, dtype=torch.float64, device="cuda"), torch.zeros(c, dtype=torch.float64, device="cuda")
    for i, (lo, hi) in enumerate(runs(n, offsets)):
        if lo == hi:
            continue
        m, r = st[i].double().unbind(1)
        u = (x[lo:hi].double().view(hi - lo, groups, -1) - m[None, :, None]) * r[None, :, None]
        flat = u.view(hi - lo, c)
        dz = dy[lo:hi].double() * act64(act, flat * w.double() + (0 if b is None else b.double()))[1]
        dw += (dz * flat).sum(0)
        db += dz.sum(0)
        p = (dz * w.double()).view_as(u)
        d = p - p.mean((0, 2), keepdim=True) - u * (p * u).mean((0, 2), keepdim=True)
        dx[lo:hi] = (r[None, :, None] * d).view(hi - lo, c)
    return dx, dw, db


@pytest.mark.parametrize("n,c,groups", [s for s in SIZES if s[0] > 1])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kind", ["one", "ragged", "inside", "none"])
def test_backward(n, c, groups, dtype, kind):
    x, w, b, dy = inputs(n, c, dtype, 3 * n + c)
    off = borders(n, kind)
    act = ["none", "silu", "gelu", "gelu_tanh"][(n + c) % 4]
    _, st = sc.group_norm(x, w, b, groups, offsets=off, activation=act, stats=True)
    dx, dw, db = sc.group_norm_backward(dy, x, w, b, groups, st, offsets=off, activation=act)
    rx, rw, rb = backward64(dy, x, w, b, groups, st, off, act)
    # few values share a mean: dx is what is left of terms that nearly cancel, each of them off by
    # 2^-19 of r |dy w|, which the bound takes as its size
    r = st[:, :, 1].max().double()
    size = (dy.double().norm() * (w.abs().max().double()) * r) if kind != "none" else 1.0
    step = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    assert (dx.double() - rx).norm() <= step * rx.norm() + 2.0 ** -19 * size
    for got, ref, terms in ((dw, rw, "w"), (db, rb, "b")):
        assert (got.double() - ref).norm() <= 2.0 ** -18 * max(ref.norm().item(), dy.double().norm().item()), terms
    none = sc.group_norm_backward(dy, x, w, None, groups, st, offsets=off, activation="none")
    assert none[2] is None and torch.isfinite(none[0]).all()
    assert sc.rows_status() == 0


def test_gradient_against_differences():
    """The directional derivative of sum(y t) along v, by central differences in 64 bits."""
    x, w, b, t = inputs(50, 24, torch.float32, 11)
    off = torch.tensor([0, 13, 50], dtype=torch.int32, device="cuda")
    _, st = sc.group_norm(x, w, b, 4, offsets=off, activation="silu", stats=True)
    dx, dw, db = sc.group_norm_backward(t, x, w, b, 4, st, offsets=off, activation="silu")
    g = gen(12)

    def value(x_, w_, b_):
        return (forward64(x_, w_, b_, 4, off, "silu", 1e-5)[0] * t.double()).sum().item()

    for which, grad in ((0, dx), (1, dw), (2, db)):
        args = [x.double(), w.double(), b.double()]
        v = torch.randn(args[which].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        lo, hi = list(args), list(args)
        lo[which], hi[which] = args[which] - h * v, args[which] + h * v
        slope = (value(*hi) - value(*lo)) / (2 * h)
        # the gradient's sums to 2^-18 of their terms, the differences to h^2 and 2^-52 / h of the values
        size = (grad.double().abs() * v.abs()).sum().item()
        assert abs((grad.double() * v).sum().item() - slope) <= 2.0 ** -16 * size + 1e-8


def test_no_rows():
    w, b = torch.ones(16, device="cuda"), torch.zeros(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, st = sc.group_norm(x, w, b, 4, offsets=off, stats=True)
    assert y.shape == (0, 16) and (st[:, :, 0] == 0).all() and torch.allclose(st[:, :, 1], torch.full((3, 4), 1e-5 ** -0.5, device="cuda"))
    dx, dw, db = sc.group_norm_backward(x, x, w, b, 4, st, offsets=off)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def test_borders_out_of_order_or_range():
    """They are reported, and nothing outside the outputs is written."""
    x, w, b, dy = inputs(1000, 64, BF, 2)
    st = torch.zeros(3, 8, 2, device="cuda")
    for cuts in ([0, 700, 300, 1000], [-5, 10, 20, 1000], [0, 10, 20, 1001], [1000, 500, 200, 0]):
        off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        sc.group_norm(x, w, b, 8, offsets=off, stats=True)
        assert sc.status_string(sc.rows_status()) == "coordinate out of range"
        sc.group_norm_backward(dy, x, w, b, 8, st, offsets=off)
        assert sc.status_string(sc.rows_status()) == "coordinate out of range"
    assert sc.rows_status() == 0


def test_refusals():
    x, w, b, _ = inputs(10, 12, BF, 1)
    st = torch.zeros(1, 3, 2, device="cuda")
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for kw in (dict(groups=5), dict(groups=0), dict(weight=None), dict(weight=w[:11]), dict(weight=w.double()),
               dict(x=x.half()), dict(x=x.cpu()), dict(x=x[0]), dict(offsets=off.long()), dict(offsets=off[:1]),
               dict(offsets=off.cpu()), dict(activation="tanh"), dict(bias=b[:3])):
        a = dict(x=x, weight=w, bias=b, groups=3) | kw
        with pytest.raises(ValueError):
            sc.group_norm(a.pop("x"), a.pop("weight"), a.pop("bias"), a.pop("groups"), **a)
    for kw in (dict(stats=st[:, :2]), dict(stats=st.double()), dict(dy=x[:9]), dict(dy=x.float())):
        a = dict(dy=x, x=x, weight=w, bias=b, groups=3, stats=st) | kw
        with pytest.raises(ValueError):
            sc.group_norm_backward(*a.values())
    with pytest.raises(sc.SpconvError):
        sc.group_norm(x, w, b, 3, eps=-1.0)
    with pytest.raises(sc.SpconvError):
        sc.group_norm(torch.zeros(2, 8200, device="cuda"), torch.ones(8200, device="cuda"), None, 2)
