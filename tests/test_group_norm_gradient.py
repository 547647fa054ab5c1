"""Group norm's gradients value by value, and the forward pass at widths that the piece kernels take one value at a time.

The gradient that arrives has a mean and a part along u, so the two means that dx subtracts are as large as dx itself, and
each scan is held to its own 1 / sqrt(var + eps): a missing or wrong mean is far outside of the bound.

Bound, from the arithmetic.  u and z = u w + b are two and three roundings (2^-23 u, 2^-22 (|u w| + |b|)); a slope is off by
its own error (2^-20: exponentials and reciprocals of 2^-22, the error function's 1.5e-7) and by at most 0.8 times z's (the
largest second derivative of the four); p = dy act'(z) w, then, is off by e_p = |dy w| (2^-20 + 2^-22 (|u w| + |b|)) +
2^-23 |p|.  A mean of M values is off by the mean of their errors and K 2^-24 of the mean of their magnitudes, with K the
additions that a value goes through: the rows of a thread, the threads of a column, the channels of a group and the blocks,
K = rows / 152 + 100 at most.  dx = r (p - a - u c) adds what p, a and u c are off by and four roundings of each.  The
column sums are off by the terms' errors and K 2^-24 of their magnitudes.  A bf16 result is one rounding more.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_group_norm import borders, check, forward64, inputs, runs
from test_rows import ACTS, BF, act64, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def grads64(dy, x, w, b, groups, st, offsets, act):
    """dx, dw, db in 64 bits from the statistics, and the bounds on what fp32 sums of them are off by."""
    n, c = x.shape
    dx = torch.zeros(n, c, dtype=torch.float64, device="cuda")
    off = torch.zeros_like(dx)
    dw, db, ew, eb = (torch.zeros(c, dtype=torch.float64, device="cuda") for _ in range(4))
    k = (n / 152 + 100) * 2.0 ** -24
    w64, b64 = w.double(), 0.0 if b is None else b.double()
    for i, (lo, hi) in enumerate(runs(n, offsets)):
        if lo == hi:
            continue
        m, r = (v[None, :, None] for v in st[i].double().unbind(1))
        u = (x[lo:hi].double().view(hi - lo, groups, -1) - m) * r
        flat = u.view(hi - lo, c)
        z = flat * w64 + b64
        d = dy[lo:hi].double()
        dz = d * act64(act, z)[1]
        e_z = d.abs() * (2.0 ** -20 + 2.0 ** -22 * ((flat * w64).abs() + abs(b64))) + 2.0 ** -23 * dz.abs()
        dw += (dz * flat).sum(0)
        db += dz.sum(0)
        ew += (e_z * flat.abs() + (2.0 ** -22 + k) * (dz * flat).abs()).sum(0)
        eb += (e_z + k * dz.abs()).sum(0)
        p, e_p = (dz * w64).view_as(u), (e_z * w64.abs() + 2.0 ** -23 * (dz * w64).abs()).view_as(u)

        def mean(v):
            return v.mean((0, 2), keepdim=True)

        a, along = mean(p), mean(p * u)
        e_a = mean(e_p) + k * mean(p.abs())
        e_along = mean(e_p * u.abs()) + (k + 2.0 ** -22) * mean((p * u).abs())
        dx[lo:hi] = (r * (p - a - u * along)).view(hi - lo, c)
        off[lo:hi] = (r * (e_p + e_a + u.abs() * e_along + 2.0 ** -22 * (p.abs() + a.abs() + (u * along).abs()))).view(hi - lo, c)
    return (dx, dw, db), (off, ew, eb)


def within(got, ref, off, what):
    step = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    bound = step * (ref.abs() + off) + 1.01 * off + 1e-37
    worst = ((got.double() - ref).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"


SIZES = [(2, 6, 3), (37, 35, 5), (300, 64, 8), (513, 128, 32), (1000, 96, 96), (40, 1000, 8), (65, 2048, 32), (9, 8192, 64),
         (33, 4099, 1), (5000, 130, 10), (20011, 128, 32), (180001, 32, 8)]


def case(n, c, groups, dtype, off, act, seed):
    x, w, b, _ = inputs(n, c, dtype, seed)
    _, st = sc.group_norm(x, w, b, groups, offsets=off, activation=act, stats=True)
    g = gen(seed + 1)
    dy = 0.5 + normal(g, n, c, std=0.5)
    for i, (lo, hi) in enumerate(runs(n, off)):
        if hi > lo:
            m, r = (v[None, :, None] for v in st[i].unbind(1))
            u = ((x[lo:hi].float().view(hi - lo, groups, -1) - m) * r).view(hi - lo, c)
            dy[lo:hi] += 0.5 * u
            # ReLU's slope jumps at 0: no gradient arrives where z is within its error of it
            z = u * w + b
            dy[lo:hi] = torch.where(z.abs() <= 2.0 ** -18 * ((u * w).abs() + b.abs()), 0.0, dy[lo:hi])
    return dy.to(dtype), x, w, b, st


@pytest.mark.parametrize("n,c,groups", SIZES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("kind", ["one", "ragged", "inside"])
def test_values(n, c, groups, dtype, kind):
    off = borders(n, kind)
    for act in ACTS if n * c < 100000 else ["relu", "silu"]:
        dy, x, w, b, st = case(n, c, groups, dtype, off, act, 7 * n + c)
        ref, tol = grads64(dy, x, w, b, groups, st, off, act)
        got = sc.group_norm_backward(dy, x, w, b, groups, st, offsets=off, activation=act)
        for name, v, r, e in zip(("dx", "dw", "db"), got, ref, tol):
            within(v, r, e, f"{name} {act}")
    assert sc.rows_status() == 0


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("n,c,groups", [(700, 48, 6), (6000, 24, 3)])
def test_relu_of_a_scan_per_row(n, c, groups, dtype):
    off = borders(n, "rows")
    dy, x, w, b, st = case(n, c, groups, dtype, off, "relu", n)
    ref, tol = grads64(dy, x, w, b, groups, st, off, "relu")
    for name, v, r, e in zip(("dx", "dw", "db"), sc.group_norm_backward(dy, x, w, b, groups, st, offsets=off, activation="relu"), ref, tol):
        within(v, r, e, name)


def test_the_means_matter():
    """The bound notices either mean being left out (planted in the 64-bit form)."""
    n, c, groups = 180001, 32, 8
    dy, x, w, b, st = case(n, c, groups, torch.float32, None, "none", 3)
    (dx, _, _), (off, _, _) = grads64(dy, x, w, b, groups, st, None, "none")
    m, r = (v[None, :, None] for v in st[0].double().unbind(1))
    u = (x.double().view(n, groups, -1) - m) * r
    p = (dy.double() * w.double()).view_as(u)
    for wrong in (r * (p - u * (p * u).mean((0, 2), keepdim=True)), r * (p - p.mean((0, 2), keepdim=True))):
        assert ((wrong.view(n, c) - dx).abs() > 100 * (2.0 ** -8 * dx.abs() + off)).float().mean() > 0.5


# more than 512 kB a scan: pieces, one and several scans, of one, two and four values at a time
@pytest.mark.parametrize("n,c,groups,scans", [(6000, 131, 1, 1), (40000, 131, 131, 7), (9001, 66, 11, 1), (30011, 90, 3, 5), (500, 4099, 1, 1),
                                              (3000, 4099, 4099, 4), (400, 8191, 1, 1), (5003, 132, 12, 1), (60000, 36, 4, 3)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_forward_of_odd_widths_in_pieces(n, c, groups, scans, dtype):
    assert n * c * 2 > scans * (512 << 10)
    x, w, b, _ = inputs(n, c, dtype, n + c)
    off = None if scans == 1 else torch.tensor([n * i // scans + (i % 3 if 0 < i < scans else 0) for i in range(scans + 1)], device="cuda").int()
    for act in ("relu", "gelu"):
        y, st = sc.group_norm(x, w, b, groups, offsets=off, activation=act, stats=True)
        ref, st64 = forward64(x, w, b, groups, off, act, 1e-5)
        check(y, ref, "y")
        check(st, st64, "stats")
        assert torch.equal(sc.group_norm(x, w, b, groups, offsets=off, activation=act), y)
    assert sc.rows_status() == 0
