"""Sizes at which the group norm and the block products take another way than in their own tests: more tiles than there
are pairs of CTAs, experts with more rows than a pass over their weights takes, inputs beyond the small ones.

Tolerances as in test_blocks.py and test_group_norm.py.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_blocks import close8, operands, product64
from test_group_norm import backward64, check, forward64, inputs
from test_rows import BF, act64, close, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


@pytest.mark.parametrize("n,c,h", [(30000, 128, 1000), (30011, 256, 768), (12000, 400, 2048)])
def test_many_tiles(n, c, h):
    """Several tiles a pair of CTAs, of one to four blocks: what a tile's bias and scales lie in is used again."""
    g = gen(n + c)
    q, s, wq, ws = operands(g, n, c, h)
    b, r = normal(g, h), normal(g, n, h).to(BF)
    z, slack = product64(q, s, wq, ws)
    # the bias is the first term of the sum: a rounding of it and z more a block
    slack2 = slack + (c / 128 + 2) * 2.0 ** -23 * (z.abs() + b.abs().double())
    close(sc.linear_blocks(q, wq, s, ws, bias=b), z + b.double(), slack2, "y")
    a = act64("relu", z + b.double())[0]
    close(sc.linear_blocks(q, wq, s, ws, bias=b, activation="relu", residual=r), a + r.double(),
          slack2 + 2.0 ** -23 * (a + r.abs().double()), "residual")
    close8(sc.linear_blocks(q, wq, s, ws, bias=b, activation="relu", quantize=True), a, slack2, "q")
    out = r.clone()
    assert torch.equal(sc.linear_blocks(q, wq, s, ws, bias=b, activation="relu", residual=out, out=out),
                       sc.linear_blocks(q, wq, s, ws, bias=b, activation="relu", residual=r))
    h8 = sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, activation="relu", quantize=True)
    up = act64("relu", z)[0] * z
    close8(h8, up, 2.1 * slack * z.abs() + slack ** 2 + 2.0 ** -22 * up.abs(), "gated")
    assert sc.rows_status() == 0


@pytest.mark.parametrize("rows,c,h", [([96, 32] * 16, 1408, 2048), ([700] + [20] * 39, 640, 1024), ([130, 0, 60, 2] * 4, 2048, 384),
                                      ([33, 31, 40, 24] * 12, 528, 1408)])
def test_uneven_experts(rows, c, h):
    """Few rows an expert on the average, but some experts take several passes."""
    e, n = len(rows), sum(rows)
    g = gen(n + c)
    q, s, wq, ws = operands(g, n, c, h, e)
    off = torch.tensor([0] + rows, device="cuda").cumsum(0).int()
    z, slack = product64(q, s, wq, ws, off)
    for _ in range(3):
        y = sc.linear_blocks(q, wq, s, ws, offsets=off)
    close(y, z, slack, "y")
    a = act64("silu", z)[0]
    ref, tol = a * z, (1.13 * slack + 2.0 ** -19 * a.abs()) * (z.abs() + slack) + a.abs() * slack
    close(sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off), ref, tol, "gated")
    close8(sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off, quantize=True), ref, tol, "gated q")
    assert sc.rows_status() == 0


@pytest.mark.parametrize("n,c,groups,cuts", [(180001, 128, 32, [0, 5, 5, 100000, 180001]), (90000, 250, 10, [0, 90000]),
                                             (60000, 128, 4, [i * 375 for i in range(161)]),
                                             (4100, 512, 64, [0, 300, 4000, 4100])])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_large_norm(n, c, groups, cuts, dtype):
    x, w, b, dy = inputs(n, c, dtype, n + c)
    off = torch.tensor(cuts, device="cuda").int()
    y, st = sc.group_norm(x, w, b, groups, offsets=off, activation="silu", stats=True)
    ref, st64 = forward64(x, w, b, groups, off, "silu", 1e-5)
    check(y, ref, "y")
    check(st, st64, "stats")
    dx, dw, db = sc.group_norm_backward(dy, x, w, b, groups, st, offsets=off, activation="silu")
    rx, rw, rb = backward64(dy, x, w, b, groups, st, off, "silu")
    size = dy.double().norm() * w.abs().max().double() * st[:, :, 1].max().double()
    assert (dx.double() - rx).norm() <= (2.0 ** -8 if dtype == BF else 2.0 ** -24) * rx.norm() + 2.0 ** -19 * size
    for got, want in ((dw, rw), (db, rb)):
        assert (got.double() - want).norm() <= 2.0 ** -18 * max(want.norm().item(), dy.double().norm().item())
    assert sc.rows_status() == 0
