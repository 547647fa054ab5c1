"""Products of few rows on the average where an expert takes several passes over its weight, its K cut over a cluster, its
columns no whole number of blocks or fours, and rows of no expert at both ends: every pass crosses the cluster's barriers
behind work of single lanes.  Tolerances as in test_blocks.py.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_blocks import close8, operands, product64
from test_rows import BF, act64, close, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


@pytest.mark.parametrize("c,h", [(2048, 130), (2048, 77), (512, 257), (4096, 3), (144, 509)])
@pytest.mark.parametrize("rows,outside", [([130, 3, 0, 5, 1, 0, 0, 17], 4), ([1, 200, 0], 0), ([0, 0, 0, 0, 65, 0, 0], 21),
                                          ([40] * 3 + [0] * 30, 2)])
def test_several_passes(rows, outside, c, h):
    e, n = len(rows), sum(rows) + 2 * outside
    g = gen(n + c + h)
    q, s, wq, ws = operands(g, n, c, h, e)
    wu, us = sc.quantize_weight_blocks(normal(g, e, c, h, std=c ** -0.5).to(BF))
    off = outside + torch.tensor([0] + rows, device="cuda").cumsum(0).int()
    b, r = normal(g, e, h), normal(g, n, h).to(BF)
    z, slack = product64(q, s, wq, ws, off)
    zu, eu = product64(q, s, wu, us, off)
    inside = torch.zeros(n, 1, dtype=torch.bool, device="cuda")
    inside[outside:n - outside] = True
    of_row = torch.repeat_interleave(torch.arange(e, device="cuda"), torch.tensor(rows, device="cuda"))
    zb = z.clone()
    zb[outside:n - outside] += b[of_row].double()
    slack_b = slack + 2.0 ** -22 * (z.abs() + b.abs().max())
    a, _ = act64("silu", z)
    slack_g = (1.13 * slack + 2.0 ** -19 * a.abs()) * (zu.abs() + eu) + a.abs() * eu
    for _ in range(2):
        close(sc.linear_blocks(q, wq, s, ws, offsets=off, bias=b), torch.where(inside, zb, 0.0), slack_b, "y")
        y = sc.linear_blocks(q, wq, s, ws, offsets=off, bias=b, activation="relu", residual=r)
        close(y, torch.where(inside, zb.clamp_min(0) + r.double(), 0.0), slack_b, "residual")
        close(sc.gated_ffn_blocks(q, wq, wu, s, ws, us, offsets=off), a * zu, slack_g, "gated")
        h8 = sc.gated_ffn_blocks(q, wq, wu, s, ws, us, offsets=off, quantize=True)
        close8(h8, a * zu, slack_g, "gated q")
        assert not y[~inside[:, 0]].any() and not h8[0][~inside[:, 0]].view(torch.uint8).any()
    assert sc.rows_status() == 0
