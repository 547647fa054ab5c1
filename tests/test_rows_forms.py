"""Forms and ranges of the row-wise operators beside those of test_rows.py, against 64-bit formulas.

Tolerances are those derived there: one rounding per output (bf16 2^-8, fp32
2^-24), and (terms / 32 + 64) 2^-23 of the sum of magnitudes for fp32 sums.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod
from test_rows import BF, close, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


# widths of every kernel of the norm's gradient: lanes (whole vectors, pairs, odd), ring, block, two passes
GRAD_WIDTHS = [(300, 64), (300, 1000), (90, 502), (90, 255), (200, 2048), (60, 1001), (40, 3001), (9, 9000), (5, 20001)]


@pytest.mark.parametrize("n,c", GRAD_WIDTHS)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("size,eps", [(1e-14, 0.0), (1e13, 1e-6), (1e15, 1e-6)])
def test_norm_backward_of_rows_far_from_unit_size(n, c, dtype, size, eps):
    """r = 1 / rms is in range for such rows, its cube is not (from 1e38 on, and below 1e-38)."""
    g = gen(n + c)
    u = normal(g, n, c)
    x = (size * u).to(dtype)
    dy = (normal(g, n, c) + 0.5 * u).to(dtype)   # (along x in part, so that the projection counts)
    w = 1 + normal(g, c, std=0.3)
    dx, dw = sc.rms_norm_backward(dy, x, w, eps=eps)
    X, D = x.double(), dy.double()
    r = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + eps)
    G, unit = D * w.double(), X * r
    along = unit * (G * unit).mean(1, keepdim=True)
    acc = (c / 32 + 64) * 2.0 ** -23
    ref = r * (G - along)
    slack = acc * (r * (G.abs() + unit.abs() * (G * unit).abs().mean(1, keepdim=True)) + ref.abs())
    close(dx, ref, slack, "dx", 2.0 ** -8 if dtype == BF else 2.0 ** -24)
    terms = D * unit
    assert ((dw.double() - terms.sum(0)).abs() <= (acc + (n / 152 + 40) * 2.0 ** -23) * terms.abs().sum(0)).all()


def test_a_wait_that_runs_out_reaches_the_status():
    """The operators' bounded wait on a barrier that nothing arrives on, with a 50 ms limit: it gives up, the
    status says so once, and the operators go on working."""
    lib, stream = sc.library(), torch.cuda.current_stream().cuda_stream
    assert sc.rows_status() == 0
    for limit in (0, 999_999, 100_000_001, -5):
        assert lib.spconv_selftest_rows_wait(limit, stream) == -1
    assert sc.rows_status() == 0
    assert lib.spconv_selftest_rows_wait(50_000_000, stream) == 0
    assert sc.rows_status() == -8
    assert sc.rows_status() == 0
    side = torch.cuda.Stream()
    assert lib.spconv_selftest_rows_wait(50_000_000, side.cuda_stream) == 0
    assert sc.rows_status(stream=side) == -8 and sc.rows_status(stream=side) == 0
    x = torch.ones(3, 64, device="cuda")
    assert torch.allclose(sc.rms_norm(x, x[0], eps=0.0), x)
    assert sc.rows_status() == 0


@pytest.mark.parametrize("n,c,h", [(1, 2048, 2048), (3000, 512, 256), (300, 501, 77), (200, 2048, 136), (20, 5001, 64)])
def test_captured_after_the_same_call(n, c, h):
    """Every operator at sizes that reach few-row, wide, cut and copying kernels: made once, then captured."""
    g = gen(n + c + h)
    x, dy = normal(g, n, c).to(BF), normal(g, n, h).to(BF)
    w, u = normal(g, c, h, std=c ** -0.5).to(BF), normal(g, c, h, std=c ** -0.5).to(BF)
    wn, b = 1 + normal(g, c, std=0.1), normal(g, h)

    def calls():
        q, scale = sc.quantize_weight(w)
        x8, xs = sc.rms_norm(x, wn, quantize=True)
        return [sc.rms_norm(x, wn), scale, xs, sc.linear(x, w, bias=b, activation="gelu"),
                sc.linear(x8, q, x_scale=xs, w_scale=scale), sc.gated_ffn(x, w, u),
                sc.gated_ffn(x8, q, q, x_scale=xs, gate_scale=scale, up_scale=scale),
                *sc.linear_backward(dy, x, w, bias=b, activation="silu"), *sc.gated_ffn_backward(dy, x, w, u),
                *sc.rms_norm_backward(x, x, wn)]
    first = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, first))
