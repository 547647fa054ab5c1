"""Forms and ranges of the row-wise operators beside those of test_rows.py, against 64-bit formulas.

Tolerances are those derived there: one rounding per output (bf16 2^-8, fp32
2^-24), and (terms / 32 + 64) 2^-23 of the sum of magnitudes for fp32 sums.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod
from submanifold_sparse_convolution_gb300 import synthetic
from test_rows import BF, act64, close, gen, grad_check, make, normal, sum_error

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


# ---- the C entries' forms that the Python ones do not take -----------------------------
def stream():
    return torch.cuda.current_stream().cuda_stream


def address(t):
    return None if t is None else t.data_ptr()


PARTS = [(5, 64, 72), (300, 64, 72), (129, 33, 50), (2000, 512, 520), (200, 2048, 136)]


@pytest.mark.parametrize("n,c,h", PARTS)
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("wants", ["x", "w", "b", "xw", "xb", "wb", "xwb"])
def test_linear_backward_of_some_outputs(n, c, h, act, wants):
    g = gen(n + c + h)
    x, (w,), _, _, X, (W,) = make(g, n, c, h, False)
    dy, b = normal(g, n, h).to(BF), normal(g, h)
    nan = float("nan")
    dx = torch.full((n, c), nan, device="cuda", dtype=BF) if "x" in wants else None
    dw = torch.full((c, h), nan, device="cuda", dtype=BF) if "w" in wants else None
    db = torch.full((h,), nan, device="cuda") if "b" in wants else None
    assert sc.library().spconv_linear_backward(dy.data_ptr(), h, x.data_ptr(), c, w.data_ptr(), n, c, h, 0, b.data_ptr(),
                                               sc.ACTIVATIONS[act], address(dx), address(dw), address(db), stream()) == 0
    z = X @ W + b.double()
    dz = dy.double() * act64(act, z)[1]
    err = dy.double().abs() * (1.1 * sum_error(X, W) + 2.0 ** -20)   # (of z, second derivatives below 1.1)
    dz_abs = dz.abs() + 2.0 ** 8 * err
    if dx is not None:
        grad_check(dx, dz @ W.t(), dz_abs @ W.abs().t(), "dx")
    if dw is not None:
        grad_check(dw, X.t() @ dz, X.abs().t() @ dz_abs, "dw")
    if db is not None:
        bound = err + dz.abs() * (n / 128 + 64) * 2.0 ** -23
        assert ((db.double() - dz.sum(0)).abs() <= bound.sum(0) + 1e-30).all()


@pytest.mark.parametrize("n,c,h", PARTS)
@pytest.mark.parametrize("wants", ["x", "w"])
def test_gated_backward_of_some_outputs(n, c, h, wants):
    g = gen(n + 5 * c + h)
    x, (wg, wu), _, _, X, (G, U) = make(g, n, c, h, False, 2)
    dh = normal(g, n, h).to(BF)
    nan = float("nan")
    dx = torch.full((n, c), nan, device="cuda", dtype=BF) if wants == "x" else None
    dwg, dwu = (torch.full((c, h), nan, device="cuda", dtype=BF) if wants == "w" else None for _ in range(2))
    assert sc.library().spconv_gated_ffn_backward(dh.data_ptr(), h, x.data_ptr(), c, wg.data_ptr(), wu.data_ptr(), n, c, h, 0,
                                                  sc.ACTIVATIONS["silu"], address(dx), address(dwg), address(dwu),
                                                  stream()) == 0
    zg, zu, D = X @ G, X @ U, dh.double()
    a, slope = act64("silu", zg)
    dg, du = D * zu * slope, D * a
    eg, eu = 1.2 * sum_error(X, G) + 2.0 ** -20, sum_error(X, U) + 2.0 ** -20
    dg_abs = dg.abs() + 2.0 ** 8 * D.abs() * (eg * (zu.abs() + eu) + 1.2 * eu)
    du_abs = du.abs() + 2.0 ** 8 * D.abs() * eg
    if dx is not None:
        grad_check(dx, dg @ G.t() + du @ U.t(), dg_abs @ G.abs().t() + du_abs @ U.abs().t(), "dx")
    else:
        grad_check(dwg, X.t() @ dg, X.abs().t() @ dg_abs, "dw_gate")
        grad_check(dwu, X.t() @ du, X.abs().t() @ du_abs, "dw_up")


@pytest.mark.parametrize("n,c", [*GRAD_WIDTHS, (1, 64), (1700, 128)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_norm_backward_onto_the_incoming_gradient(n, c, dtype):
    """dx may be dres: the same bits as into memory of its own."""
    g = gen(n + 7 * c)
    x, dy, dres = (normal(g, n, c).to(dtype) for _ in range(3))
    w = 1 + normal(g, c, std=0.3)
    dx, dw = sc.rms_norm_backward(dy, x, w, dres)
    own = torch.full((c,), float("nan"), device="cuda")
    assert sc.library().spconv_rms_norm_backward(dy.data_ptr(), c, x.data_ptr(), c, w.data_ptr(), dres.data_ptr(), c, n, c,
                                                 0 if dtype == BF else 1, 1e-6, dres.data_ptr(), own.data_ptr(), stream()) == 0
    assert torch.equal(dres, dx) and torch.equal(own, dw)


def test_scratch_is_given_back():
    """The pool keeps a gated gradient's scratch (4 n c_hidden bytes) until it is trimmed; a map in it stays."""
    wl = synthetic.random_cloud(31, 3000, shape=(16, 16, 16), c_in=64, c_out=64)
    m = sc.build_map(wl.coords.cuda(), wl.spatial_shape, wl.batch_size)
    feats, weights = wl.feats.cuda(), wl.weights[0].cuda()
    ref = sc.subm_forward(m, feats, weights)
    g = gen(32)
    n, c, h = 16384, 64, 4096
    x, dh = normal(g, n, c).to(BF), normal(g, n, h).to(BF)
    wg, wu = normal(g, c, h).to(BF), normal(g, c, h).to(BF)
    first = sc.gated_ffn_backward(dh, x, wg, wu)
    torch.cuda.synchronize()
    held = torch.cuda.mem_get_info()[0]
    sc.trim_pool()
    assert torch.cuda.mem_get_info()[0] - held >= 4 * n * h
    assert all(torch.equal(a, b) for a, b in zip(sc.gated_ffn_backward(dh, x, wg, wu), first))
    assert torch.equal(sc.subm_forward(m, feats, weights), ref) and sc.map_status(m) == 0
    m.destroy()
    sc.trim_pool(1 << 40)                     # keeps all
    with pytest.raises(sc.SpconvError):
        sc.trim_pool(-1)
