"""Products of e4m3 operands with block scales, for one weight and for the experts of sorted rows, against 64 bits.

Tolerances, from the arithmetic: each block of 128 is one fp32 sum of exact products (16 at a time: at most 8 + 8
roundings of 2^-24 of the sum of their magnitudes, and the tensor core's own alignment, 2^-23 of it a step), the
blocks are added one multiply-add each, so z is off by at most (kb + 48) 2^-23 of the sum of magnitudes.  A bf16
output is one rounding more (2^-8); an e4m3 one is within half a step (2^-4 of the value, or half of the smallest
step, 2^-10, of its block's scale).
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import ACTS, BF, E4M3, act64, close, gen, normal, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def rows64(q, scale):
    return q.double() * scale.double().t().repeat_interleave(128, 1)[:, :q.shape[1]]


def weight64(q, scale):
    s = scale.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
    return q.double() * s[..., :q.shape[-2], :q.shape[-1]]


def operands(g, n, c, h, experts=None):
    x = normal(g, n, c) * torch.exp(normal(g, n, 1))
    q, s = sc.quantize_blocks(x.to(BF))
    w = (normal(g, *([experts] if experts else []), c, h, std=c ** -0.5)).to(BF)
    wq, ws = sc.quantize_weight_blocks(w)
    return q, s, wq, ws


def runs_of(n, offsets, experts):
    at = offsets.tolist() if offsets is not None else [0, n]
    return [(e, lo, hi) for e, (lo, hi) in enumerate(zip(at, at[1:])) if hi > lo]


def product64(q, s, wq, ws, offsets=None):
    """(z, bound on its error) of rows and the weights of their runs."""
    n = q.shape[0]
    w3, s3 = (wq, ws) if wq.dim() == 3 else (wq[None], ws[None])
    z = torch.zeros(n, w3.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(z)
    x = rows64(q, s)
    for e, lo, hi in runs_of(n, offsets, w3.shape[0]):
        w = weight64(w3[e], s3[e]).t()
        z[lo:hi] = x[lo:hi] @ w
        mag[lo:hi] = x[lo:hi].abs() @ w.abs()
    return z, (q.shape[1] / 128 + 49) * 2.0 ** -23 * mag


def close8(got, ref, slack, what=""):
    """e4m3 values and scales of ``ref`` known within ``slack``."""
    q, scale = got
    n, c = q.shape
    nb = -(-c // 128)
    pad = torch.zeros(n, nb * 128, dtype=torch.float64, device="cuda")
    pad[:, :c] = ref.abs()
    most = pad.view(n, nb, 128).amax(2)
    pad[:, :c] = slack
    tol = pad.view(n, nb, 128).amax(2)
    assert ((scale.t().double() - most / 448).abs() <= tol / 448 + 2.0 ** -23 * most / 448 + 1e-44).all(), what + " scale"
    v = rows64(q, scale)
    step = (scale.t().double().repeat_interleave(128, 1)[:, :c])
    # half a step of the value, half of the smallest step, and what the sum and the scale are off
    bound = 2.0 ** -4 * ref.abs() * 1.01 + 2.0 ** -10 * step + slack * 1.1 + 2.0 ** -20 * ref.abs() + 1e-44
    bad = (v - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} off"


SIZES = [(1, 16, 1), (1, 128, 128), (1, 4096, 4096), (2, 144, 130), (7, 2048, 96), (16, 512, 257), (17, 640, 384), (33, 1024, 1000),
         (64, 8192, 256), (65, 256, 128), (100, 16, 300), (129, 400, 255), (256, 128, 256), (257, 1040, 511), (300, 4096, 512),
         (700, 272, 77), (1024, 2048, 1024), (2500, 512, 640), (5000, 128, 136)]


@pytest.mark.parametrize("n,c,h", SIZES)
@pytest.mark.parametrize("bias,residual,extra", [(False, False, 0), (True, True, 0), (True, False, 3), (False, True, 8)])
def test_linear(n, c, h, bias, residual, extra):
    g = gen(n + c + h)
    q, s, wq, ws = operands(g, n, c, h)
    act = ACTS[(n + h) % 5]
    b = normal(g, h) if bias else None
    r = normal(g, n, h).to(BF) if residual else None
    z, slack = product64(q, s, wq, ws)
    z = z + (b.double() if bias else 0)
    ref = act64(act, z)[0] + (r.double() if residual else 0)
    # the activations' slopes are at most 1.13, their own error 2^-20 of the value and 1.5e-7 of z (erf)
    slack = 1.13 * slack + 2.0 ** -19 * ref.abs() + 2e-7 * z.abs() + (2.0 ** -23 * b.double().abs() if bias else 0)
    out = strided(torch.zeros(n, h, device="cuda", dtype=BF), extra) if extra else None
    y = sc.linear_blocks(strided(q.float(), extra).to(E4M3) if extra == 8 else q, wq, s, ws, bias=b, activation=act,
                         residual=None if r is None else strided(r, extra), out=out)
    assert out is None or y.data_ptr() == out.data_ptr()
    close(y, ref, slack, "y")
    if residual:
        same = r.clone()
        assert torch.equal(sc.linear_blocks(q, wq, s, ws, bias=b, activation=act, residual=same, out=same), y) and torch.equal(same, y)
    else:
        close8(sc.linear_blocks(q, wq, s, ws, bias=b, activation=act, quantize=True), ref, slack, "q")
    assert sc.rows_status() == 0


@pytest.mark.parametrize("n,c,h", SIZES)
def test_gated(n, c, h):
    g = gen(2 * n + c + h)
    q, s, wg, gs = operands(g, n, c, h)
    wu, us = sc.quantize_weight_blocks(normal(g, c, h, std=c ** -0.5).to(BF))
    act = ACTS[1:][(n + h) % 4]
    zg, eg = product64(q, s, wg, gs)
    zu, eu = product64(q, s, wu, us)
    a = act64(act, zg)[0]
    ref = a * zu
    slack = (1.13 * eg + 2.0 ** -19 * a.abs() + 2e-7 * zg.abs()) * (zu.abs() + eu) + a.abs() * eu
    close(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, activation=act), ref, slack, "h")
    close8(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, activation=act, quantize=True), ref, slack, "q")
    assert sc.rows_status() == 0


def split(n, e, g, kind):
    """Offsets of n rows over e experts."""
    if kind == "all":
        cuts = torch.randint(0, n + 1, (e - 1,), generator=g, device="cuda").sort()[0]
        ends = [0, n]
    elif kind == "some":     # rows of no expert at both ends, empty experts
        cuts = torch.randint(n // 5, n - n // 5 + 1, (e - 1,), generator=g, device="cuda").sort()[0]
        ends = [n // 5, n - n // 5]
    elif kind == "one":      # the last expert has everything
        cuts = torch.zeros(e - 1, dtype=torch.int64, device="cuda")
        ends = [0, n]
    else:                    # nobody has anything
        cuts = torch.full((e - 1,), n // 2, device="cuda")
        ends = [n // 2, n // 2]
    t = torch.tensor(ends, device="cuda")
    return torch.cat((t[:1], cuts, t[1:])).int()


EXPERTS = [(5, 1, 256, 128), (16, 8, 256, 130), (64, 4, 512, 384), (100, 128, 144, 96), (300, 3, 400, 200), (1000, 7, 256, 300),
           (2000, 16, 128, 256), (3000, 5, 640, 520), (1500, 300, 64, 40), (40, 600, 32, 17)]


@pytest.mark.parametrize("n,e,c,h", EXPERTS)
@pytest.mark.parametrize("kind", ["all", "some", "one", "none"])
def test_experts(n, e, c, h, kind):
    g = gen(n + e)
    q, s, wq, ws = operands(g, n, c, h, e)
    off = split(n, e, g, kind)
    b = normal(g, e, h)
    z, slack = product64(q, s, wq, ws, off)
    inside = torch.zeros(n, 1, dtype=torch.bool, device="cuda")
    for i, lo, hi in runs_of(n, off, e):
        z[lo:hi] += b[i].double()
        inside[lo:hi] = True
    y = sc.linear_blocks(q, wq, s, ws, offsets=off, bias=b)
    close(y, torch.where(inside, z, 0.0), slack + 2.0 ** -23 * z.abs(), "y")
    assert not y[~inside[:, 0]].any()
    r = normal(g, n, h).to(BF)
    close(sc.linear_blocks(q, wq, s, ws, offsets=off, bias=b, residual=r), torch.where(inside, z + r.double(), 0.0),
          slack + 2.0 ** -22 * z.abs(), "with residual")
    wu, us = sc.quantize_weight_blocks(normal(g, e, c, h, std=c ** -0.5).to(BF))
    zg, eg = product64(q, s, wq, ws, off)
    zu, eu = product64(q, s, wu, us, off)
    a = act64("silu", zg)[0]
    slack = (1.13 * eg + 2.0 ** -19 * a.abs()) * (zu.abs() + eu) + a.abs() * eu
    close(sc.gated_ffn_blocks(q, wq, wu, s, ws, us, offsets=off), a * zu, slack, "gated")
    h8 = sc.gated_ffn_blocks(q, wq, wu, s, ws, us, offsets=off, quantize=True)
    close8(h8, a * zu, slack, "gated q")
    assert not h8[0][~inside[:, 0]].view(torch.uint8).any() and not h8[1][:, ~inside[:, 0]].any()
    assert sc.rows_status() == 0


def test_neighbours_do_not_matter():
    """NaN rows and weights of other experts, and scales of other rows, leave a run as it is."""
    g = gen(5)
    n, e, c, h = 600, 3, 256, 200
    q, s, wq, ws = operands(g, n, c, h, e)
    for cuts in ([0, 150, 300, 600], [0, 10, 20, 600]):
        off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        lo, hi = cuts[1], cuts[2]
        want = sc.linear_blocks(q, wq, s, ws, offsets=off)[lo:hi]
        q2, s2, wq2, ws2 = q.clone(), s.clone(), wq.clone(), ws.clone()
        q2.view(torch.uint8)[:lo] = 0x7F
        q2.view(torch.uint8)[hi:] = 0x7F
        s2[:, :lo] = s2[:, hi:] = float("nan")
        wq2.view(torch.uint8)[0] = 0x7F
        wq2.view(torch.uint8)[2] = 0x7F
        ws2[0] = ws2[2] = float("inf")
        assert torch.equal(sc.linear_blocks(q2, wq2, s2, ws2, offsets=off)[lo:hi], want)


def test_not_finite():
    g = gen(6)
    for n in (3, 300):
        q, s, wq, ws = operands(g, n, 256, 136)
        s[1, 2] = float("inf")
        y = sc.linear_blocks(q, wq, s, ws)
        assert not torch.isfinite(y[2]).any() and torch.isfinite(y[:2]).all() and torch.isfinite(y[3:]).all()
        v, scale = sc.linear_blocks(q, wq, s, ws, quantize=True)
        back = v.float() * scale.t().repeat_interleave(128, 1)[:, :136]
        assert torch.isnan(back[2]).all() and torch.isfinite(back[:2]).all()


def test_borders_out_of_order_or_range():
    """They are reported, and nothing outside the outputs is read or written."""
    g = gen(7)
    for n in (40, 900):
        q, s, wq, ws = operands(g, n, 128, 64, 3)
        for cuts in ([0, n - 3, 7, n], [-5, 3, 20, n], [0, 10, 20, n + 1], [n, 20, 10, 0], [0, 2 ** 31 - 1, -2 ** 31, n]):
            off = torch.tensor(cuts, device="cuda").int()
            sc.linear_blocks(q, wq, s, ws, offsets=off)
            assert sc.status_string(sc.rows_status()) == "coordinate out of range"
            sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off, quantize=True)
            assert sc.status_string(sc.rows_status()) == "coordinate out of range"
    assert sc.rows_status() == 0


def test_no_rows():
    g = gen(8)
    _, _, wq, ws = operands(g, 1, 128, 64, 2)
    q, s = sc.quantize_blocks(torch.empty(0, 128, device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert sc.linear_blocks(q, wq, s, ws, offsets=off).shape == (0, 64)
    assert [v.shape for v in sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off, quantize=True)] == [(0, 64), (1, 0)]


def test_refusals():
    g = gen(9)
    q, s, wq, ws = operands(g, 4, 128, 64)
    w3, s3 = wq[None].expand(2, 64, 128).contiguous(), ws[None].expand(2, 1, 1).contiguous()
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    bf = torch.zeros(4, 64, device="cuda", dtype=BF)
    bad = [lambda: sc.linear_blocks(q.float(), wq, s, ws), lambda: sc.linear_blocks(q, wq.float(), s, ws),
           lambda: sc.linear_blocks(q, wq, s.t(), ws), lambda: sc.linear_blocks(q, wq, s, ws[0]),
           lambda: sc.linear_blocks(q, wq[:, :64], s, ws), lambda: sc.linear_blocks(q, w3, s, s3),
           lambda: sc.linear_blocks(q, wq, s, ws, offsets=off), lambda: sc.linear_blocks(q, w3, s, s3, offsets=off.long()),
           lambda: sc.linear_blocks(q, w3, s, s3, offsets=off[:2]), lambda: sc.linear_blocks(q, wq, s, ws, bias=bf[0]),
           lambda: sc.linear_blocks(q, w3, s, s3, offsets=off, bias=torch.zeros(64, device="cuda")),
           lambda: sc.linear_blocks(q, wq, s, ws, residual=bf, quantize=True), lambda: sc.linear_blocks(q, wq, s, ws, out=bf, quantize=True),
           lambda: sc.linear_blocks(q, wq, s, ws, out=bf[:3]), lambda: sc.linear_blocks(q, wq, s, ws, activation="x"),
           lambda: sc.linear_blocks(q.cpu(), wq, s, ws), lambda: sc.linear_blocks(q, wq, s.cpu(), ws),
           lambda: sc.gated_ffn_blocks(q, wq, w3, s, ws, s3), lambda: sc.gated_ffn_blocks(q, wq, wq, s, ws, s3[0, :0])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    odd, so = sc.quantize_blocks(torch.zeros(4, 24, device="cuda"))
    wo, wso = sc.quantize_weight_blocks(torch.zeros(24, 16, device="cuda", dtype=BF))
    with pytest.raises(sc.SpconvError):
        sc.linear_blocks(odd, wo, so, wso)
