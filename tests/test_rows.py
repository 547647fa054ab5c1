"""The row-wise operators (RMS norm, linear, gated feed-forward) against plain 64-bit forms.

Tolerances, from the arithmetic: a bf16 output is one rounding of an fp32
value (relative 2^-8); an fp32 sum of K products taken 16 at a time is off by
at most (K / 16 + 16) 2^-23 of the sum of their magnitudes; a gradient that
goes through a bf16 operand carries 2^-8 of each of its terms as well.
"""
import math

import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def strided(t, extra):
    """The same rows inside a wider buffer, the rest NaN."""
    if not extra:
        return t.contiguous()
    b = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device).to(t.dtype)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def act64(name, z):
    """(act, act') in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def sum_error(a, b):
    """Bound on the error of the fp32 product a @ b (64-bit operands)."""
    k = a.shape[1]
    return (k / 16 + 16) * 2.0 ** -23 * (a.abs() @ b.abs())


def close(got, ref, slack, what="", ulp=2.0 ** -8):
    """|got - ref| <= one rounding (ulp) of the larger of the two, and slack."""
    got = got.double()
    assert got.shape == ref.shape, what
    bound = ulp * 1.01 * (ref.abs() + slack) + slack + 1e-37
    bad = (got - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / bound).max():.3g} of the bound"


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-300)).item()


# ---- RMS norm -------------------------------------------------------------------
NORM_SIZES = [(1, 1), (3, 7), (1, 2048), (5, 16), (33, 64), (129, 128), (77, 136), (40, 256), (9, 1000), (7, 1001),
              (300, 2048), (31, 4096), (3, 4100), (5, 8192), (2, 16384), (3, 16385), (2, 20000), (1, 65536), (2, 40001)]


def norm64(h, w, eps):
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("n,c", NORM_SIZES)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(n, c, dtype, residual):
    g = gen(n * 131 + c)
    x, r = normal(g, n, c).to(dtype), (3 * normal(g, n, c)).to(dtype)
    w = 1 + normal(g, c, std=0.3)
    h = x.double() + (r.double() if residual else 0)
    ref = norm64(h, w.double(), 1e-6)
    out = sc.rms_norm(x, w, r if residual else None)
    y = out[0] if residual else out
    # fp32: the sum of squares (relative c / 32 additions at most), the root and two products
    slack = (c / 32 + 64) * 2.0 ** -24 * ref.abs()
    close(y, ref, slack, "y", 2.0 ** -8 if dtype == BF else 2.0 ** -24)
    if residual:
        close(out[1], h, 2.0 ** -24 * h.abs(), "sum", 2.0 ** -8 if dtype == BF else 2.0 ** -24)
    res8 = sc.rms_norm(x, w, r if residual else None, quantize=True)
    q, scale = res8[0], res8[1]
    assert q.dtype == E4M3 and scale.shape == (n,)
    s64 = ref.abs().amax(1) / 448
    assert ((scale.double() - s64).abs() <= (c / 32 + 64) * 2.0 ** -24 * s64).all()
    # e4m3 keeps 4 significant bits (2^-4 of the value at most), steps of 2^-9 below 2^-6
    back = q.double() * scale.double()[:, None]
    bound = (2.0 ** -4 * ref.abs()).maximum(2.0 ** -10 * s64[:, None]) * (1 + 1e-3)
    assert ((back - ref).abs() <= bound).all()
    assert (q.float().abs().amax(1) == 448).all()
    if residual:
        assert torch.equal(res8[2], out[1])


def test_norm_strides_and_in_place():
    g = gen(5)
    x, r = normal(g, 50, 96).to(BF), normal(g, 50, 96).to(BF)
    w = normal(g, 96)
    y, h = sc.rms_norm(x, w, r)
    for extra in (1, 8, 13):                   # odd strides leave rows unaligned
        y2, h2 = sc.rms_norm(strided(x, extra), w, strided(r, extra))
        assert torch.equal(h2, h)
        assert rel(y2, y.double()) < 2.0 ** -8
    base = torch.empty(50 * 96 + 3, dtype=BF, device="cuda")[3:].view(50, 96)   # an odd address
    base.copy_(x)
    y3, h3 = sc.rms_norm(base, w, r)
    assert torch.equal(h3, h)
    r2 = r.clone()
    y4, h4 = sc.rms_norm(x, w, r2, sum_out=r2)  # the residual stream updated in place
    assert h4 is r2 and torch.equal(r2, h) and torch.equal(y4, y)
    wide_x, wide_r = normal(g, 3, 20000).to(BF), normal(g, 3, 20000).to(BF)
    ww = normal(g, 20000)
    a = sc.rms_norm(wide_x, ww, wide_r, quantize=True)
    b = sc.rms_norm(wide_x, ww, wide_r, quantize=True, sum_out=wide_r)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_norm_special_rows():
    x = torch.zeros(6, 40, device="cuda")
    x[1] = 1.0
    x[2, 3] = float("inf")
    x[3, 5] = float("nan")
    x[4] = 1e-30
    x[5] = 3e4
    w = torch.full((40,), 0.5, device="cuda")
    for dtype in (BF, torch.float32):
        y = sc.rms_norm(x.to(dtype), w, eps=0.0).float().cpu()
        assert torch.isnan(y[0]).all()                     # 0 / 0: eps = 0 leaves nothing to divide by
        assert torch.allclose(y[1], torch.full((40,), 0.5), atol=1e-6)
        assert torch.isnan(y[2, 3]) and (y[2, :3] == 0).all()
        assert torch.isnan(y[3]).all()
        y = sc.rms_norm(x.to(dtype), w, eps=1e-6).float().cpu()
        assert (y[0] == 0).all()
        q, scale = sc.rms_norm(x.to(dtype), w, eps=1e-6, quantize=True)
        q, scale = q.float().cpu(), scale.cpu()
        assert scale[0] == 0 and (q[0] == 0).all()          # a row of zeros
        assert torch.isnan(scale[3]) and torch.isnan(q[3]).all()
        assert torch.isnan(scale[2])                         # inf * 0
        assert (q[1] == 448).all() and (q[4] == 448).all() and (q[5] == 448).all()
    # a weight of zeros and a denormal one
    q, scale = sc.rms_norm(x[1:2], torch.zeros(40, device="cuda"), quantize=True)
    assert scale.item() == 0 and (q.float() == 0).all()
    q, scale = sc.rms_norm(x[1:2], torch.full((40,), 1e-37, device="cuda"), quantize=True)
    assert (q.float() == 448).all()


@pytest.mark.parametrize("n,c", NORM_SIZES + [(2000, 72), (3001, 1000), (1100, 2049), (700, 3001), (300, 4095), (400, 2502), (300, 4094)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("with_dres", [False, True])
def test_norm_backward(n, c, dtype, with_dres):
    g = gen(n * 17 + c)
    x = (2 * normal(g, n, c)).to(dtype)
    dy, dres = normal(g, n, c).to(dtype), normal(g, n, c).to(dtype)
    w = 1 + normal(g, c, std=0.3)
    dx, dw = sc.rms_norm_backward(dy, x, w, dres if with_dres else None, eps=1e-5)
    X, D, W = x.double(), dy.double(), w.double()
    r = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-5)
    G = D * W
    along = X * r ** 3 * (G * X).mean(1, keepdim=True)
    ref = r * G - along + (dres.double() if with_dres else 0)
    acc = (c / 32 + 64) * 2.0 ** -23
    slack = acc * ((r * G).abs() + X.abs() * r ** 3 * (G * X).abs().mean(1, keepdim=True) + ref.abs())
    close(dx, ref, slack, "dx", 2.0 ** -8 if dtype == BF else 2.0 ** -24)
    terms = D * X * r
    assert ((dw.double() - terms.sum(0)).abs() <= (acc + (n / 152 + 40) * 2.0 ** -23) * terms.abs().sum(0) + 1e-30).all()


def test_norm_backward_differences():
    """dx and dw against central differences of the 64-bit forward along random directions."""
    g = gen(8)
    x, dy, dres = normal(g, 37, 200), normal(g, 37, 200), normal(g, 37, 200)
    w = 1 + normal(g, 200, std=0.3)
    dx, dw = sc.rms_norm_backward(dy, x, w, dres, eps=1e-5)

    def loss(X, W):
        return (dy.double() * norm64(X, W, 1e-5)).sum() + (dres.double() * X).sum()
    for k in range(4):
        d, e, t = normal(g, 37, 200).double(), normal(g, 200).double(), 1e-4
        X, W = x.double(), w.double()
        num = (loss(X + t * d, W + t * e) - loss(X - t * d, W - t * e)) / (2 * t)
        ana = (dx.double() * d).sum() + (dw.double() * e).sum()
        assert abs(num - ana) <= 1e-6 * (dx.double().norm() * d.norm() + dw.double().norm() * e.norm())


# ---- linear and gated feed-forward ---------------------------------------------
# rows x c_in x c_out: one token to long ones, odd channel counts, edges of 16, 64, 128 and 256
SIZES = [(1, 64, 64), (1, 1, 1), (1, 4096, 4096), (2, 16, 16), (7, 2048, 600), (16, 128, 512), (33, 24, 40), (63, 200, 136),
         (64, 64, 256), (65, 72, 264), (100, 17, 33), (127, 129, 65), (128, 128, 128), (129, 512, 96), (200, 1000, 1001),
         (256, 256, 256), (257, 320, 520), (65, 3000, 24), (130, 4096, 256), (300, 2048, 100), (1000, 1536, 36), (500, 33, 8), (1000, 8, 700), (1025, 640, 384), (3000, 128, 512), (4111, 520, 72)]


def make(g, n, c, h, eight, k=1):
    x = normal(g, n, c)
    ws = [normal(g, c, h, std=c ** -0.5) for _ in range(k)]
    if not eight:
        x, ws = x.to(BF), [w.to(BF) for w in ws]
        return x, ws, None, [None] * k, x.double(), [w.double() for w in ws]
    xs = x.abs().amax(1) / 448
    xq = (x / xs.clamp_min(1e-30)[:, None]).to(E4M3)
    qs = [sc.quantize_weight(w.to(BF)) for w in ws]
    return (xq, [q for q, _ in qs], xs, [s for _, s in qs], xq.double() * xs.double()[:, None],
            [(q.double() * s.double()[:, None]).t() for q, s in qs])


@pytest.mark.parametrize("n,c,h", SIZES)
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, True)])
def test_linear(n, c, h, eight, act, bias, residual):
    g = gen(n + 3 * c + 7 * h)
    x, (w,), xs, (ws,), X, (W,) = make(g, n, c, h, eight)
    b = normal(g, h) if bias else None
    r = normal(g, n, h).to(BF) if residual else None
    y = sc.linear(x, w, bias=b, activation=act, residual=r, x_scale=xs, w_scale=ws)
    z = X @ W + (b.double() if bias else 0)
    ref = act64(act, z)[0] + (r.double() if residual else 0)
    slack = 1.2 * sum_error(X, W) + 2.0 ** -21 * (z.abs() + ref.abs() + (b.double().abs() if bias else 0)) + 1e-7
    close(y, ref, slack, "y")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,c,h", [(5, 64, 72), (300, 96, 130), (700, 256, 512)])
def test_activations(act, n, c, h):
    g = gen(h)
    x, (w,), _, _, X, (W,) = make(g, n, c, h, False)
    x = (x.float() * 8).to(BF)                 # far into both tails
    X = x.double()
    z = X @ W
    y = sc.linear(x, w, activation=act)
    close(y, act64(act, z)[0], 1.2 * sum_error(X, W) + 2.0 ** -21 * z.abs() + 1e-7, act)
    u = sc.gated_ffn(x, w, w, activation=act)
    a = act64(act, z)[0]
    e = sum_error(X, W)
    close(u, a * z, (1.2 * e + 2.0 ** -21 * z.abs() + 1e-7) * (z.abs() + e) + a.abs() * e, "gated " + act)


@pytest.mark.parametrize("n,c,h", SIZES)
@pytest.mark.parametrize("eight", [False, True])
def test_gated(n, c, h, eight):
    g = gen(11 * n + c + h)
    x, (wg, wu), xs, (gs, us), X, (G, U) = make(g, n, c, h, eight, 2)
    out = sc.gated_ffn(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us)
    zg, zu = X @ G, X @ U
    a = act64("silu", zg)[0]
    eg, eu = 1.2 * sum_error(X, G) + 2.0 ** -21 * zg.abs() + 1e-7, sum_error(X, U) + 2.0 ** -22 * zu.abs()
    close(out, a * zu, eg * (zu.abs() + eu) + a.abs() * eu, "h")


GRAD_SIZES = [(1, 16, 16), (1, 1, 1), (3, 40, 24), (64, 128, 64), (100, 17, 33), (129, 72, 264), (257, 320, 136), (1000, 8, 700),
              (1500, 513, 130), (4111, 128, 512), (9001, 64, 64), (20000, 40, 16), (200, 2048, 136), (300, 1500, 91),
              (40, 4096, 260)]


def grad_check(got, ref, terms, what):
    """A product whose one operand was rounded to bf16 (2^-8 of each term), rounded itself."""
    close(got, ref, 2.0 ** -8 * 1.05 * terms + 1e-30, what)
    if ref.numel() > 64:
        # independent roundings: sqrt(2) of one's rms error (2^-8 / sqrt 3 of the value at most)
        assert rel(got, ref) < 2.0 ** -8 * math.sqrt(2 / 3) * 1.3, what


@pytest.mark.parametrize("n,c,h", GRAD_SIZES)
@pytest.mark.parametrize("act,bias", [("none", True), ("silu", True), ("gelu", False), ("gelu_tanh", True)])
def test_linear_backward(n, c, h, act, bias):
    g = gen(n + c + h)
    x, (w,), _, _, X, (W,) = make(g, n, c, h, False)
    dy = normal(g, n, h).to(BF)
    b = normal(g, h) if bias else None
    dx, dw, db = sc.linear_backward(dy, x, w, bias=b, activation=act)
    z = X @ W + (b.double() if bias else 0)
    dz = dy.double() * act64(act, z)[1]
    # second derivatives are below 1.1: the error of z, carried through
    dz_abs = dz.abs() + 2.0 ** 8 * dy.double().abs() * (1.1 * sum_error(X, W) + 2.0 ** -20)
    grad_check(dx, dz @ W.t(), dz_abs @ W.abs().t(), "dx")
    grad_check(dw, X.t() @ dz, X.abs().t() @ dz_abs, "dw")
    assert (db is not None) == bias
    if bias:
        err = dy.double().abs() * (1.1 * sum_error(X, W) + 2.0 ** -20) + dz.abs() * (n / 128 + 64) * 2.0 ** -23
        assert ((db.double() - dz.sum(0)).abs() <= err.sum(0) + 1e-30).all()


def test_linear_backward_relu_mask():
    """z exact in fp32 (small whole numbers): the ReLU's gradient is 0 where z <= 0, whole numbers elsewhere."""
    g = gen(3)
    x = torch.randint(-3, 4, (300, 40), generator=g, device="cuda").to(BF)
    w = torch.randint(-3, 4, (40, 56), generator=g, device="cuda").to(BF)
    dy = torch.randint(-3, 4, (300, 56), generator=g, device="cuda").to(BF)
    dx, dw, db = sc.linear_backward(dy, x, w, bias=torch.zeros(56, device="cuda"), activation="relu")
    dz = dy.double() * (x.double() @ w.double() > 0)
    assert torch.equal(db.double(), dz.sum(0))
    assert torch.equal(dx, (dz @ w.double().t()).to(BF))
    assert torch.equal(dw, (x.double().t() @ dz).to(BF))


@pytest.mark.parametrize("n,c,h", GRAD_SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "none"])
def test_gated_backward(n, c, h, act):
    g = gen(n + 5 * c + h)
    x, (wg, wu), _, _, X, (G, U) = make(g, n, c, h, False, 2)
    dh = normal(g, n, h).to(BF)
    dx, dwg, dwu = sc.gated_ffn_backward(dh, x, wg, wu, activation=act)
    zg, zu, D = X @ G, X @ U, dh.double()
    a, slope = act64(act, zg)
    dg, du = D * zu * slope, D * a
    eg, eu = 1.2 * sum_error(X, G) + 2.0 ** -20, sum_error(X, U) + 2.0 ** -20
    dg_abs = dg.abs() + 2.0 ** 8 * D.abs() * (eg * (zu.abs() + eu) + 1.2 * eu)
    du_abs = du.abs() + 2.0 ** 8 * D.abs() * eg
    grad_check(dx, dg @ G.t() + du @ U.t(), dg_abs @ G.abs().t() + du_abs @ U.abs().t(), "dx")
    grad_check(dwg, X.t() @ dg, X.abs().t() @ dg_abs, "dw_gate")
    grad_check(dwu, X.t() @ du, X.abs().t() @ du_abs, "dw_up")


def test_gradients_against_differences():
    """Along random directions, <gradient, d> is the central difference of the 64-bit forward, up to the
    bf16 rounding of the gradients (2^-8 of their norm, random signs)."""
    g = gen(21)
    n, c, h = 150, 72, 88
    x, (wg, wu), _, _, X, (G, U) = make(g, n, c, h, False, 2)
    dy = normal(g, n, h).to(BF)
    b = normal(g, h)
    D, t = dy.double(), 1e-5
    for act in ("silu", "gelu", "gelu_tanh"):
        dx, dwg, dwu = sc.gated_ffn_backward(dy, x, wg, wu, activation=act)
        gx, gw, gb = sc.linear_backward(dy, x, wg, bias=b, activation=act)

        def gated(X, G, U):
            return (D * act64(act, X @ G)[0] * (X @ U)).sum()

        def lin(X, G, B):
            return (D * act64(act, X @ G + B)[0]).sum()
        for _ in range(3):
            ex, eg, eu, eb = (normal(g, *s).double() for s in ((n, c), (c, h), (c, h), (h,)))
            num = (gated(X + t * ex, G + t * eg, U + t * eu) - gated(X - t * ex, G - t * eg, U - t * eu)) / (2 * t)
            ana = (dx.double() * ex).sum() + (dwg.double() * eg).sum() + (dwu.double() * eu).sum()
            size = sum((a.double().norm() ** 2 for a in (dx, dwg, dwu))) ** 0.5
            assert abs(num - ana) <= 2.0 ** -8 * 4 * size      # 4 sigma of the directions' scatter
            B = b.double()
            num = (lin(X + t * ex, G + t * eg, B + t * eb) - lin(X - t * ex, G - t * eg, B - t * eb)) / (2 * t)
            ana = (gx.double() * ex).sum() + (gw.double() * eg).sum() + (gb.double() * eb).sum()
            size = sum((a.double().norm() ** 2 for a in (gx, gw))) ** 0.5
            assert abs(num - ana) <= 2.0 ** -8 * 4 * size


@pytest.mark.parametrize("n,c,h", [(5, 64, 72), (300, 128, 264), (300, 40, 33), (300, 64, 36), (520, 1056, 60)])
def test_strides_and_in_place(n, c, h):
    g = gen(4)
    x, (wg, wu), _, _, _, _ = make(g, n, c, h, False, 2)
    r, dy = normal(g, n, h).to(BF), normal(g, n, h).to(BF)
    y, f = sc.linear(x, wg, residual=r), sc.gated_ffn(x, wg, wu)
    d1, d2 = sc.linear_backward(dy, x, wg, activation="silu"), sc.gated_ffn_backward(dy, x, wg, wu)
    for extra in (8, 24, 3, 4):
        xs, rs, ds = strided(x, extra), strided(r, extra), strided(dy, extra)
        ys = strided(torch.zeros_like(y), extra)
        fs = strided(torch.zeros_like(f), extra)
        assert torch.equal(sc.linear(xs, wg, residual=rs, out=ys), y)
        assert torch.equal(sc.gated_ffn(xs, wg, wu, out=fs), f)
        for t in (ys, fs):                     # the padding beside the rows is untouched
            assert torch.isnan(t.as_strided((n, extra), (h + extra, 1), h)[:-1]).all()
        for a, b in zip(sc.linear_backward(ds, xs, wg, activation="silu"), d1):
            assert a is b is None or torch.equal(a, b)
        for a, b in zip(sc.gated_ffn_backward(ds, xs, wg, wu), d2):
            assert torch.equal(a, b)
    r2 = r.clone()
    assert sc.linear(x, wg, residual=r2, out=r2) is r2 and torch.equal(r2, y)
    odd = torch.empty(x.numel() + 1, dtype=BF, device="cuda")[1:].view_as(x)   # 2-byte aligned only
    odd.copy_(x)
    assert torch.equal(sc.linear(odd, wg, residual=r), y)
    assert torch.equal(sc.gated_ffn(odd, wg, wu), f)


def test_infinities_and_nan_stay_in_their_rows():
    g = gen(6)
    for n in (4, 300):
        x, (wg, wu), _, _, X, (G, U) = make(g, n, 128, 96, False, 2)
        y0, f0 = sc.linear(x, wg), sc.gated_ffn(x, wg, wu)
        x2 = x.clone()
        x2[1, 7] = float("inf")
        x2[n - 1, 0] = float("nan")
        y, f = sc.linear(x2, wg), sc.gated_ffn(x2, wg, wu)
        keep = [i for i in range(n) if i not in (1, n - 1)]
        assert torch.equal(y[keep], y0[keep]) and torch.equal(f[keep], f0[keep])
        assert torch.isnan(y[n - 1]).all() and torch.isnan(f[n - 1]).all()
        assert torch.equal(y[1].float(), torch.where(wg[7] > 0, float("inf"), -float("inf")))
        big = torch.full((n, 128), 1e4, device="cuda").to(BF)
        assert torch.isfinite(sc.linear(big, wg, activation="silu")).all()


def test_no_rows():
    w = torch.randn(32, 48, device="cuda").to(BF)
    x, dy = torch.empty(0, 32, device="cuda", dtype=BF), torch.empty(0, 48, device="cuda", dtype=BF)
    b = torch.zeros(48, device="cuda")
    assert sc.linear(x, w, bias=b).shape == (0, 48) and sc.gated_ffn(x, w, w).shape == (0, 48)
    dx, dw, db = sc.linear_backward(dy, x, w, bias=b, activation="silu")
    assert dx.shape == (0, 32) and (dw == 0).all() and (db == 0).all()
    dx, dg, du = sc.gated_ffn_backward(dy, x, w, w)
    assert dx.shape == (0, 32) and (dg == 0).all() and (du == 0).all()
    wn = torch.ones(32, device="cuda")
    assert sc.rms_norm(x, wn).shape == (0, 32)
    q, s = sc.rms_norm(x, wn, quantize=True)
    assert q.shape == (0, 32) and s.shape == (0,)
    dx, dw = sc.rms_norm_backward(x, x, wn)
    assert dx.shape == (0, 32) and (dw == 0).all()


@pytest.mark.parametrize("c,h", [(1, 1), (64, 64), (130, 77), (1000, 24), (16, 3000)])
def test_quantize_weight(c, h):
    g = gen(c)
    w = normal(g, c, h, std=0.05).to(BF)
    w[:, 0] = 0
    if h > 2:
        w[:, 1] = 1e-37
    q, s = sc.quantize_weight(w)
    m = w.float().abs().amax(0)
    assert ((s.double() - m.double() / 448).abs() <= 2.0 ** -24 * s.double() + 2.0 ** -149).all()
    assert (q[0].float() == 0).all() and s[0] == 0
    if h > 2:
        assert (q[1].float() == 448).all()
    W = w.double().t()
    back = q.double() * s.double()[:, None]
    keep = slice(2, None)
    bound = (2.0 ** -4 * W.abs()).maximum(2.0 ** -10 * s.double()[:, None]) * 1.001
    assert ((back - W).abs() <= bound)[keep].all()


def test_same_bits_every_run():
    g = gen(12)
    x, (wg, wu), _, _, _, _ = make(g, 3001, 264, 520, False, 2)
    dy = normal(g, 3001, 520).to(BF)
    b = normal(g, 520)
    wn = normal(g, 264)

    def once():
        return [*sc.linear_backward(dy, x, wg, bias=b, activation="silu"), *sc.gated_ffn_backward(dy, x, wg, wu),
                *sc.rms_norm_backward(x, x, wn), sc.linear(x[:5], wg), sc.gated_ffn(x[:5], wg, wu)]
    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(once(), first))


def test_another_stream():
    """Inputs made on the default stream, the operators on another: results and later reuse are ordered."""
    g = gen(13)
    side = torch.cuda.Stream()
    x, (wg, wu), _, _, _, _ = make(g, 5000, 256, 512, False, 2)
    dy = normal(g, 5000, 512).to(BF)
    wn = normal(g, 256)
    ref = [sc.linear(x, wg, activation="silu"), sc.gated_ffn(x, wg, wu), *sc.gated_ffn_backward(dy, x, wg, wu),
           sc.rms_norm(x, wn), *sc.rms_norm_backward(x, x, wn)]
    side.wait_stream(torch.cuda.current_stream())
    got = [sc.linear(x.clone(), wg, activation="silu")]
    xc, dc = x.clone(), dy.clone()
    side.wait_stream(torch.cuda.current_stream())
    got += [sc.gated_ffn(xc, wg, wu, stream=side), *sc.gated_ffn_backward(dc, xc, wg, wu, stream=side),
            sc.rms_norm(xc, wn, stream=side), *sc.rms_norm_backward(xc, xc, wn, stream=side)]
    del xc, dc                                   # freed while the side stream may still read them
    junk = [torch.full_like(x, 7.0) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    del junk


def test_captured_in_a_graph():
    g = gen(14)
    x, (wg, wu), _, _, _, _ = make(g, 70, 128, 256, False, 2)
    wd = normal(g, 256, 128, std=1 / 16).to(BF)
    wn = normal(g, 128)
    dy = normal(g, 70, 256).to(BF)

    def block():
        y, h = sc.rms_norm(x, wn, x)
        return [sc.linear(sc.gated_ffn(y, wg, wu), wd, residual=h), *sc.gated_ffn_backward(dy, x, wg, wu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    x.copy_(normal(g, 70, 128).to(BF))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, block()))


def test_refusals():
    x = torch.randn(8, 32, device="cuda").to(BF)
    w = torch.randn(32, 48, device="cuda").to(BF)
    wn = torch.ones(32, device="cuda")
    b = torch.zeros(48, device="cuda")
    q, s = sc.quantize_weight(w)
    xq, xs = sc.rms_norm(x, wn, quantize=True)
    dy = torch.randn(8, 48, device="cuda").to(BF)
    bad = [
        lambda: sc.linear(x, w.t()), lambda: sc.linear(x, w.t().contiguous()), lambda: sc.linear(x.cpu(), w),
        lambda: sc.linear(x.float(), w.float()), lambda: sc.linear(x, w.float()), lambda: sc.linear(x, w, bias=b.to(BF)),
        lambda: sc.linear(x, w, bias=b[:-1]), lambda: sc.linear(x, w, activation="swish"),
        lambda: sc.linear(x, w, residual=dy[:4]), lambda: sc.linear(x, w, residual=dy.float()),
        lambda: sc.linear(x, w, x_scale=xs), lambda: sc.linear(xq, q), lambda: sc.linear(xq, w, x_scale=xs, w_scale=s),
        lambda: sc.linear(xq, q, x_scale=xs, w_scale=s[:-1]), lambda: sc.linear(x.t(), w),
        lambda: sc.linear(x[:1].expand(8, 32), w), lambda: sc.linear(x, w, out=dy.float()),
        lambda: sc.gated_ffn(x, w, w[:, :40]), lambda: sc.gated_ffn(x, w, w.t()), lambda: sc.gated_ffn(xq, q, q, x_scale=xs),
        lambda: sc.linear_backward(dy[:, :40], x, w), lambda: sc.linear_backward(dy, xq, q),
        lambda: sc.gated_ffn_backward(x, x, w, w), lambda: sc.rms_norm(x, wn[:-1]), lambda: sc.rms_norm(x, wn.to(BF)),
        lambda: sc.rms_norm(x.half(), wn), lambda: sc.rms_norm(x, wn, x.float()), lambda: sc.rms_norm(x[0], wn),
        lambda: sc.rms_norm(x, wn, sum_out=x[:4]), lambda: sc.rms_norm(x, None), lambda: sc.rms_norm_backward(dy, x, wn),
        lambda: sc.quantize_weight(w.float()), lambda: sc.quantize_weight(w.t()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    buf = torch.zeros(8 * 96, device="cuda", dtype=BF)
    overlapping = buf[16:16 + 8 * 48].view(8, 48)
    for f in (lambda: sc.linear(x, w, out=buf[:8 * 48].view(8, 48), residual=overlapping),
              lambda: sc.linear(buf[:8 * 32].view(8, 32), w, out=overlapping),
              lambda: sc.gated_ffn(buf[:8 * 32].view(8, 32), w, w, out=overlapping),
              lambda: sc.rms_norm(buf[:256].view(8, 32), wn, sum_out=buf[8:264].view(8, 32))):
        with pytest.raises(sc.SpconvError) as e:
            f()
        assert e.value.code == -7
    with pytest.raises(sc.SpconvError):
        sc.rms_norm(x, wn, eps=-1.0)
    with pytest.raises(sc.SpconvError):
        sc.rms_norm(x, wn, eps=float("nan"))


@pytest.mark.parametrize("n,c,dtype", [(3, 24, BF), (900, 1000, BF), (900, 1001, BF), (900, 2048, BF), (40, 17000, BF),
                                       (900, 512, torch.float32)])
def test_weight_written_by_the_call_before(n, c, dtype):
    """A norm whose weight the preceding kernel writes reads what that kernel wrote."""
    g = gen(77)
    x, w = normal(g, n, c).to(dtype), normal(g, c)
    grads = [(normal(gen(78), n, c, std=1e-2) * 2.0 ** i).to(dtype) for i in range(12)]   # (powers of two: scaled exactly)
    out = []
    for dy in grads:
        dw = sc.rms_norm_backward(dy, x, w)[1]   # (its memory is the last pass's again)
        y = sc.rms_norm(x, dw)
        dw = sc.rms_norm_backward(dy, x, w)[1]
        out.append((y, sc.rms_norm_backward(grads[0], x, dw)[0]))
    torch.cuda.synchronize()
    for i, (y, dx) in enumerate(out):
        assert torch.equal(y, out[0][0] * 2.0 ** i) and torch.equal(dx, out[0][1] * 2.0 ** i)
    assert out[0][0].abs().max() > 0 and out[0][1].abs().max() > 0


def test_no_wait_ran_out():
    """The status word of the operators' bounded waits after everything above."""
    assert sc.rows_status() == 0


def test_strided_outputs_past_32_bits():
    """Rows so far apart that the last ones lie past 2^31 elements and 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB free")
    g = gen(15)
    n, ld = 300, 1 << 24                          # 300 * 2^24 elements: 10 GB
    x, (wg, wu), _, _, X, (G, U) = make(g, n, 64, 80, False, 2)
    far = torch.empty(n * ld, dtype=BF, device="cuda").view(n, ld)
    far[:, :64] = x
    y = sc.linear(far[:, :64], wg, residual=None, out=far[:, 128:208])
    assert torch.equal(y, sc.linear(x, wg))
    wn = normal(g, 64)
    assert rel(sc.rms_norm(far[:, :64], wn), sc.rms_norm(x, wn).double()) < 2.0 ** -8
    dy = normal(g, n, 80).to(BF)
    for a, b in zip(sc.gated_ffn_backward(dy, far[:, :64], wg, wu), sc.gated_ffn_backward(dy, x, wg, wu)):
        assert torch.equal(a, b)
