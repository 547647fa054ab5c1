"""Argument checks of the row-wise operators' C entries: every one returns before any CUDA call."""
import pytest

from submanifold_sparse_convolution_gb300 import _native
from submanifold_sparse_convolution_gb300 import build as build_mod

BF16, FP32, E4M3 = 0, 1, 2
INVALID, UNSUPPORTED, ALIAS = -1, -2, -7


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _native.load()


# far apart addresses that nothing reads: every case below is refused first
A, B, C, D, E, F = (0x100000000 * (i + 1) for i in range(6))


def linear(lib, x=A, ldx=64, xs=None, w=B, ws=None, n=4, ci=64, co=32, dt=BF16, bias=None, act=0, res=None, ldr=0, out=C,
           ldo=32):
    return lib.spconv_linear(x, ldx, xs, w, ws, n, ci, co, dt, bias, act, res, ldr, out, ldo, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INVALID), (dict(n=1 << 30), INVALID), (dict(ci=0), INVALID), (dict(co=65537), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(ldx=63), INVALID), (dict(ldo=31), INVALID), (dict(x=A + 1), INVALID),
    (dict(dt=7), INVALID), (dict(dt=FP32), UNSUPPORTED), (dict(xs=D), INVALID), (dict(dt=E4M3), INVALID),
    (dict(dt=E4M3, xs=D), INVALID), (dict(dt=E4M3, xs=D + 2, ws=E), INVALID), (dict(bias=D + 1), INVALID),
    (dict(res=D, ldr=8), INVALID), (dict(out=A), ALIAS), (dict(out=B + 64), ALIAS), (dict(res=C + 16, ldr=32), ALIAS),
    (dict(res=C, ldr=40), ALIAS), (dict(n=0, x=None, out=None), 0)])
def test_linear(lib, kw, rc):
    assert linear(lib, **kw) == rc
    assert lib.spconv_last_launch_count() == 0


def gated(lib, x=A, ldx=64, xs=None, wg=B, gs=None, wu=C, us=None, n=4, ci=64, ch=32, dt=BF16, act=2, out=D, ldo=32):
    return lib.spconv_gated_ffn(x, ldx, xs, wg, gs, wu, us, n, ci, ch, dt, act, out, ldo, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), INVALID), (dict(act=9), INVALID), (dict(wu=None), INVALID), (dict(dt=FP32), UNSUPPORTED),
    (dict(dt=E4M3, xs=E, gs=F), INVALID), (dict(us=E), INVALID), (dict(out=C), ALIAS), (dict(ldx=1), INVALID), (dict(n=0), 0)])
def test_gated(lib, kw, rc):
    assert gated(lib, **kw) == rc


def test_backward(lib):
    def lin(dy=A, ldy=32, x=B, ldx=64, w=C, n=4, ci=64, co=32, dt=BF16, bias=None, act=0, dx=D, dw=E, db=F):
        return lib.spconv_linear_backward(dy, ldy, x, ldx, w, n, ci, co, dt, bias, act, dx, dw, db, None)
    for kw, rc in [(dict(n=-2), INVALID), (dict(dt=E4M3), UNSUPPORTED), (dict(dt=FP32), UNSUPPORTED), (dict(dt=5), INVALID),
                   (dict(dy=None), INVALID), (dict(dx=B), ALIAS), (dict(dw=D + 8), ALIAS), (dict(db=F + 2), INVALID),
                   (dict(act=77), INVALID), (dict(dx=None, dw=None, db=None), 0),
                   (dict(n=0, dw=None, db=None), 0)]:
        assert lin(**kw) == rc, kw

    def gat(dh=A, ldh=32, x=B, ldx=64, wg=C, wu=C + 0x10000, n=4, ci=64, ch=32, dt=BF16, act=2, dx=D, dg=E, du=F):
        return lib.spconv_gated_ffn_backward(dh, ldh, x, ldx, wg, wu, n, ci, ch, dt, act, dx, dg, du, None)
    for kw, rc in [(dict(ch=0), INVALID), (dict(dt=FP32), UNSUPPORTED), (dict(dg=None), INVALID), (dict(du=E), ALIAS),
                   (dict(dx=A), ALIAS), (dict(ldh=31), INVALID), (dict(dx=None, dg=None, du=None), 0),
                   (dict(n=0, dg=None, du=None), 0)]:
        assert gat(**kw) == rc, kw


def test_norm(lib):
    def fwd(x=A, ldx=32, r=B, ldr=32, w=C, n=4, c=32, dt=BF16, eps=1e-6, s=D, out=E, odt=BF16, scale=None):
        return lib.spconv_rms_norm(x, ldx, r, ldr, w, n, c, dt, eps, s, out, odt, scale, None)
    for kw, rc in [(dict(c=0), INVALID), (dict(dt=E4M3, odt=E4M3), INVALID), (dict(odt=FP32), INVALID), (dict(odt=E4M3), INVALID),
                   (dict(scale=F), INVALID), (dict(eps=-1.0), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID),
                   (dict(ldr=31), INVALID), (dict(out=A), ALIAS), (dict(out=D), ALIAS), (dict(s=B + 64), ALIAS),
                   (dict(s=B, ldr=40), ALIAS), (dict(odt=E4M3, scale=E), ALIAS), (dict(n=0), 0)]:
        assert fwd(**kw) == rc, kw

    def bwd(dy=A, x=B, w=C, dres=None, n=4, c=32, dt=BF16, eps=1e-6, dx=D, dw=E):
        return lib.spconv_rms_norm_backward(dy, 32, x, 32, w, dres, 32, n, c, dt, eps, dx, dw, None)
    for kw, rc in [(dict(dt=E4M3), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(dx=A), ALIAS),
                   (dict(dw=D), ALIAS), (dict(dres=D + 64), ALIAS)]:
        assert bwd(**kw) == rc, kw


def test_quantize_weight(lib):
    def q(w=A, ci=8, co=8, out=B, s=C):
        return lib.spconv_quantize_weight(w, ci, co, out, s, None)
    for kw, rc in [(dict(w=None), INVALID), (dict(ci=0), INVALID), (dict(out=None), INVALID), (dict(s=None), INVALID),
                   (dict(out=A), ALIAS), (dict(s=B), ALIAS)]:
        assert q(**kw) == rc, kw


def test_outputs_on_vectors(lib):
    """An output may not lie on a bias, a scale or a norm's weight either."""
    cases = [linear(lib, bias=C + 8), linear(lib, dt=E4M3, xs=C + 64, ws=D), linear(lib, dt=E4M3, xs=D, ws=C),
             gated(lib, dt=E4M3, xs=D + 16, gs=E, us=F), gated(lib, dt=E4M3, xs=E, gs=D, us=F),
             gated(lib, dt=E4M3, xs=E, gs=F, us=D + 128)]
    for dx, dw, db in ((D, E, F), (E, D, F), (E, F, D)):
        cases.append(lib.spconv_linear_backward(A, 32, B, 64, C, 4, 64, 32, BF16, D, 2, dx, dw, db, None))
    for s, out, odt, scale in ((C, E, BF16, None), (D, C + 64, BF16, None), (D, E, E4M3, C)):
        cases.append(lib.spconv_rms_norm(A, 32, B, 32, C, 4, 32, BF16, 1e-6, s, out, odt, scale, None))
    for dx, dw in ((C, E), (D, C)):
        cases.append(lib.spconv_rms_norm_backward(A, 32, B, 32, C, None, 32, 4, 32, BF16, 1e-6, dx, dw, None))
    assert cases == [ALIAS] * len(cases)
