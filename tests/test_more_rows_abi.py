"""Argument checks of the C entries of group norm, sorted rows and block products: every one returns before any CUDA call."""
import pytest

from submanifold_sparse_convolution_gb300 import _native
from submanifold_sparse_convolution_gb300 import build as build_mod

BF16, FP32, E4M3 = 0, 1, 2
INVALID, UNSUPPORTED, ALIAS = -1, -2, -7

# far apart addresses that nothing reads: every case below is refused first
A, B, C, D, E, F, G, H = (0x100000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _native.load()


def check(call, cases):
    for kw, rc in cases:
        assert call(**kw) == rc, kw


def test_group_norm(lib):
    def fwd(x=A, ldx=32, w=B, b=C, off=D, scans=2, n=4, c=32, groups=4, dt=BF16, act=0, eps=1e-5, out=E, st=F):
        return lib.spconv_group_norm(x, ldx, w, b, off, scans, n, c, groups, dt, act, eps, out, st, None)
    check(fwd, [(dict(n=-1), INVALID), (dict(c=0), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
                (dict(scans=0), INVALID), (dict(scans=(1 << 20) + 1), INVALID), (dict(off=None), INVALID), (dict(off=D + 2), INVALID),
                (dict(dt=E4M3), INVALID), (dict(act=9), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                (dict(w=None), INVALID), (dict(w=B + 2), INVALID), (dict(b=C + 1), INVALID), (dict(st=F + 4), INVALID),
                (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(ldx=31), INVALID), (dict(x=A + 1), INVALID),
                (dict(c=8193, groups=1, ldx=8193), UNSUPPORTED), (dict(out=A), ALIAS), (dict(out=B + 64), ALIAS), (dict(out=C), ALIAS),
                (dict(out=D), ALIAS), (dict(st=E + 8), ALIAS), (dict(st=A), ALIAS), (dict(n=0, st=None, x=None, out=None), 0)])

    def bwd(dy=A, x=B, w=C, b=D, st=E, off=F, scans=2, n=4, c=32, groups=4, dt=BF16, act=2, dx=G, dw=H, db=H + 4096):
        return lib.spconv_group_norm_backward(dy, 32, x, 32, w, b, st, off, scans, n, c, groups, dt, act, dx, dw, db, None)
    check(bwd, [(dict(st=None), INVALID), (dict(st=E + 4), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID),
                (dict(dy=None), INVALID), (dict(groups=3), INVALID), (dict(dx=A), ALIAS), (dict(dx=B), ALIAS), (dict(dw=C), ALIAS),
                (dict(db=H + 64), ALIAS), (dict(dx=E), ALIAS), (dict(dw=G + 16), ALIAS), (dict(dt=7), INVALID)])


def test_experts(lib):
    def plan(e=A, ib=4, t=8, k=2, ne=4, off=B, pairs=C, slots=D):
        return lib.spconv_expert_plan(e, ib, t, k, ne, off, pairs, slots, None)
    check(plan, [(dict(ib=2), INVALID), (dict(t=-1), INVALID), (dict(k=0), INVALID), (dict(ne=0), INVALID), (dict(ne=1025), INVALID),
                 (dict(k=1025), INVALID), (dict(t=1 << 29, k=2), INVALID), (dict(e=None), INVALID), (dict(e=A + 2), INVALID),
                 (dict(off=None), INVALID), (dict(pairs=None), INVALID), (dict(slots=D + 1), INVALID), (dict(pairs=A), ALIAS),
                 (dict(slots=C + 4), ALIAS), (dict(off=D), ALIAS)])

    def gather(x=A, ldx=32, slots=B, off=C, t=8, k=2, ne=4, c=32, dt=BF16, out=D, odt=BF16, scale=None):
        return lib.spconv_expert_gather(x, ldx, slots, off, t, k, ne, c, dt, out, odt, scale, None)
    check(gather, [(dict(dt=E4M3), INVALID), (dict(odt=FP32), INVALID), (dict(scale=E), INVALID), (dict(odt=E4M3), INVALID),
                   (dict(slots=None), INVALID), (dict(off=None), INVALID), (dict(ldx=8), INVALID), (dict(out=A), ALIAS),
                   (dict(out=B + 8), ALIAS), (dict(odt=E4M3, scale=D + 64), ALIAS), (dict(odt=E4M3, scale=A), ALIAS), (dict(t=0), 0)])

    def combine(y=A, ldy=32, slots=B, w=C, r=D, ldr=32, t=8, k=2, c=32, dt=BF16, out=E):
        return lib.spconv_expert_combine(y, ldy, slots, w, r, ldr, t, k, c, dt, out, None)
    check(combine, [(dict(y=None), INVALID), (dict(slots=None), INVALID), (dict(w=C + 2), INVALID), (dict(ldr=4), INVALID),
                    (dict(dt=3), INVALID), (dict(out=A), ALIAS), (dict(out=C), ALIAS), (dict(out=D + 64), ALIAS),
                    (dict(out=D, ldr=40), ALIAS), (dict(t=0), 0)])

    def grad(d=A, y=B, slots=C, off=D, w=E, t=8, k=2, ne=4, c=32, dt=BF16, dy=F, dw=G):
        return lib.spconv_expert_combine_backward(d, 32, y, 32, slots, off, w, t, k, ne, c, dt, dy, dw, None)
    check(grad, [(dict(d=None), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID), (dict(off=None), INVALID),
                 (dict(dy=A), ALIAS), (dict(dy=B), ALIAS), (dict(dw=E), ALIAS), (dict(dw=F), ALIAS), (dict(t=0), 0)])


def test_quantise(lib):
    def rows(x=A, ldx=200, n=4, c=200, dt=BF16, q=B, s=C):
        return lib.spconv_quantize_blocks(x, ldx, n, c, dt, q, s, None)
    check(rows, [(dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(s=C + 2), INVALID),
                 (dict(dt=E4M3), INVALID), (dict(ldx=199), INVALID), (dict(q=A), ALIAS), (dict(s=B + 8), ALIAS), (dict(s=A), ALIAS), (dict(n=0), 0)])

    def weight(w=A, count=2, ci=32, co=48, q=B, s=C):
        return lib.spconv_quantize_weight_blocks(w, count, ci, co, q, s, None)
    check(weight, [(dict(w=None), INVALID), (dict(w=A + 1), INVALID), (dict(count=0), INVALID), (dict(count=1025), INVALID),
                   (dict(ci=0), INVALID), (dict(q=A + 64), ALIAS), (dict(s=B), ALIAS), (dict(s=None), INVALID)])


def test_products(lib):
    def linear(x=A, ldx=64, xs=B, w=C, ws=D, off=None, ne=1, n=4, ci=64, co=32, b=None, act=0, r=None, ldr=32, out=E, ldo=32, os=None):
        return lib.spconv_linear_blocks(x, ldx, xs, w, ws, off, ne, n, ci, co, b, act, r, ldr, out, ldo, os, None)
    check(linear, [(dict(n=-1), INVALID), (dict(ci=0), INVALID), (dict(ci=24, ldx=24), UNSUPPORTED), (dict(act=7), INVALID),
                   (dict(ne=2), INVALID), (dict(ne=0), INVALID), (dict(off=F, ne=1025), INVALID), (dict(off=F + 2), INVALID),
                   (dict(x=None), INVALID), (dict(xs=None), INVALID), (dict(xs=B + 1), INVALID), (dict(w=None), INVALID),
                   (dict(w=C + 8), INVALID), (dict(ws=None), INVALID), (dict(b=F + 2), INVALID), (dict(out=None), INVALID),
                   (dict(ldo=31), INVALID), (dict(ldx=63), INVALID), (dict(r=F, ldr=31), INVALID), (dict(r=F, os=G), UNSUPPORTED),
                   (dict(os=G + 2), INVALID), (dict(out=A), ALIAS), (dict(out=C + 64), ALIAS), (dict(out=B), ALIAS), (dict(out=D), ALIAS),
                   (dict(b=E + 8), ALIAS), (dict(os=E), ALIAS), (dict(os=B), ALIAS), (dict(r=E + 16), ALIAS), (dict(off=E), ALIAS),
                   (dict(r=E, ldr=40), ALIAS), (dict(n=0, x=None, w=None, out=None), 0)])

    def gated(x=A, xs=B, wg=C, gs=D, wu=E, us=F, off=None, ne=1, n=4, ci=64, ch=32, act=2, out=G, ldo=32, os=None):
        return lib.spconv_gated_ffn_blocks(x, 64, xs, wg, gs, wu, us, off, ne, n, ci, ch, act, out, ldo, os, None)
    check(gated, [(dict(wu=None), INVALID), (dict(us=None), INVALID), (dict(wg=None), INVALID), (dict(wu=E + 1), INVALID),
                  (dict(out=E), ALIAS), (dict(out=F), ALIAS), (dict(os=G + 4), ALIAS), (dict(ci=8), UNSUPPORTED), (dict(n=0), 0)])
    assert lib.spconv_last_launch_count() == 0
