"""The e4m3 results of the block products have the bits of ``quantize_blocks``: scale = max / 448, q = e4m3(v / scale), both
divisions rounded to nearest, of fp32 values v.

The products here have one term and its scale, so v is known to the bit: v = acc xs rounded once, acc a whole multiple of a
power of two, xs the row's scale.  The columns' acc are the middles of two e4m3 values and 448, so nearly every quotient
lies at or next to the middle of two e4m3 values, where the last bit of the division decides.  Nothing is tolerated.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import ACTS, E4M3, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def sums(h, g, experts=None):
    """(acc [.., h], weights whose first two columns add up to it, their scales of 1)"""
    e4 = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(E4M3).float()   # 0 to 448, ascending
    low, high = e4[56:-1], e4[57:]                                                   # from 1 on
    n = experts or 1
    pick = torch.randint(0, low.numel(), (n, h), generator=g, device="cuda")
    sign = 1.0 - 2.0 * torch.randint(0, 2, (n, h), generator=g, device="cuda")
    w = torch.zeros(n, h, 128, device="cuda")
    w[:, :, 0], w[:, :, 1] = low[pick] / 2 * sign, high[pick] / 2 * sign   # (halves of values from 1 on are e4m3 values)
    first = torch.arange(h, device="cuda") % 128 == 5                      # each block's largest
    w[:, first, 0], w[:, first, 1] = 448.0, 0.0
    acc = w.sum(2)
    scale = torch.ones(n, -(-h // 128), 1, device="cuda")
    w = w.to(E4M3)
    return (acc, w, scale) if experts else (acc[0], w[0], scale[0])


def rows(n, g):
    x = torch.zeros(n, 128, device="cuda")
    x[:, :2] = 1
    xs = torch.exp(2 * normal(g, 1, n))
    special = torch.tensor([0.0, 1e-44, 3e-39, 2e-36, 1e-30, 1e30, float("inf"), float("nan")], device="cuda")
    # scales a few units from a multiple of an eighth, where the borders of the quotients lie closest to them
    near = 1 + torch.randint(0, 8, (1, n), generator=g, device="cuda") / 8 + torch.randint(-9, 10, (1, n), generator=g, device="cuda") * 2.0 ** -23
    xs[0, 2::5] = (near * 2.0 ** torch.randint(-20, 21, (1, n), generator=g, device="cuda"))[0, 2::5]
    xs[0, 1::9] = special.repeat(n)[:xs[0, 1::9].numel()]   # zeros, scales below 2^-126, no scale at all
    return x.to(E4M3), xs


def quotients(v):
    """(q, scale) of fp32 values, by divisions in 64 bits rounded to 32 (which rounds as one division in 32 bits does).
    A scale of the smallest numbers may be rounded so far down that a quotient is past 448: it stays there."""
    n, h = v.shape
    pad = torch.nn.functional.pad(v, (0, -h % 128)).view(n, -1, 128)
    most = pad.abs().amax(2)
    scale = (most.double() / 448).float()
    q = torch.where(scale[:, :, None] == 0, 0.0, (pad.double() / scale.double()[:, :, None]).float()).clamp(-448, 448)
    return q.reshape(n, -1)[:, :h].to(E4M3), scale.t()


def same(got, v):
    for want in (quotients(v), sc.quantize_blocks(v)):
        assert torch.equal(torch.nan_to_num(got[1], 7.0, 8.0), torch.nan_to_num(want[1], 7.0, 8.0)), "scales"
        a, b = got[0].float(), want[0].float()
        assert torch.equal(torch.isnan(a), torch.isnan(b)), "NaN"
        off = (got[0].view(torch.uint8) != want[0].view(torch.uint8)) & ~torch.isnan(b)
        assert not off.any(), f"{int(off.sum())} of {off.numel()} values"


# few rows (one pass and several), whole row tiles, ragged ones; blocks of columns whole and not, rows of 16 bytes and not
SIZES = [(1, 128), (16, 200), (64, 256), (65, 128), (300, 144), (1000, 131), (2049, 512), (700, 133), (50, 67)]


@pytest.mark.parametrize("n,h", SIZES)
def test_linear(n, h):
    g = gen(n + h)
    acc, w, ws = sums(h, g)
    x, xs = rows(n, g)
    v = acc[None] * xs.t()
    same(sc.linear_blocks(x, w, xs, ws, quantize=True), v)
    same(sc.linear_blocks(x, w, xs, ws, activation="relu", quantize=True), torch.where(v < 0, 0.0, v))


@pytest.mark.parametrize("n,h", SIZES)
def test_gated(n, h):
    """The up product is the row's scale or its negative: v = (acc xs) xs, each rounded; what ReLU makes 0 has
    zeros of both signs."""
    g = gen(2 * n + h)
    acc, w, ws = sums(h, g)
    x, xs = rows(n, g)
    up = torch.zeros(h, 128, device="cuda")
    up[:, 0] = 1.0 - 2.0 * torch.randint(0, 2, (h,), generator=g, device="cuda")
    z, u = acc[None] * xs.t(), up[:, 0][None] * xs.t()
    up = up.to(E4M3)
    same(sc.gated_ffn_blocks(x, w, up, xs, ws, ws, activation="none", quantize=True), z * u)
    same(sc.gated_ffn_blocks(x, w, up, xs, ws, ws, activation="relu", quantize=True), torch.where(z < 0, 0.0, z) * u)


@pytest.mark.parametrize("n,e,h", [(40, 8, 144), (900, 3, 272)])
def test_experts(n, e, h):
    g = gen(n + e)
    acc, w, ws = sums(h, g, e)
    x, xs = rows(n, g)
    cuts = torch.randint(0, n - 3, (e - 1,), generator=g, device="cuda").sort()[0].int()
    ends = torch.tensor([2, n - 3], dtype=torch.int32, device="cuda")
    off = torch.cat((ends[:1], cuts.clamp_min(2), ends[1:]))
    v = torch.zeros(n, h, device="cuda")
    at = off.tolist()
    for i, (lo, hi) in enumerate(zip(at, at[1:])):
        v[lo:hi] = acc[i][None] * xs.t()[lo:hi]
    same(sc.linear_blocks(x, w, xs, ws, offsets=off, quantize=True), v)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [20, 400])
def test_the_values_are_the_bf16_results(n, act):
    """Whatever the activation: q times its scale is within half an e4m3 step of the bf16 result (2^-8 more)."""
    g = gen(n)
    x, xs = sc.quantize_blocks(normal(g, n, 256))
    w, ws = sc.quantize_weight_blocks(normal(g, 256, 160, std=1 / 16).bfloat16())
    y = sc.linear_blocks(x, w, xs, ws, activation=act).double()
    q, s = sc.linear_blocks(x, w, xs, ws, activation=act, quantize=True)
    step = s.t().double().repeat_interleave(128, 1)[:, :160]
    assert ((q.double() * step - y).abs() <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -11) * y.abs() + 2.0 ** -10 * step).all()
    assert sc.rows_status() == 0
