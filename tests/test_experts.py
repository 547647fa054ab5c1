"""Rows sorted by expert and back, their gradients, and rows and weights in e4m3 blocks, against plain 64-bit forms.

Tolerances, from the arithmetic: a copy is exact; a bf16 output is one rounding of an fp32 sum (relative 2^-8)
of k products, each step of the sum off by 2^-24 of its size; a dot product of C terms taken W at a time by T
threads is off by at most (C / T + 8) 2^-24 of the sum of their magnitudes.  The e4m3 form is exact: scale and
quotient are single roundings of fp32 divisions.
"""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import BF, E4M3, close, gen, normal, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def choices(t, k, e, seed, kind="some"):
    """Experts int32 [t, k]; ``kind``: all valid, ``some`` dropped, ``none``, ``one`` expert takes all, ``twice`` the
    same expert."""
    g = gen(seed)
    v = torch.randint(0, e, (t, k), generator=g, device="cuda", dtype=torch.int32)
    if kind == "some":
        v = torch.where(torch.rand(t, k, generator=g, device="cuda") < 0.2, -1, v)
    elif kind == "none":
        v.fill_(-1)
    elif kind == "one":
        v.fill_(e - 1)
    elif kind == "twice":
        v = v[:, :1].expand(t, k).contiguous()
    return v


def plan64(experts, e):
    """offsets, pairs, slots, by a stable sort on the host."""
    flat = experts.flatten().tolist()
    order = sorted((i for i, v in enumerate(flat) if 0 <= v < e), key=lambda i: flat[i])
    slots = [-1] * len(flat)
    for s, i in enumerate(order):
        slots[i] = s
    offsets = [sum(1 for v in flat if 0 <= v < x) for x in range(e + 1)] if e < 40 else None
    if offsets is None:
        count = torch.bincount(experts.flatten()[experts.flatten() >= 0].long(), minlength=e).cumsum(0).tolist()
        offsets = [0] + count
    return offsets, order + [-1] * (len(flat) - len(order)), slots


SIZES = [(1, 1, 1), (1, 8, 128), (3, 2, 2), (31, 3, 5), (257, 4, 64), (1000, 1, 7), (1025, 2, 1024), (5000, 8, 33),
         (40000, 4, 256)]


@pytest.mark.parametrize("t,k,e", SIZES)
@pytest.mark.parametrize("kind", ["all", "some", "none", "one", "twice"])
def test_plan(t, k, e, kind):
    experts = choices(t, k, e, t + e, kind)
    plan = sc.expert_plan(experts, e)
    offsets, pairs, slots = plan64(experts, e)
    assert plan.offsets.tolist() == offsets and plan.pairs.tolist() == pairs and plan.slots.flatten().tolist() == slots
    wide = sc.expert_plan(experts.long(), e)
    assert torch.equal(wide.offsets, plan.offsets) and torch.equal(wide.pairs, plan.pairs) and torch.equal(wide.slots, plan.slots)
    assert sc.rows_status() == 0


def test_plan_of_many_pairs():
    """More pairs than one pass of every chunk takes."""
    t, k, e = 150000, 4, 19
    experts = choices(t, k, e, 5)
    plan = sc.expert_plan(experts, e)
    flat = experts.flatten().long()
    key = torch.where(flat < 0, e, flat)
    order = torch.sort(key, stable=True)[1]
    live = int((flat >= 0).sum())
    assert torch.equal(plan.pairs[:live].long(), order[:live]) and (plan.pairs[live:] == -1).all()
    assert plan.offsets.tolist() == [0] + torch.bincount(flat[flat >= 0], minlength=e).cumsum(0).tolist()
    assert torch.equal(plan.slots.flatten()[order[:live]].long(), torch.arange(live, device="cuda"))


def test_an_expert_out_of_range_is_none_and_an_error():
    for dtype in (torch.int32, torch.int64):
        experts = torch.tensor([[0, 5], [2, 1], [-7, 0]], dtype=dtype, device="cuda")
        if dtype == torch.int64:
            experts[0, 1] = 1 << 40
        plan = sc.expert_plan(experts, 3)
        assert plan.offsets.tolist() == [0, 2, 3, 4] and plan.slots.tolist() == [[0, -1], [3, 2], [-1, 1]]
        assert sc.status_string(sc.rows_status()) == "coordinate out of range"
    assert sc.rows_status() == 0


def test_no_tokens():
    plan = sc.expert_plan(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert plan.offsets.tolist() == [0] * 6 and plan.slots.shape == (0, 2)
    x = torch.empty(0, 32, device="cuda")
    assert sc.expert_gather(x, plan).shape == (0, 32)
    assert sc.expert_combine(x, plan, torch.empty(0, 2, device="cuda")).shape == (0, 32)
    assert [v.shape for v in sc.expert_gather(x, plan, quantize=True)] == [(0, 32), (1, 0)]


ROWS = [(1, 8, 16, 2048), (1, 1, 1, 1), (37, 3, 5, 35), (129, 2, 8, 128), (300, 4, 6, 136), (65, 6, 64, 1000), (33, 8, 9, 4096),
        (50, 5, 4, 514), (20, 9, 30, 2052)]


def padded(plan, t, k):
    live = int(plan.offsets[-1])
    return live, plan.pairs[:live].long() // k


@pytest.mark.parametrize("t,k,e,c", ROWS)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("extra", [0, 8, 3])
@pytest.mark.parametrize("kind", ["some", "none", "twice"])
def test_rows_out_and_back(t, k, e, c, dtype, extra, kind):
    g = gen(t + c)
    plan = sc.expert_plan(choices(t, k, e, t * k, kind), e)
    live, token = padded(plan, t, k)
    x, w = normal(g, t, c).to(dtype), normal(g, t, k)
    w[plan.slots < 0] = float("nan")     # a pair of no expert has no weight
    rows = sc.expert_gather(strided(x, extra), plan)
    assert torch.equal(rows[:live], x[token]) and not rows[live:].any()
    y = normal(g, t * k, c).to(dtype)
    y[live:] = float("nan")              # nor a row
    step = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    hit = (plan.slots >= 0)[:, :, None]
    part = torch.where(hit, y[plan.slots.clamp_min(0).long()].double(), 0.0)
    terms = torch.where(hit, part * w.double()[:, :, None], 0.0)
    res = normal(g, t, c).to(dtype)
    slack = (k + 2) * 2.0 ** -24
    close(sc.expert_combine(strided(y, extra), plan, w), terms.sum(1), slack * terms.abs().sum(1), "sum", step)
    close(sc.expert_combine(y, plan, w, residual=strided(res, extra)), terms.sum(1) + res.double(),
          slack * (terms.abs().sum(1) + res.double().abs()), "sum and residual", step)
    close(sc.expert_gather_backward(strided(y, extra), plan), part.sum(1), slack * part.abs().sum(1), "dx", step)
    # gradients of the weighted sum
    dout = normal(g, t, c).to(dtype)
    w2 = torch.nan_to_num(w)
    dy, dw = sc.expert_combine_backward(strided(dout, extra), strided(y, extra), plan, w)
    want = w2.double().flatten()[plan.pairs[:live].long()][:, None] * dout.double()[token]
    close(dy[:live], want, 2.0 ** -24 * want.abs(), "dy", step)
    assert not dy[live:].any()
    dot = (part * dout.double()[:, None, :]).sum(2)
    mag = (part * dout.double()[:, None, :]).abs().sum(2)
    assert ((dw.double() - dot).abs() <= (c / 32 + 8 + 8) * 2.0 ** -24 * mag + 1e-37).all()


def test_gradient_against_differences():
    g = gen(4)
    t, k, e, c = 20, 3, 4, 24
    plan = sc.expert_plan(choices(t, k, e, 3), e)
    y, w, dout = normal(g, t * k, c), normal(g, t, k), normal(g, t, c)
    dy, dw = sc.expert_combine_backward(dout, y, plan, w)
    hit = (plan.slots >= 0)[:, :, None]

    def value(y_, w_):
        part = torch.where(hit, y_[plan.slots.clamp_min(0).long()], 0.0)
        return ((part * w_[:, :, None]).sum(1) * dout.double()).sum().item()

    # (the sum is linear in each: a difference is its derivative)
    vy, vw = (torch.randn(s, generator=g, device="cuda", dtype=torch.float64) for s in ((t * k, c), (t, k)))
    y, w = y.double(), w.double()
    for got, slope, size in (((dy.double() * vy).sum(), value(y + vy, w) - value(y - vy, w), (dy.double() * vy).abs().sum()),
                             ((dw.double() * vw).sum(), value(y, w + vw) - value(y, w - vw), (dw.double() * vw).abs().sum())):
        assert abs(got.item() - slope / 2) <= 2.0 ** -20 * size.item()


def blocks64(x):
    """q and scale of quantize_blocks, from its definition in fp32."""
    n, c = x.shape
    nb = -(-c // 128)
    v = torch.zeros(n, nb * 128, device=x.device)
    v[:, :c] = x.float()
    v = v.view(n, nb, 128)
    m = v.abs().amax(2)
    scale = m / torch.full_like(m, 448.0)
    q = torch.where(scale[:, :, None] > 0, v / scale[:, :, None], torch.zeros_like(v)).clamp(-448, 448)
    return q.view(n, -1)[:, :c].to(E4M3), scale.t().contiguous()


@pytest.mark.parametrize("n,c", [(1, 1), (1, 2048), (3, 127), (5, 128), (77, 129), (33, 1000), (300, 2056), (9, 4099), (1000, 64)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_rows_in_blocks(n, c, dtype):
    g = gen(n + c)
    x = (normal(g, n, c) * torch.exp(2 * normal(g, n, 1))).to(dtype)
    x[n // 2] = 0
    if dtype == torch.float32:
        x[n // 3] *= 1e-30
    for extra in (0, 8, 3):
        q, scale = sc.quantize_blocks(strided(x, extra))
        q2, scale2 = blocks64(x)
        assert torch.equal(scale, scale2) and torch.equal(q.view(torch.uint8) & 0x7F, q2.view(torch.uint8) & 0x7F)
        assert torch.equal(q.float(), q2.float())
    plan = sc.expert_plan(choices(n, 3, 5, n), 5)
    live, token = padded(plan, n, 3)
    rows, rscale = sc.expert_gather(x, plan, quantize=True)
    assert torch.equal(rows[:live].float(), q.float()[token]) and not rows[live:].view(torch.uint8).any()
    assert torch.equal(rscale[:, :live], scale[:, token]) and not rscale[:, live:].any()


def test_rows_in_blocks_not_finite():
    x = torch.ones(4, 256, device="cuda")
    x[1, 7], x[2, 200] = float("nan"), float("inf")
    q, scale = sc.quantize_blocks(x)
    v = q.float() * scale.t().repeat_interleave(128, 1)
    assert torch.isnan(v[1, 7]) and torch.isnan(v[2, 200]) and torch.isnan(v[1, :128]).all() and torch.isnan(v[2, 128:]).all()
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[1, :128] = keep[2, 128:] = False
    # 1 / (1 / 448) is within a rounding of 448, which e4m3 holds
    assert torch.equal(q.float()[keep], torch.full_like(x, 448.0)[keep])


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 257), (16, 1000), (1000, 20), (3, 256, 128), (5, 48, 300)])
def test_weights_in_blocks(shape):
    g = gen(sum(shape))
    w = normal(g, *shape).to(BF)
    w[..., 0, :] = 0
    q, scale = sc.quantize_weight_blocks(w)
    w3 = (w if w.dim() == 3 else w[None]).float().transpose(1, 2)
    e, h, c = w3.shape
    hb, cb = -(-h // 128), -(-c // 128)
    v = torch.zeros(e, hb * 128, cb * 128, device="cuda")
    v[:, :h, :c] = w3
    v = v.view(e, hb, 128, cb, 128)
    m = v.abs().amax((2, 4))
    s = m / torch.full_like(m, 448.0)
    ref = torch.where(s[:, :, None, :, None] > 0, v / s[:, :, None, :, None], torch.zeros_like(v)).clamp(-448, 448)
    ref = ref.reshape(e, hb * 128, cb * 128)[:, :h, :c].to(E4M3)
    assert torch.equal(scale.view_as(s), s)
    assert torch.equal(q.view(ref.shape).float(), ref.float())


def test_refusals():
    x = torch.zeros(4, 32, device="cuda")
    experts = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    plan = sc.expert_plan(experts, 3)
    w = torch.ones(4, 2, device="cuda")
    y = torch.zeros(8, 32, device="cuda")
    bad = [lambda: sc.expert_plan(experts.float(), 3), lambda: sc.expert_plan(experts[:, 0], 3), lambda: sc.expert_plan(experts.cpu(), 3),
           lambda: sc.expert_plan(experts, 0), lambda: sc.expert_plan(experts.t(), 3),
           lambda: sc.expert_gather(x[:3], plan), lambda: sc.expert_gather(x.half(), plan), lambda: sc.expert_gather(x.cpu(), plan),
           lambda: sc.expert_gather(x, sc.ExpertPlan(plan.offsets, plan.pairs, plan.slots.long())),
           lambda: sc.expert_gather(x, sc.ExpertPlan(plan.offsets.cpu(), plan.pairs, plan.slots)),
           lambda: sc.expert_combine(y[:7], plan, w), lambda: sc.expert_combine(y, plan, w[:, :1]),
           lambda: sc.expert_combine(y, plan, None), lambda: sc.expert_combine(y, plan, w, residual=x.bfloat16()),
           lambda: sc.expert_combine(y, plan, w.double()), lambda: sc.expert_gather_backward(x, plan),
           lambda: sc.expert_combine_backward(x[:2], y, plan, w), lambda: sc.expert_combine_backward(x, y.bfloat16(), plan, w),
           lambda: sc.quantize_blocks(x.half()), lambda: sc.quantize_blocks(x[0]), lambda: sc.quantize_weight_blocks(x),
           lambda: sc.quantize_weight_blocks(x.bfloat16()[0]), lambda: sc.quantize_weight_blocks(x.bfloat16().t())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(sc.SpconvError):
        sc.expert_plan(experts, 1025)


def test_a_plan_that_points_outside_is_not_followed():
    """Slots out of range count as none (a plan may come from elsewhere)."""
    plan = sc.expert_plan(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 3)
    slots = plan.slots.clone()
    slots[1, 0], slots[2, 1] = 8, -5
    off = plan.offsets.clone()
    off[-1] = -3
    bad = sc.ExpertPlan(off, plan.pairs, slots)
    x, y, w = torch.ones(4, 32, device="cuda"), torch.ones(8, 32, device="cuda"), torch.ones(4, 2, device="cuda")
    sc.expert_gather(x, bad)
    sc.expert_gather(x, bad, quantize=True)
    assert sc.expert_combine(y, bad, w)[:, 0].tolist() == [2, 1, 1, 2]
    assert sc.expert_combine_backward(x, y, bad, w)[1].tolist() == [[32, 32], [0, 32], [32, 0], [32, 32]]
