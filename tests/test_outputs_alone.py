"""Whatever borders and slots hold, only the outputs are written: every output lies between guard bytes, which stay."""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import BF, gen, normal

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


class Guards:
    """Stands in for torch.empty: tensors inside larger buffers."""

    def __init__(self):
        self.buffers = []

    def __call__(self, shape, *, dtype, device):
        size = torch.Size(shape).numel() * dtype.itemsize
        buf = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=device)
        self.buffers.append((buf, size))
        return buf[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self, what):
        assert self.buffers, what
        for buf, size in self.buffers:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + size:] == 0xA5).all(), what
        self.buffers.clear()


@pytest.fixture
def guards(monkeypatch):
    g = Guards()
    monkeypatch.setattr(torch, "empty", g)
    return g


def borders(n, runs):
    """In order, out of order, out of range, before and behind all rows."""
    step = [n * i // runs for i in range(runs + 1)]
    return [step, step[::-1], [-7] + step[1:], step[:-1] + [n + 9], [n // 2] * (runs + 1), [2 ** 31 - 1] * (runs + 1),
            [-2 ** 31] * (runs + 1), [0] + [2 ** 31 - 1, -2 ** 31] * (runs // 2) + [n] * (runs % 2 + 0)]


# clusters, pieces of one scan and of several; whole vectors and single values
@pytest.mark.parametrize("n,c,groups,scans", [(1000, 64, 8, 4), (997, 35, 5, 4), (9001, 130, 10, 2), (40000, 66, 6, 2), (50, 8191, 1, 2)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_group_norm(n, c, groups, scans, dtype, guards):
    g = gen(n)
    x, w = normal(g, n, c).to(dtype), 1 + normal(g, c)
    for cuts in borders(n, scans):
        off = torch.tensor(cuts[:scans + 1], dtype=torch.int64, device="cuda").int()
        _, st = sc.group_norm(x, w, w, groups, offsets=off, activation="silu", stats=True)
        guards.check(f"group_norm {cuts}")
        sc.group_norm_backward(x, x, w, w, groups, torch.ones_like(st), offsets=off, activation="silu")
        guards.check(f"group_norm_backward {cuts}")
    sc.rows_status()


@pytest.mark.parametrize("n,c,h", [(40, 256, 64), (41, 2048, 77), (900, 128, 64), (901, 272, 131)])
def test_products(n, c, h, guards):
    g = gen(n)
    e = 4
    q, s = sc.quantize_blocks(normal(g, n, c))
    wq, ws = sc.quantize_weight_blocks(normal(g, e, c, h).to(BF))
    guards.check("quantised")
    r, b = normal(g, n, h).to(BF), normal(g, e, h)
    for cuts in borders(n, e):
        off = torch.tensor(cuts[:e + 1], dtype=torch.int64, device="cuda").int()
        sc.linear_blocks(q, wq, s, ws, offsets=off, bias=b, residual=r)
        sc.linear_blocks(q, wq, s, ws, offsets=off, quantize=True)
        sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off)
        sc.gated_ffn_blocks(q, wq, wq, s, ws, ws, offsets=off, quantize=True)
        guards.check(f"products {cuts}")
        # columns of a wider buffer: the others stay
        for extra in (8, 3):
            wide = torch.full((n, h + extra), 7.0, dtype=BF, device="cuda")
            sc.linear_blocks(q, wq, s, ws, offsets=off, out=wide[:, :h])
            assert (wide[:, h:] == 7).all()
    sc.rows_status()


@pytest.mark.parametrize("t,k,c", [(40, 2, 64), (333, 3, 35), (2000, 4, 136)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_experts(t, k, c, dtype, guards):
    g = gen(t)
    e = 5
    x, y, w = normal(g, t, c).to(dtype), normal(g, t * k, c).to(dtype), normal(g, t, k)
    for low, high in ((0, e), (-3, e), (-2 ** 31, 2 ** 31 - 1)):
        chosen = torch.randint(low, high, (t, k), generator=g, device="cuda", dtype=torch.int64)
        for size in (torch.int32, torch.int64):
            sc.expert_plan(chosen.to(size), e)
        guards.check(f"plan {low}")
    for slots in (torch.randint(-5, t * k + 5, (t, k), generator=g, device="cuda"), torch.full((t, k), 2 ** 31 - 1, device="cuda"),
                  torch.full((t, k), -2 ** 31, device="cuda")):
        for last in (0, t * k, t * k + 100, -100, 2 ** 31 - 1):
            off = torch.tensor([0] * e + [last], device="cuda").int()
            plan = sc.ExpertPlan(off, torch.zeros(t * k, dtype=torch.int32, device="cuda"), slots.int())
            sc.expert_gather(x, plan)
            sc.expert_gather(x, plan, quantize=True)
            sc.expert_combine(y, plan, w, residual=x)
            sc.expert_gather_backward(y, plan)
            sc.expert_combine_backward(x, y, plan, w)
            guards.check(f"experts {last}")
    sc.rows_status()
