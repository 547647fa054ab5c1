"""Group norm, sorted rows and block products as they are used together: the example's block, captured and replayed
calls, several streams, and the same bits every time."""
import os
import sys

import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_rows import BF, gen, normal

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def test_the_example_runs_and_its_gradients():
    """8 bits: operands are off by up to 2^-4 each (about 2^-5.5 in the mean square), through three products of
    about 2^-5 each; gradients carry a few bf16 roundings (2^-9 in the mean square each) through two products
    and a norm."""
    r = expert_block.run(3000, 64, 96, 5, time=False)
    assert r.pop("y_8bit") < 3 * 2.0 ** -5
    for name, value in r.items():
        assert value < 8 * 2.0 ** -9, f"{name}: {value:.3g}"


def calls(n, c, h, e, k, seed):
    """Every operator once, on inputs of its own: a list of functions that give lists of tensors."""
    g = gen(seed)
    x, w, b, dy = normal(g, n, c).to(BF), 1 + normal(g, c, std=0.2), normal(g, c, std=0.2), normal(g, n, c).to(BF)
    off = torch.tensor([0, n // 3, n // 3, n - n // 8], dtype=torch.int32, device="cuda")
    _, st = sc.group_norm(x, w, b, 4, offsets=off, activation="silu", stats=True)
    experts = torch.randint(-1, e, (n, k), generator=g, device="cuda", dtype=torch.int32)
    plan = sc.expert_plan(experts, e)
    weights, rows = normal(g, n, k), normal(g, n * k, c).to(BF)
    wg, gs = sc.quantize_weight_blocks(normal(g, e, c, h, std=c ** -0.5).to(BF))
    wu, us = sc.quantize_weight_blocks(normal(g, e, c, h, std=c ** -0.5).to(BF))
    q, qs = sc.quantize_blocks(rows)
    one, ones = sc.quantize_blocks(x)

    def flat(v):
        return [v] if isinstance(v, torch.Tensor) else list(v)

    return [lambda: flat(sc.group_norm(x, w, b, 4, offsets=off, activation="silu", stats=True)),
            lambda: flat(sc.group_norm_backward(dy, x, w, b, 4, st, offsets=off, activation="silu")),
            lambda: [getattr(sc.expert_plan(experts, e), f) for f in ("offsets", "pairs", "slots")],
            lambda: flat(sc.expert_gather(x, plan)), lambda: flat(sc.expert_gather(x, plan, quantize=True)),
            lambda: flat(sc.expert_combine(rows, plan, weights, residual=x)), lambda: flat(sc.expert_gather_backward(rows, plan)),
            lambda: flat(sc.expert_combine_backward(dy, rows, plan, weights)), lambda: flat(sc.quantize_blocks(x)),
            lambda: flat(sc.linear_blocks(q, wg, qs, gs, offsets=plan.offsets)),
            lambda: flat(sc.gated_ffn_blocks(q, wg, wu, qs, gs, us, offsets=plan.offsets, quantize=True)),
            lambda: flat(sc.linear_blocks(one, wg[0], ones, gs[0], activation="gelu")),
            lambda: flat(sc.gated_ffn_blocks(one, wg[0], wu[0], ones, gs[0], us[0]))]


# few rows (clusters take scans and weights), many (all kernels of large inputs)
SHAPES = [(40, 128, 64, 6, 2), (3000, 256, 136, 4, 3), (90000, 256, 128, 3, 1)]


def alike(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SHAPES)
def test_the_same_bits_every_time(shape):
    for call in calls(*shape, seed=1):
        first = call()
        assert alike(first, call()) and alike(first, call())
    assert sc.rows_status() == 0


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_and_replayed(shape):
    """Two graphs of the same calls, replayed in turn and at once, give what the calls gave."""
    ops = calls(*shape, seed=2)
    want = [op() for op in ops]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append([op() for op in ops])
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            for group in o:
                for t in group:
                    t.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(alike(a, b) for a, b in zip(o, want))
    assert sc.rows_status() == 0


def test_streams_at_once():
    """Calls on several streams share nothing: interleaved, they give what they gave alone."""
    sets = [calls(2500, 256, 72, 4, 2, seed=s) for s in (3, 4, 5)]
    want = [[op() for op in ops] for ops in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[] for _ in sets]
    for _ in range(4):
        got = [[] for _ in sets]
        for i in range(len(sets[0])):
            for s, ops, g in zip(streams, sets, got):
                with torch.cuda.stream(s):
                    g.append(ops[i]())
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(alike(a, b) for a, b in zip(g, w))
    assert sc.rows_status() == 0


def test_a_stream_argument():
    g = gen(6)
    x, w = normal(g, 500, 64).to(BF), torch.ones(64, device="cuda")
    experts = torch.randint(0, 4, (500, 2), generator=g, device="cuda", dtype=torch.int32)
    wq, ws = sc.quantize_weight_blocks(normal(g, 4, 64, 48).to(BF))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def all_of(**kw):
        y, st = sc.group_norm(x, w, None, 4, stats=True, **kw)
        plan = sc.expert_plan(experts, 4, **kw)
        q, scale = sc.expert_gather(y, plan, quantize=True, **kw)
        out = sc.linear_blocks(q, wq, scale, ws, offsets=plan.offsets, **kw)
        weights = torch.ones(500, 2, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        back = sc.expert_combine(out, plan, weights, **kw)
        dy, dw = sc.expert_combine_backward(back, out, plan, weights, **kw)
        dx = sc.group_norm_backward(sc.expert_gather_backward(sc.expert_gather(x, plan, **kw), plan, **kw), x, w, None, 4, st, **kw)[0]
        return [y, st, q, scale, out, back, dy, dw, dx, *sc.quantize_blocks(x, **kw)]

    want = all_of()
    torch.cuda.synchronize()
    got = all_of(stream=s)
    torch.cuda.synchronize()
    assert alike(want, got)


@pytest.mark.parametrize("n,c", [(70000, 512), (9, 4096)])
def test_offsets_past_31_bits_of_bytes(n, c):
    """Rows of a wide buffer whose last bytes lie past 2^31 (the stride is as large as it has to be)."""
    ld = (1 << 31) // (2 * n) // 8 * 8 + 4096
    buf = torch.empty(n * ld, dtype=BF, device="cuda")
    x = buf.view(n, ld)[:, :c]
    g = gen(n)
    for lo in range(0, n, 8192):
        x[lo:lo + 8192] = normal(g, min(8192, n - lo), c).to(BF)
    flat = x.contiguous()
    w = torch.ones(c, device="cuda")
    assert torch.equal(sc.group_norm(x, w, None, 8), sc.group_norm(flat, w, None, 8))
    experts = torch.randint(0, 4, (n, 1), generator=g, device="cuda", dtype=torch.int32)
    plan = sc.expert_plan(experts, 4)
    assert torch.equal(sc.expert_gather(x, plan), sc.expert_gather(flat, plan))
    assert alike(sc.quantize_blocks(x), sc.quantize_blocks(flat))
    weights = normal(g, n, 1)
    assert torch.equal(sc.expert_combine(x, plan, weights), sc.expert_combine(flat, plan, weights))
