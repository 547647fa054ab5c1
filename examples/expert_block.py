"""A block over the voxels of a batch of scans whose feed-forward part is made of experts.

    c = conv(x)                                    submanifold convolution on the batch's map
    h = silu(group_norm(c))                        statistics of each scan and group
    p = softmax of the k largest of h W_router     the experts of each voxel and their weights
    y = x + sum_j p_j W_down,e (silu(h W_gate,e) * (h W_up,e)),  e the voxel's j-th expert

``serve`` runs the experts in 8 bits: rows are sorted by expert as e4m3 with a
scale for each 128 values, both products of all experts are one launch each,
the hidden rows stay in 8 bits between them, and the weighted sum brings the
rows back with the residual.  ``gradients`` gives the gradients of everything
after the router's choice in bf16, each expert's products on its own run of the
sorted rows.  Run as a program it compares both with 64-bit torch and prints the
time of a pass:

    python examples/expert_block.py [--voxels 20000] [--channels 128] [--hidden 256] [--experts 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import submanifold_sparse_convolution_gb300 as sc  # noqa: E402
from submanifold_sparse_convolution_gb300 import synthetic  # noqa: E402

GROUPS = 16


class Block:
    """The block's weights; the convolution's pack and the 8-bit weights are made once."""

    def __init__(self, channels: int, hidden: int, experts: int, k: int = 2, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.experts, self.k = experts, k
        self.pack = sc.wpack_create(normal(27, channels, channels, std=(27 * channels) ** -0.5).bfloat16())
        self.norm, self.shift = 1 + normal(channels, std=0.1), normal(channels, std=0.1)
        self.router = normal(channels, experts, std=channels ** -0.5).bfloat16()
        self.gate, self.up = (normal(experts, channels, hidden, std=channels ** -0.5).bfloat16() for _ in range(2))
        self.down = normal(experts, hidden, channels, std=hidden ** -0.5).bfloat16()
        self.gate8, self.up8, self.down8 = (sc.quantize_weight_blocks(w) for w in (self.gate, self.up, self.down))

    def route(self, h: torch.Tensor):
        """(where each voxel's rows go, their weights)"""
        top, chosen = sc.linear(h, self.router).float().topk(self.k, dim=1)
        return sc.expert_plan(chosen, self.experts), torch.softmax(top, 1)

    def serve(self, m: sc.Map, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        h = sc.group_norm(sc.subm_forward_packed(m, x, self.pack), self.norm, self.shift, GROUPS, offsets=offsets, activation="silu")
        return self.feed_forward(h, x, *self.route(h))

    def feed_forward(self, h: torch.Tensor, x: torch.Tensor, plan: sc.ExpertPlan, weights: torch.Tensor) -> torch.Tensor:
        q, scale = sc.expert_gather(h, plan, quantize=True)
        q, scale = sc.gated_ffn_blocks(q, self.gate8[0], self.up8[0], scale, self.gate8[1], self.up8[1], offsets=plan.offsets,
                                       quantize=True)
        y = sc.linear_blocks(q, self.down8[0], scale, self.down8[1], offsets=plan.offsets)
        return sc.expert_combine(y, plan, weights, residual=x)

    def gradients(self, c: torch.Tensor, offsets: torch.Tensor, plan: sc.ExpertPlan, weights: torch.Tensor, dy: torch.Tensor) -> dict:
        """Gradients of sum(y dy), c the convolution's output, for a given choice of experts."""
        h, stats = sc.group_norm(c, self.norm, self.shift, GROUPS, offsets=offsets, activation="silu", stats=True)
        rows = sc.expert_gather(h, plan)
        at = plan.offsets.tolist()   # (the experts' runs, for products one by one)
        hidden = [sc.gated_ffn(rows[lo:hi], self.gate[e], self.up[e]) for e, (lo, hi) in enumerate(zip(at, at[1:]))]
        y = torch.zeros_like(rows)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            sc.linear(hidden[e], self.down[e], out=y[lo:hi])
        d_rows, d_weights = sc.expert_combine_backward(dy, y, plan, weights)
        d_in = torch.zeros_like(rows)
        grads = {"gate": torch.zeros_like(self.gate), "up": torch.zeros_like(self.up), "down": torch.zeros_like(self.down)}
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            dh, grads["down"][e], _ = sc.linear_backward(d_rows[lo:hi], hidden[e], self.down[e])
            d_in[lo:hi], grads["gate"][e], grads["up"][e] = sc.gated_ffn_backward(dh, rows[lo:hi], self.gate[e], self.up[e])
        dh = sc.expert_gather_backward(d_in, plan)
        dc, d_norm, d_shift = sc.group_norm_backward(dh, c, self.norm, self.shift, GROUPS, stats, offsets=offsets, activation="silu")
        return grads | {"c": dc, "norm": d_norm, "shift": d_shift, "weights": d_weights}

    def exact(self, c: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, plan: sc.ExpertPlan, weights: torch.Tensor, dy: torch.Tensor):
        """y and the gradients in 64 bits from the convolution's output, by torch's autograd."""
        leaves = {"c": c, "norm": self.norm, "shift": self.shift, "gate": self.gate, "up": self.up, "down": self.down, "weights": weights}
        v = {name: t.double().requires_grad_() for name, t in leaves.items()}
        at = offsets.tolist()
        h = torch.cat([torch.nn.functional.group_norm(v["c"][lo:hi].t()[None], GROUPS, v["norm"], v["shift"], 1e-5)[0].t()
                       for lo, hi in zip(at, at[1:])])
        h = torch.nn.functional.silu(h)
        y, run = x.double(), plan.offsets.tolist()
        for e, (lo, hi) in enumerate(zip(run, run[1:])):
            pair = plan.pairs[lo:hi].long()
            rows = h[pair // self.k]
            out = (torch.nn.functional.silu(rows @ v["gate"][e]) * (rows @ v["up"][e])) @ v["down"][e]
            y = y.index_add(0, pair // self.k, out * v["weights"].reshape(-1)[pair][:, None])
        y.backward(dy.double())
        return y.detach(), {name: t.grad for name, t in v.items()}


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    return ((a.double() - b).norm() / b.norm()).item()


def run(voxels: int, channels: int, hidden: int, experts: int, time: bool = True, seed: int = 1) -> dict:
    """Errors of each path against 64 bits, and microseconds of a pass."""
    wl = synthetic.random_cloud(7, voxels, shape=(100, 100, 40), batch_size=3, c_in=channels, c_out=channels)
    order = torch.sort(wl.coords[:, 0], stable=True)[1]   # scan by scan
    coords, x = wl.coords[order].cuda(), wl.feats[order].cuda().bfloat16().contiguous()
    offsets = torch.searchsorted(coords[:, 0].contiguous(), torch.arange(4, device="cuda", dtype=torch.int32)).int()
    m = sc.build_map(coords, wl.spatial_shape, wl.batch_size)
    block = Block(channels, hidden, experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dy = (torch.randn(x.shape, generator=g, device="cuda") * 1e-2).bfloat16()
    c = sc.subm_forward_packed(m, x, block.pack)
    h = sc.group_norm(c, block.norm, block.shift, GROUPS, offsets=offsets, activation="silu")
    plan, weights = block.route(h)
    y, grads = block.exact(c, x, offsets, plan, weights, dy)
    got = block.gradients(c, offsets, plan, weights, dy)
    result = {"y_8bit": relative(block.serve(m, x, offsets).double() - x.double(), y - x.double())}
    result.update({"d_" + k: relative(v, grads[k]) for k, v in got.items()})
    if sc.map_status(m) != 0 or sc.rows_status() != 0:
        raise RuntimeError("a kernel reported an error")
    if time:
        for _ in range(5):
            block.serve(m, x, offsets)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        for _ in range(50):
            block.serve(m, x, offsets)
        b.record()
        torch.cuda.synchronize()
        result["us_serve"] = a.elapsed_time(b) * 20
    m.destroy()
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--voxels", type=int, default=20000)
    ap.add_argument("--channels", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--experts", type=int, default=8)
    a = ap.parse_args()
    for name, value in run(a.voxels, a.channels, a.hidden, a.experts).items():
        print(f"{name:14s} {value:9.1f} us" if name.startswith("us_") else f"{name:14s} {value:9.2e} relative error")


if __name__ == "__main__":
    main()
