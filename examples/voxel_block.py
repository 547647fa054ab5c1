"""A residual block over the voxels of one scan, served and trained.

    x' = x + conv(x)                       submanifold convolution on the scan's map
    n  = rms_norm(x') w                    (the sum and the norm in one kernel)
    y  = x' + W_down (silu(n W_gate) * (n W_up))

The convolution, the norm with the residual's addition, the gated up-projections
and the down-projection with its residual are one launch each.  ``serve`` runs
the block in bf16, ``serve_8bit`` with the feed-forward part's first product in
e4m3, and ``feed_forward_gradients`` gives the gradients of everything after the
convolution.  Run as a program it compares each with 64-bit torch and prints the
time of a pass:

    python examples/voxel_block.py [--voxels 32371] [--channels 128] [--hidden 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import submanifold_sparse_convolution_gb300 as sc  # noqa: E402
from submanifold_sparse_convolution_gb300 import synthetic  # noqa: E402

EPS = 1e-6


class Block:
    """The block's weights; the e4m3 ones and the convolution's pack are made once."""

    def __init__(self, channels: int, hidden: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape, fan_in):
            return (torch.randn(shape, generator=g, device="cuda") * fan_in ** -0.5).bfloat16()

        self.conv = weight(27, channels, channels, fan_in=27 * channels)
        self.pack = sc.wpack_create(self.conv)
        self.norm = 1 + 0.1 * torch.randn(channels, generator=g, device="cuda")
        self.gate, self.up = (weight(channels, hidden, fan_in=channels) for _ in range(2))
        self.down = weight(hidden, channels, fan_in=hidden)
        self.gate8, self.gate_scale = sc.quantize_weight(self.gate)
        self.up8, self.up_scale = sc.quantize_weight(self.up)

    def serve(self, m: sc.Map, x: torch.Tensor) -> torch.Tensor:
        n, s = sc.rms_norm(sc.subm_forward_packed(m, x, self.pack), self.norm, residual=x, eps=EPS)
        return sc.linear(sc.gated_ffn(n, self.gate, self.up), self.down, residual=s, out=s)

    def serve_8bit(self, m: sc.Map, x: torch.Tensor) -> torch.Tensor:
        q, scale, s = sc.rms_norm(sc.subm_forward_packed(m, x, self.pack), self.norm, residual=x, eps=EPS, quantize=True)
        h = sc.gated_ffn(q, self.gate8, self.up8, x_scale=scale, gate_scale=self.gate_scale, up_scale=self.up_scale)
        return sc.linear(h, self.down, residual=s, out=s)

    def feed_forward_gradients(self, c: torch.Tensor, x: torch.Tensor, dy: torch.Tensor) -> dict:
        """Gradients of sum(y dy), c the convolution's output: of c and of x (``sum``: both are added
        into x', so it is the same) and of the weights."""
        n, s = sc.rms_norm(c, self.norm, residual=x, eps=EPS)
        h = sc.gated_ffn(n, self.gate, self.up)
        dh, d_down, _ = sc.linear_backward(dy, h, self.down)
        dn, d_gate, d_up = sc.gated_ffn_backward(dh, n, self.gate, self.up)
        ds, d_norm = sc.rms_norm_backward(dn, s, self.norm, dres=dy, eps=EPS)
        return {"sum": ds, "norm": d_norm, "gate": d_gate, "up": d_up, "down": d_down}

    def exact(self, c: torch.Tensor, x: torch.Tensor, dy: torch.Tensor):
        """y and the gradients in 64 bits from the convolution's output, by torch's autograd."""
        s, norm, gate, up, down = (t.double().requires_grad_() for t in
                                   (c.double() + x.double(), self.norm, self.gate, self.up, self.down))
        n = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * norm
        y = s + (torch.nn.functional.silu(n @ gate) * (n @ up)) @ down
        y.backward(dy.double())
        return y.detach(), {"sum": s.grad, "norm": norm.grad, "gate": gate.grad, "up": up.grad, "down": down.grad}


def relative(a: torch.Tensor, b: torch.Tensor) -> float:
    return ((a.double() - b).norm() / b.norm()).item()


def run(voxels: int, channels: int, hidden: int, time: bool = True, seed: int = 1) -> dict:
    """Errors of each path against 64 bits, and microseconds of a pass; ``seed``: of the gradient that arrives."""
    wl = synthetic.random_cloud(7, voxels, shape=(200, 200, 40), batch_size=1, c_in=channels, c_out=channels)
    m = sc.build_map(wl.coords.cuda(), wl.spatial_shape, wl.batch_size)
    x = wl.feats.cuda().bfloat16().contiguous()
    block = Block(channels, hidden)
    g = torch.Generator(device="cuda")   # (the default one starts from another seed in every process)
    g.manual_seed(seed)
    dy = (torch.randn(x.shape, generator=g, device="cuda") * 1e-2).bfloat16()
    c = sc.subm_forward_packed(m, x, block.pack)
    y, grads = block.exact(c, x, dy)
    got = block.feed_forward_gradients(c, x, dy)
    result = {"y": relative(block.serve(m, x), y), "y_8bit": relative(block.serve_8bit(m, x), y)}
    result.update({"d_" + k: relative(v, grads[k]) for k, v in got.items()})
    if sc.map_status(m) != 0 or sc.rows_status() != 0:
        raise RuntimeError("a kernel reported an error")
    if time:
        for name, f in (("serve", lambda: block.serve(m, x)), ("serve_8bit", lambda: block.serve_8bit(m, x)),
                        ("gradients", lambda: block.feed_forward_gradients(c, x, dy))):
            for _ in range(5):
                f()
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            for _ in range(50):
                f()
            b.record()
            torch.cuda.synchronize()
            result["us_" + name] = a.elapsed_time(b) * 20
    m.destroy()
    return result


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--voxels", type=int, default=32371)
    ap.add_argument("--channels", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=512)
    a = ap.parse_args()
    for name, value in run(a.voxels, a.channels, a.hidden).items():
        print(f"{name:14s} {value:9.1f} us" if name.startswith("us_") else f"{name:14s} {value:9.2e} relative error")


if __name__ == "__main__":
    main()
