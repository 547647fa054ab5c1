"""The example block (convolution, norm, gated feed-forward, residuals) served and trained on one scan.

Bounds: every bf16 tensor along the way carries an rms rounding error of at most
2^-8 / sqrt 3 = 2.3e-3 of its values.  Served: the sum, the norm's output, h and
the result, each one rounding, the norm's output entering twice (gate and up):
below sqrt(6) 2.3e-3.  In 8 bits the norm's output and the two weights carry
e4m3's 2^-4 / sqrt 3 = 3.6e-2 each, on the feed-forward part only.  Gradients: dh,
dn and the operands' roundings, below sqrt(8) 2.3e-3.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("voxel_block", os.path.join(ROOT, "examples", "voxel_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("voxels,channels,hidden", [(1, 16, 32), (50, 64, 96), (3001, 64, 200), (15052, 128, 512)])
def test_block_against_64_bits(voxels, channels, hidden):
    from submanifold_sparse_convolution_gb300 import build as build_mod
    build_mod.build()
    r = load().run(voxels, channels, hidden, time=False)
    u = 2.0 ** -8 / 3 ** 0.5
    assert r["y"] < 6 ** 0.5 * u
    assert r["y_8bit"] < 6 ** 0.5 * u + 3 ** 0.5 * 2.0 ** -4 / 3 ** 0.5
    for k in ("d_sum", "d_norm", "d_gate", "d_up", "d_down"):
        assert r[k] < 8 ** 0.5 * u, (k, r[k])
