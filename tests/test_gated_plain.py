"""A gated product without activation: both products' sums multiplied.  Tolerances as in test_blocks.py."""
import pytest
import torch

import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod

from test_blocks import SIZES, close8, operands, product64, split
from test_rows import BF, close, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


@pytest.mark.parametrize("n,c,h", SIZES)
def test_gated_without_activation(n, c, h):
    g = gen(3 * n + c + h)
    q, s, wg, gs = operands(g, n, c, h)
    wu, us = sc.quantize_weight_blocks(normal(g, c, h, std=c ** -0.5).to(BF))
    zg, eg = product64(q, s, wg, gs)
    zu, eu = product64(q, s, wu, us)
    ref, slack = zg * zu, eg * (zu.abs() + eu) + zg.abs() * eu + 2.0 ** -24 * (zg * zu).abs()
    close(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, activation="none"), ref, slack, "h")
    close8(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, activation="none", quantize=True), ref, slack, "q")
    assert sc.rows_status() == 0


@pytest.mark.parametrize("n,e,c,h", [(64, 4, 512, 384), (1000, 7, 256, 300)])
def test_of_experts(n, e, c, h):
    g = gen(n + e)
    q, s, wg, gs = operands(g, n, c, h, e)
    wu, us = sc.quantize_weight_blocks(normal(g, e, c, h, std=c ** -0.5).to(BF))
    off = split(n, e, g, "some")
    zg, eg = product64(q, s, wg, gs, off)
    zu, eu = product64(q, s, wu, us, off)
    ref, slack = zg * zu, eg * (zu.abs() + eu) + zg.abs() * eu + 2.0 ** -24 * (zg * zu).abs()
    close(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, offsets=off, activation="none"), ref, slack, "h")
    close8(sc.gated_ffn_blocks(q, wg, wu, s, gs, us, offsets=off, activation="none", quantize=True), ref, slack, "q")
    assert sc.rows_status() == 0
