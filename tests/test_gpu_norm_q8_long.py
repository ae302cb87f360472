"""The scale of the 8-bit norm's longest rows, of one value over and over: every sum that
grows by the same addend rounds the same way through a whole binade.

Tolerance (u = 2^-24).  A thread's sum of squares is 17 additions deep in a round (16-bit types; 9
in fp32), 32 rounds and D / (32 * 16384) sums of those (fp32: 8192), then 10 steps of trees: at
most 115 u at D = 2^24, of which the root keeps half.  With 10 u from the largest value, the
products and rsqrtf, 68 u of the scale; the largest value is the same in every column.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    yield


@pytest.mark.parametrize("D", [1 << 24, (1 << 24) - 8, 1 << 20, 100000])
@pytest.mark.parametrize("residual", [False, True], ids=["x", "x+r"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_constant_rows(D, residual, dt):
    for value in (127 / 64, 129 / 128):
        x = torch.full((1, D), value, dtype=DT[dt], device=DEV)
        res = torch.zeros_like(x) if residual else None
        w = torch.ones(D, dtype=DT[dt], device=DEV)
        codes, scale, _ = rn.rmsnorm_fwd_q8(x, w, 1e-6, 0.0, res)
        want = value / (value * value + 1e-6) ** 0.5 / 448
        assert abs(scale.item() - want) <= 68 * 2.0 ** -24 * want, (scale.item() / want - 1) * 2 ** 24
        assert (codes.float() == 448).all()
