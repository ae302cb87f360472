"""Codes of the 8-bit cache on the border of two: values whose quotient by their scale is one exactly.

No tolerance.  A value x and its group's largest a of p bits each (11 at most) have a quotient
t = x top / a, and T is the border of two codes (5 bits for e4m3, 8 for int8): |t - T| is
|x top - T a| / a, a difference of two numbers of at most 19 bits, so that t is T itself or
2^-20 of T away from it.  The kernels' t is rounded once, 2^-24 of itself: it is T where t is,
and on t's side of T everywhere else.  Every code is then that of the 64-bit quotient.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn
from q8_reference import FLOOR, TOP

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FMT = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def nearest(x, fmt):
    """The codes' values of x [..., n], its last dimension a group, and how many lie on a border."""
    top = TOP[fmt]
    a = x.abs().amax(-1, keepdim=True).clamp(min=top * FLOOR)
    t = x * top / a
    if fmt == torch.int8:
        step = torch.ones_like(t)
    else:
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(t / step) * step, int(((t / step).abs().frac() == 0.5).sum())


@pytest.mark.parametrize("Dh,rot", [(128, 64), (64, 64), (90, 40), (126, 62), (125, 62), (256, 256), (513, 100), (1024, 600), (1022, 1000)])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append(Dh, rot, fmt, dt):
    """v, and k at position 0, whose cosines are 1 and whose sines are 0; fp32 values of 11 bits."""
    g = torch.Generator().manual_seed(Dh)
    T, H = 400, 3
    q, k, v = (torch.randn(T, H, Dh, generator=g).to(DT[dt if dt != "f32" else "f16"]).to(DT[dt]).to(DEV) for _ in range(3))
    kc, vc = (torch.zeros(T, H, Dh, dtype=torch.uint8, device=DEV).view(FMT[fmt]) for _ in range(2))
    ks, vs = torch.zeros(T, H, device=DEV), torch.zeros(T, H, device=DEV)
    inv, _ = rn.rope_frequencies(rot)
    none = torch.zeros(T, dtype=torch.int64, device=DEV)
    for interleaved in (False, True):
        rn.rmsnorm_kv_append(q, k, v, none, torch.arange(T, device=DEV), kc, vc, inv, k_scale=ks, v_scale=vs,
                             interleaved=interleaved)
        for name, cache, x in (("k", kc, k), ("v", vc, v)):
            want, borders = nearest(x.double(), FMT[fmt])
            assert borders > 0
            wrong = int((cache.double() != want).sum())
            assert wrong == 0, (name, wrong, borders)
