"""Cosines and sines of fp32 rotations, seen one by one: a pair (1, 0) becomes (cos, sin).

Tolerance.  Both products and the sum with 0 are exact.  sincospif is off by one step of fp32 at
most (2^-24 below 1), the sum with what the angle lost by half a step; the rest of the angle is
within 2^-24 of its own last part, 2^-24 of the turns, and of its 48-bit frequency: 3 x 2^-48 x
20000 turns x 2 pi = 0.03 x 2^-24.  1.6 x 2^-24 covers them; the reduced angle's own rounding
(2^-26 turns, 1.57 x 2^-24) has no room in it.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ALLOW = 1.6 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    yield


def pairs(T, H, Dh, interleaved):
    x = torch.zeros(T, H, Dh, device=DEV)
    if interleaved:
        x[..., 0::2] = 1
    else:
        x[..., :Dh // 2] = 1
    return x


def check(name, got, angle, interleaved, sign=1.0):
    half = got.shape[-1] // 2
    c, s = (got[..., 0::2], got[..., 1::2]) if interleaved else (got[..., :half], got[..., half:])
    angle = angle[:, None, :]
    off = max(float((c.double() - angle.cos()).abs().max()), float((s.double() - sign * angle.sin()).abs().max()))
    assert off <= ALLOW, (name, off * 2 ** 24)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("inverse", [False, True], ids=["there", "back"])
@pytest.mark.parametrize("Dh", [128, 64, 90])
def test_fp32_angles(Dh, inverse, interleaved):
    g = torch.Generator().manual_seed(Dh)
    T, sign = 20000, -1.0 if inverse else 1.0
    q = pairs(T, 1, Dh, interleaved)
    inv, _ = rn.rope_frequencies(Dh, 10000.0)
    f = inv.to(DEV)
    p = torch.randint(0, 120000, (3, T), generator=g).to(DEV)
    how = dict(interleaved=interleaved, inverse=inverse)
    check("one axis", rn.rmsnorm_rope(q, None, p[0], inv, **how)[0], p[0, :, None].double() * f, interleaved, sign)
    axis = rn.rope_sections((Dh // 2 - 20, 15, 5), in_turn=True)
    angle = p.double()[axis.long().to(DEV)].t() * f
    check("axes", rn.rmsnorm_rope_axes(q, q, p, inv, axis, **how)[1], angle, interleaved, sign)
    if inverse:
        return
    slots = torch.arange(T, device=DEV)
    k, v = (torch.zeros(T, 1, Dh, device=DEV) for _ in range(2))
    check("append", rn.rmsnorm_rope_kv_append_ex(q, q, q, p[0], slots, k, v, inv, interleaved=interleaved),
          p[0, :, None].double() * f, interleaved)
    check("append, k", k, p[0, :, None].double() * f, interleaved)
    rn.rmsnorm_kv_append(q, q, q, p, slots, k, v, inv, pair_axis=axis, interleaved=interleaved)
    check("append with axes", k, angle, interleaved)
    k8, v8 = (torch.zeros(T, 1, Dh, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(T, 1, device=DEV) for _ in range(2))
    qo = rn.rmsnorm_kv_append(q, q, q, p, slots, k8, v8, inv, k_scale=ks, v_scale=vs, pair_axis=axis, interleaved=interleaved)
    check("append to 8 bits", qo, angle, interleaved)
