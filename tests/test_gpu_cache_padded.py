"""The append into 8-bit caches from padded buffers: token and head strides of their own for
q, k and v, starts off 16-byte boundaries, and one head, whose stride divides nothing.

Tolerances as in test_gpu_kv_cache8.py.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn
from test_gpu_kv_cache8 import DEV, DT, check_written, make_cache, untouched
from test_gpu_rope_axes import check, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def padded(g, T, H, Dh, dtype, more, wider, first):
    """(heads, their buffer): [T, H, Dh] out of [T, H + more, Dh + wider], from element `first` of a head on."""
    buf = torch.full((T, H + more, Dh + wider), 9.0, dtype=dtype, device=DEV)
    x = buf[:, :H, first:first + Dh]
    x.copy_(torch.randn(T, H, Dh, generator=g) * 2)
    return x, buf


SHAPES = [  # T, Hq, Hkv, Dh, pairs
    (5, 1, 1, 30, (14,)), (1, 1, 1, 30, (14,)), (40, 4, 1, 30, (6, 8)), (9, 1, 3, 62, (20,)), (300, 1, 1, 126, (62,)),
    (7, 2, 1, 254, (126,)), (2500, 1, 1, 100, (50,)), (3, 1, 1, 510, (254,)), (6, 3, 1, 128, (64,)), (4, 1, 2, 64, (16,)),
    (5, 1, 1, 31, (15,)), (3, 1, 1, 1022, (510,)), (11, 8, 2, 96, (24, 24)), (2, 1, 1, 2, (1,)), (3, 1, 1, 6, (2,)),
]
PADS = [(1, 1, 0), (1, 0, 0), (0, 1, 1), (2, 3, 2), (1, 2, 1), (0, 8, 0)]


@pytest.mark.parametrize("T,Hq,Hkv,Dh,pairs", SHAPES, ids=["t%d_h%d_%d_d%d_a%d" % (*s[:4], len(s[4])) for s in SHAPES])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append_from_padded_buffers(T, Hq, Hkv, Dh, pairs, interleaved, dt):
    g = torch.Generator().manual_seed(T + Dh + len(pairs))
    rot = 2 * sum(pairs)
    inv, _ = rn.rope_frequencies(rot)
    axis = rn.rope_sections(pairs) if len(pairs) > 1 else None
    of = axis if axis is not None else torch.zeros(rot // 2, dtype=torch.int32)
    kerr = 4e-7 if dt == "f32" else 8e-7
    for n, (more, wider, first) in enumerate(PADS):
        fmt = ("e4m3", "i8")[n % 2]
        (q, q_buf), (k, _), (v, _) = (padded(g, T, h, Dh, DT[dt], more, wider, first) for h in (Hq, Hkv, Hkv))
        kc, vc, ks, vs = make_cache(g, T + 5, Hkv, Dh, fmt, ("dense", "between", "packed")[n % 3])
        before = [t.contiguous().clone() for t in (kc, vc, ks, vs)]
        pos = torch.randint(0, 50000, (len(pairs), T), generator=g).to(DEV)
        slots = torch.randperm(T + 5, generator=g)[:T]
        slots[2::4] = -1
        slots = slots.to(DEV)
        how = dict(k_scale=ks, v_scale=vs, pair_axis=axis, interleaved=interleaved)
        p = pos if axis is not None else pos[0]
        want, terms = turned(q, pos, of, inv, 1.0, interleaved)
        check("q", rn.rmsnorm_kv_append(q, k, v, p, slots, kc, vc, inv, **how), want, terms, rot)
        wk, tk = turned(k, pos, of, inv, 1.0, interleaved)
        check_written("k", kc, ks, slots, wk, kerr * tk)
        check_written("v", vc, vs, slots, v.double(), torch.zeros_like(wk))
        untouched(kc, ks, slots, before[0], before[2])
        untouched(vc, vs, slots, before[1], before[3])
        # into another padded buffer, then in place: the padding stays as it was
        out, out_buf = padded(g, T, Hq, Dh, DT[dt], more, wider, first)
        rn.rmsnorm_kv_append(q, k, v, p, slots, kc, vc, inv, q_out=out, **how)
        check("q", out, want, terms, rot)
        rn.rmsnorm_kv_append(q, k, v, p, slots, kc, vc, inv, q_out=q, **how)
        assert torch.equal(q, out)
        for buf in (q_buf, out_buf):
            assert (buf[:, Hq:] == 9).all() and (buf[:, :, :first] == 9).all() and (buf[:, :, first + Dh:] == 9).all()


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("Dh,pairs", [(30, (7, 7)), (128, (32, 32)), (31, (7, 8))])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_padded_head_with_axes(Dh, pairs, interleaved, dt):
    """The same layouts without codes: the rotation, and a cache of the inputs' type."""
    g = torch.Generator().manual_seed(Dh)
    T, rot = 37, 2 * sum(pairs)
    inv, _ = rn.rope_frequencies(rot)
    axis = rn.rope_sections(pairs, in_turn=True)
    pos = torch.randint(0, 50000, (2, T), generator=g).to(DEV)
    slots = torch.randperm(T, generator=g).to(DEV)
    for more, wider, first in PADS:
        q, k, v = (padded(g, T, 1, Dh, DT[dt], more, wider, first)[0] for _ in range(3))
        qo, ko = rn.rmsnorm_rope_axes(q, k, pos, inv, axis, interleaved=interleaved)
        want_q, want_k = (turned(x, pos, axis, inv, 1.0, interleaved) for x in (q, k))
        check("q", qo, *want_q, rot)
        check("k", ko, *want_k, rot)
        kc, vc = (torch.zeros(T, 2, Dh + 1, dtype=DT[dt], device=DEV)[:, :1, 1:] for _ in range(2))
        got = rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, pair_axis=axis, interleaved=interleaved)
        # (The cache's start may ask for smaller units than the rotation's outputs: of a cos - b sin
        # those of one element round the second product, the others the first.)
        check("q", got, *want_q, rot)
        check("k", kc[slots], *want_k, rot)
        assert torch.equal(vc[slots], v)
