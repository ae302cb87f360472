"""rmsnorm_rope, rmsnorm_rope_kv_append_ex and rope against complex rotation in
64 bits: partial heads, both layouts, stretched frequencies, far positions,
strided and transposed heads, in place, backward, paged caches.

Tolerance.  An output is attn_scale (a c - b s): its fp32 products and their
difference are within 4 u (u = 2^-24) of |a| + |b|, and the angle's error (1e-8
turns at positions near 10^7, plus the reduced angle's own rounding, 2^-25 turns
or 2e-7 radians) and the sine's (2^-21 from the SFU, 2 u in fp32) move it by as
much times |a| + |b|: 8e-7 for 16-bit, 4e-7 for fp32 types.  Then one rounding.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def _turn(x, pos, inv, scale, interleaved, sign=1.0):
    """(rotated, |a| + |b| of each element's pair) in 64 bits; x [..., H, Dh], pos [...]."""
    x = x.double()
    rot = 2 * inv.numel()
    ang = sign * pos.double()[..., None] * inv.to(x.device)
    by = torch.polar(torch.full_like(ang, scale), ang)[..., None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    z = torch.complex(a.contiguous(), b.contiguous()) * by
    size = (a.abs() + b.abs()) * abs(scale)
    if interleaved:
        f, t = torch.stack([z.real, z.imag], -1).flatten(-2), size.repeat_interleave(2, -1)
    else:
        f, t = torch.cat([z.real, z.imag], -1), torch.cat([size, size], -1)
    return torch.cat([f, x[..., rot:]], -1), torch.cat([t, torch.zeros_like(x[..., rot:])], -1)


def _check(name, got, want, terms, rot):
    k = 4e-7 if got.dtype == torch.float32 else 8e-7
    allow = torch.finfo(got.dtype).eps / 2 * (want.abs() + k * terms) + k * terms + TINY[got.dtype]
    off = (got.double() - want).abs() - allow
    assert torch.isfinite(got).all() and off.max() <= 0, (name, off.max())
    assert torch.equal(got[..., rot:].double(), want[..., rot:]), name + ": unrotated elements"


def _heads(g, B, S, H, Dh, dtype, layout):
    """[B, S, H, Dh] in one of the layouts."""
    x = torch.randn(B, S, H, Dh, generator=g).to(dtype).to(DEV)
    if layout == "heads_first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "wide":  # heads and tokens a stride apart, off 16-byte boundaries
        buf = torch.zeros(B, S, H + 1, Dh + 3, dtype=dtype, device=DEV)
        v = buf[:, :, :H, 1:Dh + 1]
        v.copy_(x)
        return v
    return x


CASES = [  # B, S, Hq, Hkv, Dh, rot
    (1, 1, 1, 1, 2, 2), (1, 1, 32, 8, 128, 128), (2, 7, 4, 2, 64, 32), (1, 300, 8, 2, 128, 64),
    (3, 50, 6, 3, 80, 32), (1, 129, 5, 1, 96, 96), (2, 33, 2, 2, 22, 10), (1, 40, 3, 1, 30, 2),
    (1, 17, 2, 1, 1024, 1024), (2, 9, 1, 1, 512, 256), (1, 5000, 4, 1, 64, 64), (1, 64, 1, 0, 128, 128),
    (1, 70, 40, 8, 72, 40), (2, 1240, 16, 4, 64, 32), (1, 2433, 24, 2, 32, 32),
]


@pytest.mark.parametrize("B,S,Hq,Hkv,Dh,rot", CASES, ids=["b%d_s%d_h%d_%d_d%d_r%d" % c for c in CASES])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_rope_shapes(B, S, Hq, Hkv, Dh, rot, interleaved, dt):
    g = torch.Generator().manual_seed(B * S + Dh + rot)
    for i, (layout, scaling) in enumerate([("dense", None), ("heads_first", "yarn"), ("wide", "llama3")]):
        kw = {} if scaling is None else dict(factor=8.0, trained_length=8192.0)
        inv, scale = rn.rope_frequencies(rot, 500000.0, scaling, **kw)
        q = _heads(g, B, S, Hq, Dh, DT[dt], layout)
        k = _heads(g, B, S, Hkv, Dh, DT[dt], layout) if Hkv else None
        pos = torch.randint(0, [2000, 131072, 10_000_000][i], (B, S), generator=g).to(DEV)
        inverse = i == 1
        qo, ko = rn.rmsnorm_rope(q, k, pos, inv, attn_scale=scale, interleaved=interleaved, inverse=inverse)
        sign = -1.0 if inverse else 1.0
        want = _turn(q, pos, inv, scale, interleaved, sign)
        _check("q", qo, *want, rot)
        if Hkv:
            wk = _turn(k, pos, inv, scale, interleaved, sign)
            _check("k", ko, *wk, rot)
        # in place, on the same layout: the same bits
        before = qo.clone()
        r = rn.rmsnorm_rope(q, k, pos, inv, attn_scale=scale, interleaved=interleaved, inverse=inverse, q_out=q,
                            k_out=k)
        assert r[0] is q and torch.equal(q, before)
        if Hkv:
            assert torch.equal(k, ko)


def test_rope_fused_projection_in_place_leaves_v_alone():
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(100, 8 + 2 + 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    keep = qkv.clone()
    inv, _ = rn.rope_frequencies(64)
    pos = torch.arange(100, device=DEV)
    q, k = qkv[:, :8], qkv[:, 8:10]
    want = rn.rmsnorm_rope(q, k, pos, inv)
    rn.rmsnorm_rope(q, k, pos, inv, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 10:], keep[:, 10:])
    # inputs may be broadcast: one key head shared by all
    shared = keep[:, 8:9].expand(100, 4, 64)
    _, ko = rn.rmsnorm_rope(keep[:, :8], shared, pos, inv)
    assert torch.equal(ko, rn.rmsnorm_rope(keep[:, 8:9], None, pos, inv)[0].expand(100, 4, 64))


def test_rope_inverse_undoes_and_matches_differences():
    g = torch.Generator().manual_seed(6)
    q = torch.randn(37, 3, 48, generator=g).to(DEV)
    pos = torch.randint(0, 5000, (37,), generator=g).to(DEV)
    inv, _ = rn.rope_frequencies(32)
    there = rn.rmsnorm_rope(q, None, pos, inv)[0]
    back = rn.rmsnorm_rope(there, None, pos, inv, inverse=True)[0]
    assert (back - q).abs().max() <= 2 * 8e-7 * 2 * q.abs().max()
    # the map is linear: <g, rope(d)> = <rope^T(g), d>, in 64 bits from fp32 results
    go, d = torch.randn(37, 3, 48, generator=g).to(DEV), torch.randn(37, 3, 48, generator=g).to(DEV)
    left = (go.double() * rn.rmsnorm_rope(d, None, pos, inv, attn_scale=1.3)[0].double()).sum()
    right = (rn.rmsnorm_rope(go, None, pos, inv, attn_scale=1.3, inverse=True)[0].double() * d.double()).sum()
    size = 1.3 * (go.abs().double() * d.abs().double()).sum() * 4
    assert abs(left - right) <= 2 * 8e-7 * size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_autograd(dt, interleaved):
    g = torch.Generator().manual_seed(7)
    mk = lambda *s: torch.randn(*s, generator=g).to(DT[dt]).to(DEV)  # noqa: E731
    x = mk(2, 6, 30, 64)  # heads first
    q = x[:, :4].transpose(1, 2).detach().requires_grad_()
    k = x[:, 4:].transpose(1, 2).detach().requires_grad_()
    pos = torch.randint(0, 9000, (2, 30), generator=g).to(DEV)
    inv, scale = rn.rope_frequencies(32, 10000.0, "yarn", factor=4.0, trained_length=2048.0)
    qo, ko = rn.rope(q, k, pos, inv, scale, interleaved)
    gq, gk = mk(2, 4, 30, 64).transpose(1, 2), mk(1, 1, 2, 64).expand(2, 30, 2, 64)
    dq, dk = torch.autograd.grad([qo, ko], [q, k], [gq, gk], retain_graph=True)
    _check("dq", dq, *_turn(gq, pos, inv, scale, interleaved, -1.0), 32)
    _check("dk", dk, *_turn(gk, pos, inv, scale, interleaved, -1.0), 32)
    only = torch.autograd.grad(ko, k, gk)[0]
    assert torch.equal(only, dk)
    assert torch.equal(rn.rope(q, None, pos, inv, scale, interleaved)[0], qo)


@pytest.mark.parametrize("T,Hq,Hkv,Dh,rot", [(1, 32, 8, 128, 128), (8, 32, 8, 128, 64), (300, 6, 3, 80, 32),
                                             (2000, 8, 2, 64, 64), (37, 4, 2, 22, 10), (9, 2, 1, 96, 48),
                                             (2450, 12, 4, 64, 64), (4870, 20, 4, 40, 16)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append(T, Hq, Hkv, Dh, rot, interleaved, dt):
    dtype = DT[dt]
    g = torch.Generator().manual_seed(T + Dh)
    inv, scale = rn.rope_frequencies(rot, 10000.0, "linear", factor=2.0)
    for fused, inter_cache in ((False, False), (True, True)):
        qkv = torch.randn(T, Hq + 2 * Hkv, Dh, generator=g).to(dtype).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        N = T + 9
        both = torch.randn(N, 2, Hkv, Dh, generator=g).to(dtype).to(DEV)
        kc, vc = (both[:, 0], both[:, 1]) if inter_cache else (both[:, 0].contiguous(), both[:, 1].contiguous())
        k0, v0 = kc.clone(), vc.clone()
        pos = torch.randint(0, 100000, (T,), generator=g).to(DEV)
        slots = torch.randperm(N, generator=g)[:T]
        slots[::5] = -1
        slots = slots.to(DEV)
        qo = rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, kc, vc, inv, attn_scale=scale, interleaved=interleaved)
        _check("q", qo, *_turn(q, pos, inv, scale, interleaved), rot)
        kept = slots >= 0
        wk, tk = _turn(k, pos, inv, scale, interleaved)
        if kept.any():
            _check("k", kc[slots[kept]], wk[kept], tk[kept], rot)
        assert torch.equal(vc[slots[kept]], v[kept])
        rest = torch.ones(N, dtype=torch.bool, device=DEV)
        rest[slots[kept]] = False
        assert torch.equal(kc[rest], k0[rest]) and torch.equal(vc[rest], v0[rest])
        # q in place
        want = qo.clone()
        rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, kc, vc, inv, attn_scale=scale, interleaved=interleaved,
                                     q_out=q)
        assert torch.equal(q, want)


def test_append_equals_the_plain_entry_point():
    """Whole heads, unstretched: the same rotation as rmsnorm_rope_kv_append, to
    the rounding of its angles."""
    g = torch.Generator().manual_seed(8)
    T, Hq, Hkv, Dh = 50, 8, 2, 128
    q, k, v = (torch.randn(T, h, Dh, generator=g).to(torch.float16).to(DEV) for h in (Hq, Hkv, Hkv))
    pos = torch.randint(0, 50000, (T,), generator=g).to(DEV)
    slots = torch.randperm(64, generator=g)[:T].to(DEV)
    caches = [torch.zeros(64, Hkv, Dh, dtype=torch.float16, device=DEV) for _ in range(4)]
    inv, _ = rn.rope_frequencies(Dh, 10000.0)
    a = rn.rmsnorm_rope_kv_append(q, k, v, pos, slots, caches[0], caches[1], rope_base=10000.0)
    b = rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, caches[2], caches[3], inv)
    assert torch.equal(caches[1], caches[3])
    for x, y in ((a, b), (caches[0], caches[2])):
        assert (x.float() - y.float()).abs().max() <= 2 ** -11 * 2 * x.abs().max()
        assert (x != y).float().mean() < 0.01


def test_append_far_rows_of_a_large_cache():
    """Offsets past 2^32 elements into the cache."""
    Hkv, Dh, N = 8, 128, (1 << 32) // 1024 + 600
    kc = torch.zeros(N, Hkv, Dh, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros(N, Hkv, Dh, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(4, h, Dh, generator=g).to(torch.bfloat16).to(DEV) for h in (8, Hkv, Hkv))
    slots = torch.tensor([N - 1, 0, N // 2, (1 << 31) // 1024], device=DEV)
    inv, _ = rn.rope_frequencies(Dh)
    pos = torch.tensor([5, 6, 7, 8], device=DEV)
    rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, kc, vc, inv)
    assert torch.equal(vc[slots], v)
    wk, tk = _turn(k, pos, inv, 1.0, False)
    _check("k", kc[slots], wk, tk, Dh)
    assert int((vc != 0).any(-1).any(-1).sum()) == 4
    del kc, vc
    torch.cuda.empty_cache()


def test_bad_positions_and_slots_are_flagged():
    T, Dh = 6, 16
    g = torch.Generator().manual_seed(10)
    q, k, v = (torch.randn(T, 2, Dh, generator=g).to(torch.float16).to(DEV) for _ in range(3))
    kc = torch.full((4, 2, Dh), 9.0, dtype=torch.float16, device=DEV)
    vc = kc.clone()
    inv, _ = rn.rope_frequencies(Dh)
    pos = torch.tensor([1, 2, -1, 3, 4, 5], device=DEV)
    slots = torch.tensor([0, 4, 1, 1 << 40, 2, -1], device=DEV)
    qo = torch.full_like(q, 7.0)
    rn.rmsnorm_device_status(clear=True)
    rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, kc, vc, inv, q_out=qo)
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert (qo[2] == 7).all() and (vc[1] == 9).all() and (vc[3] == 9).all()
    assert torch.equal(vc[0], v[0]) and torch.equal(vc[2], v[4])
    ok = torch.tensor([0, 1, 3, 4, 5], device=DEV)
    w, t = _turn(q, pos.clamp(min=0), inv, 1.0, False)
    _check("q", qo[ok], w[ok], t[ok], Dh)
    r = rn.rmsnorm_rope(q, None, pos, inv, q_out=torch.full_like(q, 7.0))[0]
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX and (r[2] == 7).all()


def test_rope_empty_graph_and_stream():
    inv, _ = rn.rope_frequencies(16)
    e = torch.zeros(0, 2, 16, dtype=torch.float16, device=DEV)
    qo, ko = rn.rmsnorm_rope(e, e, torch.zeros(0, dtype=torch.int64, device=DEV), inv)
    assert qo.shape == e.shape and ko.shape == e.shape
    g = torch.Generator().manual_seed(11)
    q = torch.randn(64, 4, 16, generator=g).to(torch.float16).to(DEV)
    pos = torch.zeros(64, dtype=torch.int64, device=DEV)
    gr = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(gr):
        rn.rmsnorm_rope(q, None, pos, inv, q_out=out)
    for p in (3, 400):
        pos.fill_(p)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rn.rmsnorm_rope(q, None, pos, inv)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = rn.rmsnorm_rope(q, None, pos, inv, stream=s)[0]
    s.synchronize()
    assert torch.equal(r, out)


def test_rope_python_refusals():
    q = torch.zeros(4, 2, 16, dtype=torch.float16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int64, device=DEV)
    inv, _ = rn.rope_frequencies(16)
    for a in ((q[0], None, pos, inv), (q, q[:2], pos, inv), (q, q.float(), pos, inv), (q, None, pos.int(), inv),
              (q, None, pos[:2], inv), (q, None, pos, inv.float()), (q, None, pos, inv.to(DEV)),
              (q, None, pos, rn.rope_frequencies(18)[0]), (q.transpose(1, 2), None, pos, inv)):
        with pytest.raises(ValueError):
            rn.rmsnorm_rope(*a)
    with pytest.raises(TypeError):
        rn.rmsnorm_rope(q.double(), None, pos, inv)
    with pytest.raises(ValueError):
        rn.rmsnorm_rope(q, None, pos, inv, k_out=q)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_rope(q, q.clone(), pos, inv, k_out=q)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_rope(q, None, pos, inv, q_out=q[:1].expand(4, 2, 16))
