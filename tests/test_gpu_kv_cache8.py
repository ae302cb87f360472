"""rmsnorm_kv_append and rmsnorm_kv_read: caches of 8 bits against their definition in 64
bits -- head layouts, strides, odd heads, both formats, several axes, bad indices, values
that are not numbers, far rows -- and a serving step that runs them together.

Tolerances.  A rotated value is off by 8e-7 (16-bit inputs) or 4e-7 (fp32) of |a| + |b|, a
head's scale by the most of that over its values and 3 u (u = 2^-24: the constant, the
product) of itself, the argument of a code by its value's error, its scale's and 3 u more.
v is not rotated: 3 u and 6 u.  What is read back is one product and one rounding.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn
from q8_reference import TOP, U, check_codes, units
from test_gpu_rope_axes import check, turned

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


def bits(t):
    return t.view(torch.uint8)


def make_cache(g, N, H, Dh, fmt, layout):
    """(k_cache, v_cache, k_scale, v_scale) with something in them, in one of the layouts."""
    fill = torch.randint(0, 100, (N, 2, H, Dh), generator=g).to(torch.uint8).to(DEV)
    sc = torch.rand(N, 2, H, generator=g).to(DEV) + 0.5
    if layout == "dense":
        k, v = fill[:, 0].contiguous(), fill[:, 1].contiguous()
        ks, vs = sc[:, 0].contiguous(), sc[:, 1].contiguous()
    elif layout == "between":  # rows of k and v in turn, and of their scales
        k, v, ks, vs = fill[:, 0], fill[:, 1], sc[:, 0], sc[:, 1]
    elif layout == "heads_first":
        k, v = (fill[:, i].transpose(0, 1).contiguous().transpose(0, 1) for i in (0, 1))
        ks, vs = (sc[:, i].t().contiguous().t() for i in (0, 1))
    else:  # "packed": a slot's k codes, v codes and scales in one record
        codes, size = 2 * H * Dh, (2 * H * Dh + 3) // 4 * 4 + 8 * H
        buf = torch.full((N, size), 9, dtype=torch.uint8, device=DEV)
        k, v = buf[:, :H * Dh].view(N, H, Dh), buf[:, H * Dh:codes].view(N, H, Dh)
        k.copy_(fill[:, 0])
        v.copy_(fill[:, 1])
        both = buf[:, size - 8 * H:].view(torch.float32)
        both.copy_(sc.view(N, 2 * H))
        ks, vs = both[:, :H], both[:, H:]
    return k.view(FMT[fmt]), v.view(FMT[fmt]), ks, vs


def check_written(name, cache, scale, slots, x, off):
    """cache and scale rows `slots` against x [T, H, Dh] in 64 bits, off the kernel's error of x."""
    kept = slots >= 0
    x, off = x[kept], off[kept]
    top = TOP[cache.dtype]
    unit = units(x, cache.dtype)
    rel = off.amax(-1) / (unit * top) + 4 * U
    got = scale[slots[kept]].double()
    assert ((got - unit).abs() <= unit * rel).all(), name
    t = x / unit[..., None]
    check_codes(name, cache[slots[kept]] if cache.dtype == torch.int8 else bits(cache.contiguous())[slots[kept]].view(cache.dtype),
                t, off / unit[..., None] + t.abs() * (rel + 4 * U)[..., None])


def untouched(cache, scale, slots, cache0, scale0):
    rest = torch.ones(cache.shape[0], dtype=torch.bool, device=DEV)
    rest[slots[slots >= 0]] = False
    assert torch.equal(bits(cache.contiguous())[rest], bits(cache0)[rest]) and torch.equal(scale[rest], scale0[rest])


CASES = [  # T, Hq, Hkv, Dh, sections
    (1, 32, 8, 128, (64,)), (8, 32, 8, 128, (16, 24, 24)), (300, 6, 3, 80, (16,)), (2000, 8, 2, 64, (12, 20)),
    (37, 4, 2, 22, (5,)), (9, 2, 1, 96, (24, 24)), (2450, 12, 4, 64, (32,)), (41, 5, 5, 125, (20, 20, 7)),
    (5, 2, 2, 1024, (512,)), (7, 3, 2, 1022, (100, 30)), (64, 8, 8, 256, (128,)), (1, 1, 1, 2, (1,)), (3, 2, 1, 3, (1,)),
    (700, 3, 3, 192, (96,)), (21, 4, 2, 512, (256,)), (19, 2, 2, 320, (64,)),
    # long runs of tokens a warp, heads that leave lanes idle, parts of a token without q or k heads
    (5000, 8, 1, 128, (64,)), (6001, 3, 1, 64, (8, 12, 12)), (4901, 2, 2, 100, (50,)), (3000, 5, 3, 126, (63,)),
    (2, 64, 1, 64, (32,)), (3, 1, 40, 16, (8,)), (1, 130, 2, 128, (64,)), (33, 2, 70, 24, (12,)), (11, 9, 4, 112, (56,)),
    (300, 4, 2, 127, (63,)), (40, 3, 2, 250, (125,)), (30, 2, 1, 257, (128,)), (9, 2, 2, 511, (10, 245)), (50, 5, 3, 36, (9, 9)),
    (9, 2, 2, 1024, (300,)), (5, 3, 1, 1024, (52, 50)), (7, 2, 1, 1016, (4, 200)),
]


@pytest.mark.parametrize("T,Hq,Hkv,Dh,sections", CASES, ids=["t%d_h%d_%d_d%d_a%d" % (*c[:4], len(c[4])) for c in CASES])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_append_and_read(T, Hq, Hkv, Dh, sections, interleaved, fmt, dt):
    g = torch.Generator().manual_seed(T + Dh)
    rot = 2 * sum(sections)
    inv, _ = rn.rope_frequencies(rot, 10000.0)
    kerr = 4e-7 if dt == "f32" else 8e-7
    for fused, layout in ((False, "dense"), (True, "between"), (False, "packed"), (True, "heads_first")):
        qkv = (torch.randn(T, Hq + 2 * Hkv, Dh, generator=g) * 3).to(DT[dt]).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not fused:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        N = T + 9
        kc, vc, ks, vs = make_cache(g, N, Hkv, Dh, fmt, layout)
        before = [t.contiguous().clone() for t in (kc, vc, ks, vs)]
        axis = rn.rope_sections(sections) if len(sections) > 1 else None
        pos = torch.randint(0, 100000, (len(sections), T), generator=g).to(DEV)
        slots = torch.randperm(N, generator=g)[:T]
        slots[1::5] = -1
        slots = slots.to(DEV)
        how = dict(k_scale=ks, v_scale=vs, pair_axis=axis, attn_scale=1.1, interleaved=interleaved)
        p = pos if axis is not None else pos[0]
        qo = rn.rmsnorm_kv_append(q, k, v, p, slots, kc, vc, inv, **how)
        of = axis if axis is not None else torch.zeros(rot // 2, dtype=torch.int32)
        check("q", qo, *turned(q, pos, of, inv, 1.1, interleaved), rot)
        wk, tk = turned(k, pos, of, inv, 1.1, interleaved)
        check_written("k", kc, ks, slots, wk, kerr * tk)
        check_written("v", vc, vs, slots, v.double(), torch.zeros_like(wk))
        untouched(kc, ks, slots, before[0], before[2])
        untouched(vc, vs, slots, before[1], before[3])
        # q in place
        q2 = q.clone() if not fused else q
        want = qo.clone()
        rn.rmsnorm_kv_append(q2, k, v, p, slots, kc, vc, inv, q_out=q2, **how)
        assert torch.equal(q2, want)
        # read back: any rows, some of them twice, some of them padding
        R = T + 7
        at = torch.randint(-1, N, (R,), generator=g).to(DEV)
        for out in (torch.float32, torch.bfloat16, torch.float16) if layout == "dense" else (DT[dt],):
            buf = torch.full((R, 2, Hkv, Dh + (layout == "between")), 5.0, dtype=out, device=DEV)
            given = layout in ("between", "packed")
            ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, at, dtype=out, k_out=buf[:, 0, :, :Dh] if given else None,
                                        v_out=buf[:, 1, :, :Dh] if given else None)
            for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
                want = torch.zeros(R, Hkv, Dh, dtype=out, device=DEV)
                there = at >= 0
                rows = at[there]
                want[there] = (c.float()[rows] * s[rows][..., None]).to(out)
                assert got.dtype == out and torch.equal(got, want)
            assert (buf[..., Dh:] == 5).all()


@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("Dh,rot,T", [(96, 64, 100), (30, 20, 70), (64, 64, 3000), (1024, 600, 9), (42, 42, 2500)])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_append_to_a_cache_of_the_inputs_type(axes, Dh, rot, T, interleaved, dt):
    """Without scales: rmsnorm_rope_kv_append_ex, with axes the rotation of rmsnorm_rope_axes."""
    g = torch.Generator().manual_seed(3)
    Hq, Hkv = 8, 2
    q, k, v = (torch.randn(T, h, Dh, generator=g).to(DT[dt]).to(DEV) for h in (Hq, Hkv, Hkv))
    kc, vc = (torch.randn(T + 5, Hkv, Dh, generator=g).to(DT[dt]).to(DEV) for _ in range(2))
    inv, _ = rn.rope_frequencies(rot)
    slots = torch.randperm(T + 5, generator=g)[:T]
    slots[::7] = -1
    slots = slots.to(DEV)
    pos = torch.randint(0, 9000, (axes, T), generator=g).to(DEV)
    k2, v2 = kc.clone(), vc.clone()
    if axes == 1:
        a = rn.rmsnorm_kv_append(q, k, v, pos[0], slots, kc, vc, inv, interleaved=interleaved)
        b = rn.rmsnorm_rope_kv_append_ex(q, k, v, pos[0], slots, k2, v2, inv, interleaved=interleaved)
    else:
        axis = rn.rope_sections((rot // 2 - 2 * (rot // 6), rot // 6, rot // 6), in_turn=True)
        a = rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, pair_axis=axis, interleaved=interleaved)
        b, kr = rn.rmsnorm_rope_axes(q, k, pos, inv, axis, interleaved=interleaved)
        kept = slots >= 0
        k2[slots[kept]], v2[slots[kept]] = kr[kept], v[kept]
    assert torch.equal(a, b) and torch.equal(kc, k2) and torch.equal(vc, v2)
    before = a.clone()
    rn.rmsnorm_kv_append(q, k, v, pos if axes > 1 else pos[0], slots, kc, vc, inv, interleaved=interleaved, q_out=q,
                         pair_axis=axis if axes > 1 else None)
    assert torch.equal(q, before) and torch.equal(kc, k2)


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("Dh", [64, 126, 1024])
def test_zeros_and_values_that_are_not_numbers(fmt, Dh):
    g = torch.Generator().manual_seed(5)
    T, H = 6, 2
    q, k, v = (torch.randn(T, H, Dh, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    k[0, 0], v[1, 1] = 0, 0
    k[2, 0, 3] = float("nan")
    v[2, 1, Dh - 1] = float("inf")
    v[3, 0, 0] = float("-inf")
    k[4] = k[4] * 1e-38  # subnormal products
    N = 8
    kc, vc, ks, vs = make_cache(g, N, H, Dh, fmt, "dense")
    inv, _ = rn.rope_frequencies(Dh)
    pos, slots = torch.zeros(T, dtype=torch.int64, device=DEV), torch.arange(T, device=DEV)
    rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs)
    ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, slots, dtype=torch.float32)
    assert (ko[0, 0] == 0).all() and (vo[1, 1] == 0).all() and ks[0, 0] == 2.0 ** -126 and vs[1, 1] == 2.0 ** -126
    assert ko[2, 0].isnan().all() and vo[2, 1].isnan().all() and vo[3, 0].isnan().all()
    assert not ks[2, 0].isfinite() and not vs[2, 1].isfinite() and not vs[3, 0].isfinite()
    ok = torch.ones(T, H, dtype=torch.bool, device=DEV)
    ok[2, 0] = ok[4] = False
    # a step of the code's grid at most, half of it on either side, relative to the head's largest value
    step = 2 ** -4 if fmt == "e4m3" else 0.5 / 127
    for got, x, good in ((ko, k, ok), (vo, v, torch.isfinite(v.float()).all(-1))):
        x = x.float()
        assert ((got - x).abs().amax(-1) <= (step + 1e-5) * x.abs().amax(-1))[good].all()
    assert torch.isfinite(ko[4]).all() and (ks[4] >= 2.0 ** -126).all()
    assert (ko[4] - k[4].float()).abs().max() <= 2.0 ** -126 + step * k[4].float().abs().max()


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("Dh", [16, 18])
def test_bad_positions_and_slots_are_flagged(fmt, Dh):
    T = 6
    g = torch.Generator().manual_seed(10)
    q, k, v = (torch.randn(T, 2, Dh, generator=g).to(torch.float16).to(DEV) for _ in range(3))
    kc, vc, ks, vs = make_cache(g, 4, 2, Dh, fmt, "dense")
    before = [t.clone() for t in (kc, vc, ks, vs)]
    inv, _ = rn.rope_frequencies(Dh)
    pos = torch.tensor([1, 2, -1, 3, 4, 5], device=DEV)
    slots = torch.tensor([0, 4, 1, 1 << 40, 2, -1], device=DEV)
    qo = torch.full_like(q, 7.0)
    rn.rmsnorm_device_status(clear=True)
    rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs, q_out=qo)
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert (qo[2] == 7).all()
    written = torch.tensor([0, -1, -1, -1, 2, -1], device=DEV)
    untouched(kc, ks, written, before[0], before[2])
    untouched(vc, vs, written, before[1], before[3])
    check_written("v", vc, vs, written, v.double(), torch.zeros_like(v.double()))
    ok = torch.tensor([0, 1, 3, 4, 5], device=DEV)
    zero = torch.zeros(Dh // 2, dtype=torch.int32)
    w, t = turned(q, pos.clamp(min=0)[None], zero, inv, 1.0, False)
    check("q", qo[ok], w[ok], t[ok], Dh)
    at = torch.tensor([0, 4, -1, 1 << 40, -(1 << 40), 2], device=DEV)
    ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, at, dtype=torch.float16)
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert (ko[1:5] == 0).all() and (vo[1:5] == 0).all()
    assert torch.equal(vo[0], (vc[0].float() * vs[0][:, None]).half())


def test_far_rows_of_a_large_cache():
    """Offsets past 2^32 bytes into the cache, and past 2^31 elements of what is read."""
    H, Dh, N = 8, 128, (1 << 32) // 1024 + 600
    kc = torch.zeros(N, H, Dh, dtype=torch.int8, device=DEV)
    vc = torch.zeros(N, H, Dh, dtype=torch.int8, device=DEV)
    ks, vs = torch.zeros(N, H, device=DEV), torch.zeros(N, H, device=DEV)
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(4, h, Dh, generator=g).to(torch.bfloat16).to(DEV) for h in (8, H, H))
    slots = torch.tensor([N - 1, 0, N // 2, (1 << 31) // 1024], device=DEV)
    inv, _ = rn.rope_frequencies(Dh)
    pos = torch.tensor([5, 6, 7, 8], device=DEV)
    rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs)
    zero = torch.zeros(Dh // 2, dtype=torch.int32)
    wk, tk = turned(k, pos[None], zero, inv, 1.0, False)
    check_written("k", kc, ks, slots, wk, 8e-7 * tk)
    check_written("v", vc, vs, slots, v.double(), torch.zeros_like(wk))
    assert int((vc != 0).any(-1).any(-1).sum()) == 4 and int((ks != 0).any(-1).sum()) == 4
    T = (1 << 31) // 1024 + 77
    at = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    at[[0, T // 2, T - 2, T - 1]] = slots
    ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, at)
    for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
        assert torch.equal(got[[0, T // 2, T - 2, T - 1]], (c[slots].float() * s[slots][..., None]).bfloat16())
        assert int((got != 0).any(-1).any(-1).sum()) == 4
    del kc, vc, ko, vo
    torch.cuda.empty_cache()


def test_graph_stream_and_empty():
    g = torch.Generator().manual_seed(11)
    T, H, Dh, N = 64, 4, 64, 100
    q, k, v = (torch.randn(T, H, Dh, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    inv, _ = rn.rope_frequencies(Dh)
    pos, slots = torch.arange(T, device=DEV), torch.randperm(N, generator=g)[:T].to(DEV)
    a, b = make_cache(g, N, H, Dh, "e4m3", "dense"), None
    b = [t.clone() for t in a]
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        rn.rmsnorm_kv_append(q, k, v, pos, slots, a[0], a[1], inv, k_scale=a[2], v_scale=a[3], q_out=qo)
        rn.rmsnorm_kv_read(*a, slots, k_out=ko, v_out=vo)
    for step in range(3):
        pos += 1000 * step
        slots.copy_(slots.roll(step))
        k.mul_(1.5)
        gr.replay()
        want_q = rn.rmsnorm_kv_append(q, k, v, pos, slots, b[0], b[1], inv, k_scale=b[2], v_scale=b[3])
        want = rn.rmsnorm_kv_read(*b, slots)
        torch.cuda.synchronize()
        assert torch.equal(qo, want_q) and torch.equal(ko, want[0]) and torch.equal(vo, want[1])
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rn.rmsnorm_kv_append(q, k, v, pos, slots, a[0], a[1], inv, k_scale=a[2], v_scale=a[3], stream=s)
    r = rn.rmsnorm_kv_read(*a, slots, stream=s)
    s.synchronize()
    assert torch.equal(r[0], ko) and torch.equal(r[1], vo)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    assert rn.rmsnorm_kv_read(*a, none)[0].shape == (0, H, Dh)
    assert rn.rmsnorm_kv_append(q[:0], k[:0], v[:0], none, none, a[0], a[1], inv, k_scale=a[2], v_scale=a[3]).shape == (0, H, Dh)
    # a cache without slots: q is rotated, every slot is padding
    e = [t[:0] for t in a]
    gone = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    got = rn.rmsnorm_kv_append(q, k, v, pos, gone, e[0], e[1], inv, k_scale=e[2], v_scale=e[3])
    assert torch.equal(got, qo) and (rn.rmsnorm_kv_read(*e, gone)[0] == 0).all()


def test_a_serving_step_in_8_bits():
    """Lengths -> plan -> 8-bit norm -> projections (plain torch here) -> append to an 8-bit cache ->
    contexts read back -> attention: against the same step in 64 bits with the same codes."""
    g = torch.Generator().manual_seed(4)
    B, W, bs, Hq, Hkv, Dh = 5, 6, 8, 4, 2, 32
    D = Hq * Dh
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    kc, vc, ks, vs = make_cache(g, 40 * bs, Hkv, Dh, "e4m3", "between")
    lens, table = i32([0] * B), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    free, count = i32(list(range(40))), i32([40])
    inv, _ = rn.rope_frequencies(32)
    axis = rn.rope_sections((4, 6, 6))
    w = (torch.rand(D, generator=g) + 0.5).to(torch.bfloat16).to(DEV)
    proj = (torch.randn(D, (Hq + 2 * Hkv) * Dh, generator=g) / D ** 0.5).to(DEV)
    seqs = [[] for _ in range(B)]
    for new in ([7, 3, 1, 0, 9], [1, 1, 1, 5, 1], [1, 1, 1, 1, 1]):
        T, n = sum(new) + 3, sum(new)  # padded
        plan = rn.rmsnorm_kv_plan(lens, i32(new), table, bs, T, free_blocks=free, free_count=count)
        x, res = (torch.randn(T, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        codes, scale, res = rn.rmsnorm_fwd_q8(x, w, 1e-6, 0.0, res)
        qkv = (codes.float() * scale[:, None]) @ proj
        qkv = qkv.to(torch.bfloat16).view(T, Hq + 2 * Hkv, Dh)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.stack([plan.positions, plan.positions // 4, plan.positions % 4])
        qo = rn.rmsnorm_kv_append(q, k, v, pos, plan.slots, kc, vc, inv, k_scale=ks, v_scale=vs, pair_axis=axis)
        ctx = rn.rmsnorm_kv_plan(torch.zeros_like(lens), lens, table, bs, int(lens.sum()) + 2, lens_out=torch.empty_like(lens))
        ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, ctx.slots, dtype=torch.float32)
        assert (ko[-2:] == 0).all() and (vo[-2:] == 0).all()
        k64 = turned(k, pos, axis, inv, 1.0, False)[0]
        for t in range(n):
            seqs[plan.requests[t]].append((k64[t], v[t].double()))
        for b in range(B):
            lo, hi = ctx.starts[b].item(), ctx.starts[b + 1].item()
            assert hi - lo == len(seqs[b])
            for i, (kt, vt) in enumerate(seqs[b]):
                # half a step of e4m3 at the head's largest value, and the rotation's error
                for got, x64 in ((ko[lo + i], kt), (vo[lo + i], vt)):
                    assert ((got - x64).abs().amax(-1) <= (2 ** -4 + 1e-5) * x64.abs().amax(-1)).all()
        for t in range(n):  # attention of each new token over its context, from what was read
            b, p = plan.requests[t].item(), plan.positions[t].item()
            lo = ctx.starts[b].item()
            kk, vv = ko[lo:lo + p + 1].repeat_interleave(2, 1), vo[lo:lo + p + 1].repeat_interleave(2, 1)
            s = torch.einsum("hd,nhd->hn", qo[t].float(), kk) / Dh ** 0.5
            y = torch.einsum("hn,nhd->hd", s.softmax(-1), vv)
            assert torch.isfinite(y).all()


def test_python_refusals():
    T, H, Dh, N = 4, 2, 16, 8
    q, k, v = (torch.zeros(T, H, Dh, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    kc, vc = (torch.zeros(N, H, Dh, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = torch.zeros(N, H, device=DEV), torch.zeros(N, H, device=DEV)
    pos, slots = torch.zeros(T, dtype=torch.int64, device=DEV), torch.arange(T, device=DEV)
    inv, _ = rn.rope_frequencies(Dh)
    both = dict(k_scale=ks, v_scale=vs)
    for a, kw in (((q, k, v, pos, slots, kc, vc, inv), {}), ((q, k, v, pos, slots, kc, vc, inv), dict(k_scale=ks)),
                  ((q, k, v, pos, slots, kc, vc.view(torch.float8_e4m3fn), inv), both),
                  ((q, k, v, pos, slots, kc.half(), vc.half(), inv), {}),
                  ((q, k, v, pos, slots, kc.bfloat16(), vc.bfloat16(), inv), both),
                  ((q, k, v, pos, slots, kc, vc[:4], inv), both), ((q, k, v, pos, slots, kc[..., :8], vc[..., :8], inv), both),
                  ((q, k, v, pos, slots, kc, vc, inv), dict(k_scale=ks[:4], v_scale=vs)),
                  ((q, k, v, pos, slots, kc, vc, inv), dict(k_scale=ks.half(), v_scale=vs)),
                  ((q, k, v, pos[None], slots, kc, vc, inv), both), ((q, k, v, pos, slots.int(), kc, vc, inv), both),
                  ((q, k, v, pos, slots, kc, vc, inv), dict(pair_axis=rn.rope_sections((8,)), **both)),
                  ((q, k[:2], v, pos, slots, kc, vc, inv), both)):
        with pytest.raises(ValueError):
            rn.rmsnorm_kv_append(*a, **kw)
    with pytest.raises(rn.RmsnormError):  # one cache, twice
        rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, kc, inv, **both)
    with pytest.raises(rn.RmsnormError):  # one scale for all of a slot's heads
        rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks[:, :1].expand(N, H), v_scale=vs)
    for a, kw in (((kc.bfloat16(), vc.bfloat16(), ks, vs, slots), {}), ((kc, vc, ks, vs, slots.int()), {}),
                  ((kc, vc, ks, vs, slots[None]), {}), ((kc, vc, ks[:2], vs, slots), {}),
                  ((kc, vc, ks, vs, slots), dict(k_out=k.float())), ((kc, vc, ks, vs, slots), dict(v_out=v[:2]))):
        with pytest.raises(ValueError):
            rn.rmsnorm_kv_read(*a, **kw)
    for d in (torch.float64, torch.int8, "bf16"):
        with pytest.raises(TypeError):
            rn.rmsnorm_kv_read(kc, vc, ks, vs, slots, dtype=d)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_kv_read(kc, vc, ks, vs, slots, k_out=k, v_out=k)
    # scales and caches may be broadcast where they are only read
    ko, _ = rn.rmsnorm_kv_read(kc, vc, ks[:, :1].expand(N, H), vs, slots)
    assert (ko == 0).all()


def test_written_tensors_count_as_changed():
    T, H, Dh, N = 4, 2, 16, 8
    q, k, v = (torch.zeros(T, H, Dh, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    kc, vc = (torch.zeros(N, H, Dh, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs, qo = torch.zeros(N, H, device=DEV), torch.zeros(N, H, device=DEV), torch.empty_like(q)
    pos, slots = torch.zeros(T, dtype=torch.int64, device=DEV), torch.arange(T, device=DEV)
    inv, _ = rn.rope_frequencies(Dh)
    t = [kc, vc, ks, vs, qo, q]
    before = [x._version for x in t]
    rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs, q_out=qo)
    assert [x._version for x in t] == [n + 1 for n in before[:5]] + before[5:]
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    before = [x._version for x in (ko, vo, kc)]
    rn.rmsnorm_kv_read(kc, vc, ks, vs, slots, k_out=ko, v_out=vo)
    assert [x._version for x in (ko, vo, kc)] == [before[0] + 1, before[1] + 1, before[2]]


def test_a_slot_read_many_times_and_scales_of_any_size():
    """The same rows over and over, and scales that take values out of the 16-bit types."""
    H, Dh, N = 2, 64, 5
    g = torch.Generator().manual_seed(12)
    kc, vc, ks, vs = make_cache(g, N, H, Dh, "i8", "dense")
    ks[1], ks[2], ks[3, 0] = 1e-30, 1e36, float("inf")
    at = torch.randint(0, N, (3000,), generator=g).to(DEV)
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, at, dtype=dt)
        for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
            want = (c.float()[at] * s[at][..., None]).to(dt)
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def test_calls_of_two_threads():
    """Two host threads, each with its own stream, caches and tokens, at once."""
    import threading
    g = torch.Generator().manual_seed(13)
    problems = []
    for T, Hq, H, Dh, fmt in ((3000, 8, 2, 128, "e4m3"), (777, 4, 4, 125, "i8")):
        q, k, v = (torch.randn(T, h, Dh, generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, H, H))
        inv, _ = rn.rope_frequencies(Dh // 4 * 2)
        pos, slots = torch.arange(T, device=DEV), torch.randperm(T + 9, generator=g)[:T].to(DEV)
        problems.append((q, k, v, pos, slots, inv, make_cache(g, T + 9, H, Dh, fmt, "dense")))

    def step(p):
        q, k, v, pos, slots, inv, c = p
        qo = rn.rmsnorm_kv_append(q, k, v, pos, slots, c[0], c[1], inv, k_scale=c[2], v_scale=c[3])
        return (qo, *rn.rmsnorm_kv_read(*c, slots))

    want = [step(p) for p in problems]
    torch.cuda.synchronize()
    same = [False, False]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [step(problems[i]) for _ in range(20)]
        s.synchronize()
        same[i] = all(torch.equal(a, b) for r in got for a, b in zip(r, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same)


@pytest.mark.parametrize("Hq,Hkv", [(0, 3), (5, 0), (1, 1), (0, 1)])
@pytest.mark.parametrize("Dh", [64, 30])
def test_without_heads_of_one_kind(Hq, Hkv, Dh):
    g = torch.Generator().manual_seed(14)
    T, N = 70, 80
    q, k, v = (torch.randn(T, h, Dh, generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    kc, vc, ks, vs = make_cache(g, N, Hkv, Dh, "i8", "dense")
    inv, _ = rn.rope_frequencies(Dh)
    pos, slots = torch.arange(T, device=DEV), torch.randperm(N, generator=g)[:T].to(DEV)
    zero = torch.zeros(Dh // 2, dtype=torch.int32)
    qo = rn.rmsnorm_kv_append(q, k, v, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs)
    if Hq:
        check("q", qo, *turned(q, pos[None], zero, inv, 1.0, False), Dh)
    if Hkv:
        wk, tk = turned(k, pos[None], zero, inv, 1.0, False)
        check_written("k", kc, ks, slots, wk, 8e-7 * tk)
        check_written("v", vc, vs, slots, v.double(), torch.zeros_like(wk))
    ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, slots)
    assert ko.shape == (T, Hkv, Dh) and vo.shape == (T, Hkv, Dh)
    axes = rn.rope_sections((Dh // 4, Dh // 2 - Dh // 4))
    both = torch.stack([pos, pos // 3])
    a, b = rn.rmsnorm_rope_axes(q, k, both, inv, axes)
    for got, x in ((a, q), (b, k)):
        if x.shape[1]:
            check("axes", got, *turned(x, both, axes, inv, 1.0, False), Dh)


@pytest.mark.parametrize("Dh", [64, 50])
def test_broadcast_inputs(Dh):
    """One head shared by all, k and v the same tensor, one token repeated."""
    g = torch.Generator().manual_seed(15)
    T, N = 40, 50
    one = torch.randn(T, 1, Dh, generator=g).to(torch.float16).to(DEV)
    row = torch.randn(1, 4, Dh, generator=g).to(torch.float16).to(DEV)
    inv, _ = rn.rope_frequencies(Dh)
    pos, slots = torch.arange(T, device=DEV), torch.arange(T, device=DEV)
    for q, k in ((one.expand(T, 4, Dh), one.expand(T, 3, Dh)), (row.expand(T, 4, Dh), row.expand(T, 4, Dh))):
        got, want = (make_cache(g, N, k.shape[1], Dh, "e4m3", "dense") for _ in range(2))
        a = rn.rmsnorm_kv_append(q, k, k, pos, slots, got[0], got[1], inv, k_scale=got[2], v_scale=got[3])
        b = rn.rmsnorm_kv_append(q.contiguous(), k.contiguous(), k.contiguous(), pos, slots, want[0], want[1], inv,
                                 k_scale=want[2], v_scale=want[3])
        assert torch.equal(a, b)
        assert all(torch.equal(bits(x)[:T], bits(y)[:T]) for x, y in zip(got, want))


@pytest.mark.parametrize("Dh,H", [(1, 3), (1, 100), (2, 33), (7, 40), (1024, 1), (1000, 5), (1023, 2), (48, 70)])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_read_head_sizes(Dh, H, fmt):
    """From one code a head to the most, from one head to more than a warp has lanes."""
    g = torch.Generator().manual_seed(Dh + H)
    for T in (1, 33, 5000):
        N = 60
        kc, vc, ks, vs = make_cache(g, N, H, Dh, fmt, "between")
        at = torch.randint(-1, N, (T,), generator=g).to(DEV)
        for dt in (torch.float16, torch.float32):
            ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, at, dtype=dt)
            for got, c, s in ((ko, kc, ks), (vo, vc, vs)):
                want = (c.float()[at] * s[at][..., None] * (at >= 0)[:, None, None]).to(dt)
                assert torch.equal(got, want)


def test_more_than_2_31_elements_of_q():
    """Offsets past 2^31 elements into q and q_out; tokens are independent."""
    T, Hq, Dh = 525_000, 32, 128
    q = torch.zeros(T, Hq, Dh, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(T, 1, Dh, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(16)
    at = torch.tensor([0, 262143, 262144, 524288, 524289, T - 1], device=DEV)
    q[at] = torch.randn(6, Hq, Dh, generator=g).to(torch.bfloat16).to(DEV)
    k[at] = torch.randn(6, 1, Dh, generator=g).to(torch.bfloat16).to(DEV)
    inv, _ = rn.rope_frequencies(Dh)
    axes = rn.rope_sections((16, 24, 24))
    pos = torch.stack([torch.arange(T, device=DEV), torch.arange(T, device=DEV) % 1000, torch.arange(T, device=DEV) // 1000])
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[at] = torch.arange(6, device=DEV)
    kc, vc, ks, vs = make_cache(g, 6, 1, Dh, "e4m3", "dense")
    qo = rn.rmsnorm_kv_append(q, k, k, pos, slots, kc, vc, inv, k_scale=ks, v_scale=vs, pair_axis=axes)
    wq, tq = turned(q[at], pos[:, at], axes, inv, 1.0, False)
    check("q", qo[at], wq, tq, Dh)
    assert int((qo != 0).any(-1).any(-1).sum()) == 6
    wk, tk = turned(k[at], pos[:, at], axes, inv, 1.0, False)
    check_written("k", kc, ks, slots[at], wk, 8e-7 * tk)
    qo, ko = rn.rmsnorm_rope_axes(q, k, pos, inv, axes, q_out=qo)
    check("q", qo[at], wq, tq, Dh)
    check("k", ko[at], wk, tk, Dh)
    del q, qo
    torch.cuda.empty_cache()
