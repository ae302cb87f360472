"""rmsnorm_rope_axes and rope(pair_axis=) against complex rotation in 64 bits: two to four
axes, both layouts, strided heads, in place, backward, bad positions.

Tolerance: as for one axis, the angle's error and the products' are 8e-7 (16-bit types)
or 4e-7 (fp32) of |a| + |b|, then one rounding.
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


def turned(x, pos, axis, inv, scale, interleaved, sign=1.0):
    """(rotated, |a| + |b| of each element's pair) in 64 bits; x [..., H, Dh], pos [axes, ...]."""
    x = x.double()
    rot = 2 * inv.numel()
    ang = torch.stack([sign * pos[a].double() * f for a, f in zip(axis.tolist(), inv.tolist())], -1)[..., None, :]
    c, s = ang.cos() * scale, ang.sin() * scale
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., first], x[..., second]
    out, size = x.clone(), torch.zeros_like(x)
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * abs(scale)
    return out, size


def check(name, got, want, terms, rot):
    k = 4e-7 if got.dtype == torch.float32 else 8e-7
    allow = torch.finfo(got.dtype).eps / 2 * (want.abs() + k * terms) + k * terms + TINY[got.dtype]
    off = (got.double() - want).abs() - allow
    assert torch.isfinite(got).all() and off.max() <= 0, (name, off.max())
    assert torch.equal(got[..., rot:].double(), want[..., rot:]), name + ": unrotated elements"


CASES = [  # B, S, Hq, Hkv, Dh, sections
    (1, 1, 1, 1, 4, (1, 1)), (1, 1, 32, 8, 128, (16, 24, 24)), (2, 7, 4, 2, 64, (5, 3, 8)), (1, 300, 8, 2, 128, (64, 0, 0)),
    (3, 50, 6, 3, 80, (20, 20)), (1, 129, 5, 1, 96, (1, 46, 1)), (2, 33, 2, 2, 22, (2, 1, 1, 1)),
    (1, 17, 2, 1, 1024, (100, 200, 100, 112)), (1, 5000, 4, 1, 64, (8, 12, 12)), (1, 64, 1, 0, 128, (30, 34)),
    (1, 2433, 24, 2, 32, (5, 11)), (1, 40, 3, 1, 30, (1,)),
    (1, 9, 2, 1, 1024, (100, 100, 100)), (2, 5, 1, 2, 1024, (6, 96)),
]


@pytest.mark.parametrize("B,S,Hq,Hkv,Dh,sections", CASES, ids=["b%d_s%d_h%d_%d_d%d_a%d" % (*c[:5], len(c[5])) for c in CASES])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "inter"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_shapes(B, S, Hq, Hkv, Dh, sections, interleaved, dt):
    g = torch.Generator().manual_seed(B * S + Dh)
    rot = 2 * sum(sections)
    for layout, in_turn, far, inverse in (("dense", False, 2000, False), ("heads_first", True, 131072, True), ("wide", True, 10_000_000, False)):
        axis = rn.rope_sections(sections, in_turn=in_turn)
        inv, _ = rn.rope_frequencies(rot, 500000.0)
        pos = torch.randint(0, far, (len(sections), B, S), generator=g).to(DEV)

        def heads(H):
            x = torch.randn(B, S, H, Dh, generator=g).to(DT[dt]).to(DEV)
            if layout == "heads_first":
                return x.transpose(1, 2).contiguous().transpose(1, 2)
            if layout == "wide":
                buf = torch.zeros(B, S, H + 1, Dh + 3, dtype=DT[dt], device=DEV)
                buf[:, :, :H, 1:Dh + 1].copy_(x)
                return buf[:, :, :H, 1:Dh + 1]
            return x
        q, k = heads(Hq), heads(Hkv) if Hkv else None
        how = dict(attn_scale=1.25, interleaved=interleaved, inverse=inverse)
        qo, ko = rn.rmsnorm_rope_axes(q, k, pos, inv, axis, **how)
        sign = -1.0 if inverse else 1.0
        check("q", qo, *turned(q, pos, axis, inv, 1.25, interleaved, sign), rot)
        if Hkv:
            check("k", ko, *turned(k, pos, axis, inv, 1.25, interleaved, sign), rot)
        before = qo.clone()
        assert rn.rmsnorm_rope_axes(q, k, pos, inv, axis, q_out=q, k_out=k, **how)[0] is q
        assert torch.equal(q, before) and (not Hkv or torch.equal(k, ko))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_axes_that_agree_are_one_axis(dt):
    """Text tokens: the same bits as rmsnorm_rope; and one axis is rmsnorm_rope itself."""
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(100, h, 128, generator=g).to(DT[dt]).to(DEV) for h in (8, 2))
    p = torch.randint(0, 100000, (100,), generator=g).to(DEV)
    inv, _ = rn.rope_frequencies(96)
    want = rn.rmsnorm_rope(q, k, p, inv)
    for sections in ((48,), (16, 32), (16, 16, 16), (12, 12, 12, 12)):
        axis = rn.rope_sections(sections, in_turn=True)
        got = rn.rmsnorm_rope_axes(q, k, p.expand(len(sections), 100).contiguous(), inv, axis)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_autograd(dt, interleaved):
    g = torch.Generator().manual_seed(7)
    mk = lambda *s: torch.randn(*s, generator=g).to(DT[dt]).to(DEV)  # noqa: E731
    x = mk(2, 6, 30, 64)  # heads first
    q = x[:, :4].transpose(1, 2).detach().requires_grad_()
    k = x[:, 4:].transpose(1, 2).detach().requires_grad_()
    pos = torch.randint(0, 9000, (3, 2, 30), generator=g).to(DEV)
    inv, scale = rn.rope_frequencies(32, 10000.0, "yarn", factor=4.0, trained_length=2048.0)
    axis = rn.rope_sections((4, 6, 6))
    qo, ko = rn.rope(q, k, pos, inv, scale, interleaved, axis)
    gq, gk = mk(2, 4, 30, 64).transpose(1, 2), mk(1, 1, 2, 64).expand(2, 30, 2, 64)
    dq, dk = torch.autograd.grad([qo, ko], [q, k], [gq, gk], retain_graph=True)
    check("dq", dq, *turned(gq, pos, axis, inv, scale, interleaved, -1.0), 32)
    check("dk", dk, *turned(gk, pos, axis, inv, scale, interleaved, -1.0), 32)
    assert torch.equal(torch.autograd.grad(ko, k, gk)[0], dk)
    # against differences: the map is linear, so a step of any size gives the gradient
    if dt == "f32":
        d = mk(2, 30, 4, 64)
        left = (gq.double() * (rn.rope(q.detach() + d, None, pos, inv, scale, interleaved, axis)[0].double() - qo.detach().double())).sum()
        right = (dq.double() * d.double()).sum()
        # both outputs within 4e-7 of their pairs' sizes, and u of theirs from q + d
        size = scale * (gq.abs().double() * 4 * (q.detach().abs().double() + d.abs().double() + 1)).sum()
        assert abs(left - right) <= 2e-6 * size


def test_bad_positions_on_any_axis_are_flagged():
    g = torch.Generator().manual_seed(10)
    q = torch.randn(5, 2, 16, generator=g).to(torch.float16).to(DEV)
    inv, _ = rn.rope_frequencies(16)
    axis = rn.rope_sections((3, 3, 2))
    pos = torch.tensor([[1, 2, -1, 3, 4], [1, -5, 1, 3, 4], [0, 1, 2, 3, -9]], device=DEV)
    rn.rmsnorm_device_status(clear=True)
    qo = rn.rmsnorm_rope_axes(q, None, pos, inv, axis, q_out=torch.full_like(q, 7.0))[0]
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert (qo[[1, 2, 4]] == 7).all()
    ok = torch.tensor([0, 3], device=DEV)
    w, t = turned(q, pos.clamp(min=0), axis, inv, 1.0, False)
    check("q", qo[ok], w[ok], t[ok], 16)


def test_graph_stream_and_empty():
    inv, _ = rn.rope_frequencies(16)
    axis = rn.rope_sections((4, 4))
    e = torch.zeros(0, 2, 16, dtype=torch.float16, device=DEV)
    qo, ko = rn.rmsnorm_rope_axes(e, e, torch.zeros(2, 0, dtype=torch.int64, device=DEV), inv, axis)
    assert qo.shape == e.shape and ko.shape == e.shape
    g = torch.Generator().manual_seed(11)
    q = torch.randn(64, 4, 16, generator=g).to(torch.float16).to(DEV)
    pos = torch.zeros(2, 64, dtype=torch.int64, device=DEV)
    out = torch.empty_like(q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        rn.rmsnorm_rope_axes(q, None, pos, inv, axis, q_out=out)
    for p in (3, 400):
        pos[1].fill_(p)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rn.rmsnorm_rope_axes(q, None, pos, inv, axis)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = rn.rmsnorm_rope_axes(q, None, pos, inv, axis, stream=s)[0]
    s.synchronize()
    assert torch.equal(r, out)


def test_python_refusals():
    q = torch.zeros(4, 2, 16, dtype=torch.float16, device=DEV)
    pos = torch.zeros(2, 4, dtype=torch.int64, device=DEV)
    inv, _ = rn.rope_frequencies(16)
    axis = rn.rope_sections((4, 4))
    for a in ((q, None, pos[0], inv, axis), (q, None, pos.int(), inv, axis), (q, None, pos[:, :2], inv, axis),
              (q, None, pos, inv, axis[:4]), (q, None, pos, inv, axis.long()), (q, None, pos, inv, axis.to(DEV)),
              (q, None, pos[:1], inv, axis), (q, None, pos, inv, axis - 1), (q, None, pos[:0], inv, axis),
              (q, None, torch.zeros(5, 4, dtype=torch.int64, device=DEV), inv, axis), (q, None, pos.t(), inv, axis),
              (q, None, pos.t().contiguous().t(), inv, axis), (q, q[:2], pos, inv, axis)):
        with pytest.raises(ValueError):
            rn.rmsnorm_rope_axes(*a)
    with pytest.raises(TypeError):
        rn.rmsnorm_rope_axes(q, None, pos, inv, None)
    with pytest.raises(ValueError):
        rn.rmsnorm_rope_axes(q, None, pos, inv, axis, k_out=q)


def test_written_tensors_count_as_changed():
    q, k = torch.zeros(4, 2, 16, device=DEV), torch.zeros(4, 1, 16, device=DEV)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    before = [t._version for t in (qo, ko, q)]
    rn.rmsnorm_rope_axes(q, k, torch.zeros(2, 4, dtype=torch.int64, device=DEV), rn.rope_frequencies(16)[0],
                         rn.rope_sections((4, 4)), q_out=qo, k_out=ko)
    assert [t._version for t in (qo, ko, q)] == [before[0] + 1, before[1] + 1, before[2]]


def test_forward_and_backward_captured_together():
    """Replayed with other inputs, positions and gradients."""
    g = torch.Generator().manual_seed(12)
    axis = rn.rope_sections((6, 5, 5))
    inv, _ = rn.rope_frequencies(32)
    q = torch.randn(2, 40, 3, 48, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    gq = torch.randn(2, 40, 3, 48, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 9000, (3, 2, 40), generator=g).to(DEV)

    def step():
        out = rn.rope(q, None, pos, inv, 1.0, True, axis)[0]
        return out, torch.autograd.grad(out, q, gq)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out, dq = step()
    for k in range(2):
        with torch.no_grad():
            q.mul_(-1.5)
            gq.add_(0.25)
            pos.add_(1000)
        gr.replay()
        torch.cuda.synchronize()
        check("out", out, *turned(q.detach(), pos, axis, inv, 1.0, True), 32)
        check("dq", dq, *turned(gq, pos, axis, inv, 1.0, True, -1.0), 32)
