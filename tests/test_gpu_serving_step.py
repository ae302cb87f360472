"""A serving step in 8 bits against the same step in 64: the norm's output, the rotated q, every
cached value and the attention over the contexts, in their order.

Tolerances.  The norm's codes and scales, q and the caches as in their own tests: a cached value is
half a step of its code from x (16 of the scale's 448 or 0.5 of 127 at most), 4 x 2^-24 of the
head's largest for its scale (two products and their constant, times a code of at most all of it),
and the kernel's error of x.  Read to fp32, a value is one product: 2^-24 of itself.  The attention of a query is
that of 64-bit scores off by d: q's bf16 rounding (2^-8) and angle, k's 2^-24, torch's fp32 sum of
32 products, all below (2^-8 + 1e-5) of the sum of |q| |k| / sqrt(Dh).  Its weights are off by
a factor of exp(2 d) at most, its output by (exp(2 d) - 1) max |v| and 1e-5 max |v| from fp32.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn
from test_gpu_kv_cache8 import DEV, make_cache
from test_gpu_norm_q8 import _check as check_norm
from test_gpu_rope_axes import check, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt,layout", [("e4m3", "between"), ("e4m3", "packed"), ("i8", "dense")])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("Hkv", [1, 2])
def test_a_step_against_64_bits(fmt, layout, group, Hkv):
    g = torch.Generator().manual_seed(14)
    B, W, bs, Hq, Dh = 5, 6, 8, 4, 32
    D, each = Hq * Dh, Hq // Hkv
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    kc, vc, ks, vs = make_cache(g, 40 * bs, Hkv, Dh, fmt, layout)
    lens, table = i32([0] * B), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    free, count = i32(list(range(39, -1, -1))), i32([40])
    inv, _ = rn.rope_frequencies(32)
    axis = rn.rope_sections((4, 6, 6))
    w = (torch.rand(D, generator=g) + 0.5).to(torch.bfloat16).to(DEV)
    proj = (torch.randn(D, (Hq + 2 * Hkv) * Dh, generator=g) / D ** 0.5).to(DEV)
    half_step = 16 / 448 if fmt == "e4m3" else 0.5 / 127
    seqs = [[] for _ in range(B)]  # of each request's tokens: the slot, k rotated and v in 64 bits
    for new in ([7, 3, 1, 0, 9], [1, 1, 1, 5, 1], [1, 1, 1, 1, 1]):
        T, n = sum(new) + 3, sum(new)  # padded
        plan = rn.rmsnorm_kv_plan(lens, i32(new), table, bs, T, free_blocks=free, free_count=count)
        x, res = (torch.randn(T, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        normed = rn.rmsnorm_fwd_q8(x, w, 1e-6, 0.0, res, group=group)
        check_norm(normed, x, res, w, 0.0, group)
        codes, scale, _ = normed
        values = codes.float() * (scale.repeat_interleave(group, 1) if group else scale[:, None])
        qkv = (values @ proj).to(torch.bfloat16).view(T, Hq + 2 * Hkv, Dh)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        pos = torch.stack([plan.positions, plan.positions // 4, plan.positions % 4])
        qo = rn.rmsnorm_kv_append(q, k, v, pos, plan.slots, kc, vc, inv, k_scale=ks, v_scale=vs, pair_axis=axis)
        q64, terms = turned(q[:n], pos[:, :n], axis, inv, 1.0, False)
        check("q", qo[:n], q64, terms, 32)
        k64, k_terms = turned(k, pos, axis, inv, 1.0, False)
        for t in range(n):
            seqs[plan.requests[t]].append((plan.slots[t].item(), k64[t], v[t].double(), k_terms[t]))
        ctx = rn.rmsnorm_kv_plan(torch.zeros_like(lens), lens, table, bs, int(lens.sum()) + 2, lens_out=torch.empty_like(lens))
        ko, vo = rn.rmsnorm_kv_read(kc, vc, ks, vs, ctx.slots, dtype=torch.float32)
        assert len({s for seq in seqs for s, *_ in seq}) == sum(map(len, seqs))
        cached = []  # each request's k and v as the cache holds them, 64 bits
        for b in range(B):
            lo, hi = ctx.starts[b].item(), ctx.starts[b + 1].item()
            assert hi - lo == len(seqs[b])
            at = torch.tensor([s for s, *_ in seqs[b]], dtype=torch.int64, device=DEV)
            held = [c.double()[at] * s.double()[at][..., None] for c, s in ((kc, ks), (vc, vs))]
            for got, want in zip((ko[lo:hi], vo[lo:hi]), held):
                assert ((got.double() - want).abs() <= 2.0 ** -24 * want.abs()).all()
            for i, (_, kt, vt, size) in enumerate(seqs[b]):
                for got, x64, off in ((held[0][i], kt, 8e-7 * size), (held[1][i], vt, 0 * size)):
                    top = x64.abs().amax(-1, keepdim=True)
                    assert ((got - x64).abs() <= (half_step + 4 * 2.0 ** -24) * top + 2 * off.amax(-1, keepdim=True)).all()
            cached.append(held)
        for t in range(n):
            b, p = plan.requests[t].item(), plan.positions[t].item()
            lo = ctx.starts[b].item()
            kk, vv = (c[lo:lo + p + 1].repeat_interleave(each, 1) for c in (ko, vo))
            s = torch.einsum("hd,nhd->hn", qo[t].float(), kk) / Dh ** 0.5
            y = torch.einsum("hn,nhd->hd", s.softmax(-1), vv)
            k_all, v_all = (c[:p + 1].repeat_interleave(each, 1) for c in cached[b])
            s64 = (q64[t] * k_all).sum(-1).t() / Dh ** 0.5  # [Hq, tokens]
            y64 = (s64.softmax(-1).t()[..., None] * v_all).sum(0)
            d = (2.0 ** -8 + 1e-5) * ((q64[t].abs() * k_all.abs()).sum(-1).t().amax(-1) / Dh ** 0.5)
            allow = (torch.expm1(2 * d) + 1e-5) * v_all.abs().amax(-1).amax(0)
            assert ((y.double() - y64).abs() <= allow[:, None]).all()
