"""rmsnorm_block_fwd, rmsnorm_block_vjp and block_norm against the formulas in
64 bits: row lengths on and off 16-byte boundaries from 1 to past what a CTA
holds, one row to thousands, gates of every grouping, strides, saved scales,
in place, streams, graphs, and the gradients through autograd."""
import pytest
import torch

import block_reference as ref
import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def _rand(g, rows, D, dtype, pad=0, off=0, std=1.0, mean=0.0):
    """[rows, D] with rows D + pad apart, `off` elements into its buffer."""
    buf = torch.zeros(off + rows * (D + pad) + 8, dtype=dtype)
    t = buf[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]
    t.copy_(torch.randn(rows, D, generator=g) * std + mean)
    dbuf = buf.to(DEV)
    return dbuf[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]


def _problem(rows, D, dtype, groups, post, wb, pad=0, off=0, seed=0, gate_pad=0):
    g = torch.Generator().manual_seed(1000 * seed + rows + D)
    p = dict(y=_rand(g, rows, D, dtype, pad, off), res=_rand(g, rows, D, dtype, pad, off, 2.0),
             h=_rand(g, rows, D, dtype, pad, off, 2.0), g=_rand(g, rows, D, dtype, pad, off),
             g_res=_rand(g, rows, D, dtype, pad, off),
             w_pre=_rand(g, 1, D, dtype, 0, off, 0.2, 1.0 - wb)[0],
             w_post=_rand(g, 1, D, dtype, 0, off, 0.2, 1.0 - wb)[0] if post else None,
             gate=_rand(g, groups, D, dtype, gate_pad, off, 0.5, 0.2) if groups else None, wb=wb)
    return p


def _check_fwd(p, scale, rstd=True, **kw):
    out, nr, rs = rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, p["wb"], p["gate"],
                                       scale, rstd=rstd, **kw)
    want_out, want_h, want_rs, t_out, t_h, kappa = ref.fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS,
                                                           p["wb"], p["gate"], scale)
    ref.check("new_residual", nr, want_h, t_h)
    ref.check("out", out, want_out, t_out)
    if rstd:
        ref.check("r_y", rs[0], want_rs[0], want_rs[0])
        ref.check("r_h", rs[1], want_rs[1], want_rs[1] * kappa)
    return out, nr, rs


def _check_vjp(p, scale, g_res=True, saved=False, **kw):
    gr = p["g_res"] if g_res else None
    rstd = None
    if saved:
        r = [1 / torch.sqrt((t.double() ** 2).mean(1) + EPS) for t in (p["y"], p["h"])]
        rstd = torch.stack(r).float()
    got = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, p["wb"], p["gate"],
                               scale, gr, rstd=rstd, **kw)
    want = ref.vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, p["wb"], p["gate"], scale, gr, rstd)
    rows = p["y"].shape[0]
    for name, t in zip(("g_y", "g_h", "gw_post", "gw_pre", "g_gate"), got):
        if name not in want:
            assert t is None
            continue
        k = 256.0 if name in ("g_y", "g_h") else 256.0 + 64.0 + rows / 8
        ref.check(name, t, *want[name], k=k)
    return got


SHAPES = [  # rows, D, groups, pad, off
    (1, 1, 0, 0, 0), (3, 1, 1, 2, 0), (5, 7, 5, 0, 0), (1, 64, 1, 0, 0), (1000, 64, 4, 0, 0),
    (33, 100, 3, 0, 0), (129, 128, 1, 8, 0), (64, 512, 0, 0, 0), (300, 520, 100, 0, 0),
    (17, 1000, 17, 3, 0), (700, 1024, 2, 0, 0), (37, 1030, 1, 0, 2), (4, 2048, 1, 0, 0),
    (513, 2048, 3, 0, 0), (8, 4096, 8, 0, 0), (1000, 4096, 8, 64, 0), (400, 4097, 1, 0, 0),
    (31, 4100, 31, 4, 0), (700, 4096, 7, 0, 1), (5, 8192, 5, 0, 0), (400, 8192, 2, 0, 0),
    (311, 8200, 0, 0, 0), (160, 12288, 1, 0, 0), (40, 16384, 4, 0, 0), (7, 16385, 7, 0, 0),
    (9, 20000, 3, 0, 0), (3, 40000, 1, 8, 0), (2, 131072, 2, 0, 0), (2000, 96, 1000, 0, 0),
]


@pytest.mark.parametrize("rows,D,groups,pad,off", SHAPES, ids=["r%d_d%d_g%d_p%d_o%d" % s for s in SHAPES])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_block_shapes(rows, D, groups, pad, off, dt):
    for i, (post, wb) in enumerate([(True, 0.0), (True, 1.0), (False, 0.0)]):
        p = _problem(rows, D, DT[dt], groups, post, wb, pad, off, seed=i, gate_pad=pad)
        _check_fwd(p, 0.7)
        _check_vjp(p, 0.7, g_res=i != 1, saved=i == 1)


@pytest.mark.parametrize("rows,D,groups,dt", [(16384, 4096, 8, "bf16"), (4096, 8192, 4096, "bf16"),
                                              (8192, 4096, 0, "f16"), (6000, 2049, 6, "bf16"),
                                              (5000, 2048, 2500, "f32"), (16384, 512, 2, "f16")])
def test_block_many_rows(rows, D, groups, dt):
    p = _problem(rows, D, DT[dt], groups, True, 0.0)
    _check_fwd(p, 1.0)
    a = _check_vjp(p, 1.0, saved=True)
    b = _check_vjp(p, 1.0, saved=True)
    for s, t in zip(a, b):  # the same bits on every run
        if s is not None:
            assert torch.equal(s, t)


@pytest.mark.parametrize("D", [512, 4096, 4099, 20000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_block_near_cancellation(D, dt):
    """The block nearly undoes the residual stream, so h is much smaller than
    its terms: its scale must come from h itself."""
    p = _problem(24, D, DT[dt], 1, True, 0.0, seed=5)
    _, h, _, _, _, _ = ref.fwd(p["y"], torch.zeros_like(p["y"]), p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 1.0)
    step = 1e-3 if dt == "f32" else 0.05
    noise = torch.randn(24, D, generator=torch.Generator().manual_seed(1)).to(DEV)
    p["res"] = (-h * (1 + step * noise)).to(DT[dt])
    _check_fwd(p, 1.0)


@pytest.mark.parametrize("D", [512, 4096, 4097, 8192])
def test_block_rows_do_not_leak(D):
    """Rows of zeros, of infinities and of NaN leave the others' bits alone,
    and zero rows give finite results."""
    p = _problem(300, D, torch.bfloat16, 3, True, 0.0, seed=2)
    out, nr, _ = rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5)
    q = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in p.items()}
    q["y"][7], q["res"][7] = 0, 0
    q["y"][100], q["res"][200], q["y"][299] = float("inf"), float("nan"), float("nan")
    out2, nr2, _ = rn.rmsnorm_block_fwd(q["y"], q["res"], q["w_post"], q["w_pre"], EPS, 0.0, q["gate"], 0.5)
    keep = [i for i in range(300) if i not in (7, 100, 200, 299)]
    assert torch.equal(out[keep], out2[keep]) and torch.equal(nr[keep], nr2[keep])
    assert (out2[7] == 0).all() and (nr2[7] == 0).all()
    assert torch.isnan(out2[200]).all() and torch.isnan(out2[299]).all()
    a = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, p["g_res"])
    q["h"][200], q["g"][100] = float("nan"), float("inf")
    q["y"][100], q["y"][299] = p["y"][100], p["y"][299]
    b = rn.rmsnorm_block_vjp(q["y"], q["h"], q["w_post"], q["w_pre"], q["g"], EPS, 0.0, q["gate"], 0.5, q["g_res"])
    keep = [i for i in range(300) if i not in (7, 100, 200)]
    for s, t in zip(a[:2], b[:2]):
        assert torch.equal(s[keep], t[keep])
    # row 7 (y = 0) has the right gradients and row 200 poisons the weights' sums
    assert torch.isfinite(b[0][7]).all() and torch.isnan(b[3]).any()


def test_block_in_place_and_buffers():
    for D in (4096, 4097, 20000):
        p = _problem(50, D, torch.bfloat16, 5, True, 0.0)
        want = rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5)
        y, r = p["y"].clone(), p["res"].clone()
        out, nr, _ = rn.rmsnorm_block_fwd(y, r, p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5, out=y,
                                          new_residual=r)
        assert out is y and nr is r and torch.equal(y, want[0]) and torch.equal(r, want[1])
        want = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5,
                                    p["g_res"])
        y, gr = p["y"].clone(), p["g_res"].clone()
        got = rn.rmsnorm_block_vjp(y, p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, gr,
                                   g_y=y, g_h=gr)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D,pad", [(512, 8), (4096, 64), (1001, 3), (20000, 16)])
def test_block_leaves_the_rest_of_its_buffers_alone(D, pad):
    """Padding between rows, rows behind the last and the bytes around the
    fp32 outputs keep what they held."""
    rows, dt = 37, torch.float16
    p = _problem(rows, D, dt, 1, True, 0.0, pad=pad)
    def guarded():
        buf = torch.full((rows + 2, D + pad), 7.0, dtype=dt, device=DEV)
        return buf, buf[1:rows + 1, :D]
    bo, out = guarded()
    bn, nr = guarded()
    rs = torch.full((4, rows), 7.0, device=DEV)
    rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5, out=out,
                         new_residual=nr, rstd=rs[1:3])
    want = ref.fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5)
    ref.check("out", out, want[0], want[3])
    for b in (bo, bn):
        assert (b[0] == 7).all() and (b[-1] == 7).all() and (b[:, D:] == 7).all()
    assert (rs[0] == 7).all() and (rs[3] == 7).all()
    by, gy = guarded()
    bh, gh = guarded()
    g32 = torch.full((9, D), 7.0, device=DEV)
    rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, p["g_res"],
                         g_y=gy, g_h=gh, gw_post=g32[1], gw_pre=g32[3], g_gate=g32[5:6])
    for b in (by, bh):
        assert (b[0] == 7).all() and (b[-1] == 7).all() and (b[:, D:] == 7).all()
    for i in (0, 2, 4, 6):
        assert (g32[i] == 7).all()


def test_block_leading_dims_and_gate_shapes():
    B, S, D = 3, 50, 1024
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    y, res, wq, wp, mod = mk(B, S, D), mk(B, S, D), mk(D), mk(D), mk(B, 6 * D)
    gate = mod[:, 2 * D:3 * D]
    a = rn.rmsnorm_block_fwd(y, res, wq, wp, EPS, 0.0, gate, rstd=True)
    b = rn.rmsnorm_block_fwd(y.view(-1, D), res.view(-1, D), wq, wp, EPS, 0.0,
                             gate.contiguous().repeat_interleave(S, 0))
    assert a[0].shape == y.shape and a[2].shape == (2, B, S)
    assert torch.equal(a[0].view(-1, D), b[0]) and torch.equal(a[1].view(-1, D), b[1])
    c = rn.rmsnorm_block_fwd(y, res, wq, wp, EPS, 0.0, gate[0])
    d = rn.rmsnorm_block_fwd(y, res, wq, wp, EPS, 0.0, gate[:1].expand(3, D).contiguous().view(3, 1, D))
    assert torch.equal(c[0], d[0])


def test_block_no_rows():
    for G, shape in ((0, (0, 64)), (2, (2, 0, 64))):
        y = torch.zeros(shape, dtype=torch.float16, device=DEV)
        w = torch.ones(64, dtype=torch.float16, device=DEV)
        gate = torch.ones(G, 64, dtype=torch.float16, device=DEV) if G else None
        out, nr, rs = rn.rmsnorm_block_fwd(y, y, w, w, EPS, 0.0, gate, rstd=True)
        assert out.shape == shape and rs.numel() == 0
        got = rn.rmsnorm_block_vjp(y, y, w, w, y, EPS, 0.0, gate)
        assert (got[2] == 0).all() and (got[3] == 0).all()
        if G:
            assert got[4].shape == (2, 64) and (got[4] == 0).all()


def test_block_side_stream_and_graph():
    p = _problem(256, 4096, torch.bfloat16, 4, True, 0.0)
    args = (p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.5)
    vargs = (p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, p["g_res"])
    want, vwant = rn.rmsnorm_block_fwd(*args, rstd=True), rn.rmsnorm_block_vjp(*vargs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, vgot = rn.rmsnorm_block_fwd(*args, rstd=True, stream=s), rn.rmsnorm_block_vjp(*vargs, stream=s)
    s.synchronize()
    for a, b in zip(got + vgot, want + vwant):
        assert torch.equal(a, b)
    # two graphs of the same problem, replayed in turn and at once on two streams
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(rn.rmsnorm_block_fwd(*args, rstd=True) + rn.rmsnorm_block_vjp(*vargs))
        graphs.append(gr)
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(3.0)
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(o, want + vwant):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gate_shape", [None, (256,), (2, 256), (2, 1, 256), (2, 40, 256)])
def test_block_norm_autograd(dt, gate_shape):
    """Gradients through autograd against the same graph in 64 bits, a strided
    y and an expanded gradient among the layouts."""
    dtype, D = DT[dt], 256
    g = torch.Generator().manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)  # noqa: E731
    wide = mk(2, 40, 2 * D)
    y, res, wq, wp = wide[..., :D], mk(2, 40, D), mk(D), mk(D)
    gate = None if gate_shape is None else mk(*gate_shape)
    leaves = [t.detach().requires_grad_() for t in (y, res, wq, wp) + (() if gate is None else (gate,))]
    out, nr = rn.block_norm(leaves[0], leaves[1], leaves[2], leaves[3], EPS, 0.0,
                            leaves[4] if gate is not None else None, 0.7)
    go = mk(1, 1, D).expand(2, 40, D)
    gn = mk(2, 40, D)
    grads = torch.autograd.grad([out, nr], leaves, [go, gn])
    p = dict(y=y.reshape(80, D), h=nr.detach().view(80, D), g=go.reshape(80, D), g_res=gn.view(80, D))
    want = ref.vjp(p["y"], p["h"], wq, wp, p["g"], EPS, 0.0, gate, 0.7, p["g_res"])
    names = ["g_y", "g_h", "gw_post", "gw_pre", "g_gate"]
    for n, t, leaf in zip(names, grads, leaves):
        assert t.shape == leaf.shape and t.dtype == leaf.dtype
        # the saved scales come from the unrounded h: an eps / 2 error of each of h's elements
        # and of each scale enters the terms
        k = 400.0 + 4 * torch.finfo(dtype).eps / ref.U
        ref.check(n, t.reshape(want[n][0].shape), *want[n], k=k)
    # only one of the outputs used
    only = torch.autograd.grad(rn.block_norm(leaves[0], leaves[1], leaves[2], leaves[3], EPS, 0.0,
                                             leaves[4] if gate is not None else None, 0.7)[1].float().sum(),
                               leaves[1])[0]
    assert (only == 1).all()
    with pytest.raises(RuntimeError):
        o, _ = rn.block_norm(leaves[0], leaves[1], leaves[2], leaves[3], EPS)
        g1 = torch.autograd.grad(o.float().square().sum(), leaves[1], create_graph=True)[0]
        torch.autograd.grad(g1.sum(), leaves[1])


def test_block_vjp_against_differences():
    """fp32 gradients against central differences of the 64-bit forward."""
    rows, D = 6, 40
    p = _problem(rows, D, torch.float32, 2, True, 0.0, seed=9)
    _, nr, rs = rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], 0.7,
                                     rstd=True)
    got = rn.rmsnorm_block_vjp(p["y"], nr, p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.7, p["g_res"],
                               rstd=rs)
    x = {k: p[k].double() for k in ("y", "res", "w_post", "w_pre", "gate")}

    def loss():
        o, h = ref.fwd(x["y"], x["res"], x["w_post"], x["w_pre"], EPS, 0.0, x["gate"], 0.7)[:2]
        return (o * p["g"].double()).sum() + (h * p["g_res"].double()).sum()
    d = 1e-5
    for name, t in zip(("y", "res", "w_post", "w_pre", "gate"), got):
        flat, worst, size = x[name].view(-1), 0.0, t.abs().max().item()
        for i in range(0, flat.numel(), 7):
            keep = flat[i].item()
            flat[i] = keep + d
            up = loss()
            flat[i] = keep - d
            down = loss()
            flat[i] = keep
            worst = max(worst, abs(((up - down) / (2 * d)).item() - t.reshape(-1)[i].item()))
        # differences: d^2 of third derivatives (below 1e2 here) and 1e-16 * 1e2 / d of rounding;
        # the kernel: 256 u of terms that are at most 10 times the largest gradient
        assert worst <= 1e-8 + 1e-9 + 10 * 256 * ref.U * size, (name, worst)


def test_block_refusals():
    y = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    bad = [
        dict(residual=y.float()), dict(residual=y[:4]), dict(w_pre=w[:32]), dict(w_post=w.float()),
        dict(gate=torch.ones(3, 64, dtype=torch.bfloat16, device=DEV)), dict(gate=w[:32]),
        dict(gate=w.float()), dict(gate=w[:1].expand(64)), dict(gate=w.view(1, 64).expand(8, 64)),
        dict(rstd=torch.zeros(8, device=DEV)), dict(out=y.t()), dict(y=y.cpu()),
        dict(residual=y[:1].expand(8, 64)),
    ]
    for kw in bad:
        a = dict(y=y, residual=y.clone(), w_post=w, w_pre=w, gate=None)
        extra = {k: kw[k] for k in kw if k not in a}
        a.update({k: v for k, v in kw.items() if k in a})
        with pytest.raises(ValueError):
            rn.rmsnorm_block_fwd(a["y"], a["residual"], a["w_post"], a["w_pre"], EPS, 0.0, a["gate"], **extra)
    with pytest.raises(TypeError):
        rn.rmsnorm_block_fwd(y.double(), y.double(), w.double(), w.double(), EPS)
    for kw in (dict(out=y[:, :]), ):
        with pytest.raises(rn.RmsnormError):  # out is y, new_residual is y too
            rn.rmsnorm_block_fwd(y, y, w, w, EPS, out=y, new_residual=y)
    for eps, wb, scale in ((-1.0, 0.0, 1.0), (EPS, float("nan"), 1.0), (EPS, 0.0, float("inf"))):
        with pytest.raises(rn.RmsnormError):
            rn.rmsnorm_block_fwd(y, y.clone(), w, w, eps, wb, None, scale)
    with pytest.raises(ValueError):
        rn.rmsnorm_block_vjp(y, y, None, w, y, EPS, gw_post=torch.zeros(64, device=DEV))
    with pytest.raises(ValueError):
        rn.rmsnorm_block_vjp(y, y, w, w, y, EPS, g_gate=torch.zeros(64, device=DEV))
    g32 = torch.zeros(64, device=DEV)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_block_vjp(y, y, w, w, y, EPS, gw_post=g32, gw_pre=g32)


def test_block_vjp_scratch():
    """The C entry points with pooled and with the caller's scratch give the same
    bits; a failed allocation and a bad workspace leave the outputs alone."""
    lib, rows, D = rn._native.lib(), 300, 512
    p = _problem(rows, D, torch.bfloat16, 3, True, 0.0)
    want = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, p["g_res"])

    def call(fn, *tail):
        out = [torch.full_like(t, 5.0) for t in want]
        st = fn(p["y"].data_ptr(), D, p["h"].data_ptr(), D, p["w_post"].data_ptr(), p["w_pre"].data_ptr(),
                p["gate"].data_ptr(), D, 3, 0.5, p["g"].data_ptr(), D, p["g_res"].data_ptr(), D, None, EPS, 0.0,
                out[0].data_ptr(), D, out[1].data_ptr(), D, out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(),
                rows, D, 1, *tail, torch.cuda.current_stream().cuda_stream)
        return st, out
    n = lib.rmsnorm_block_vjp_workspace_size(rows, D, 1)
    ws = torch.full((n + 512,), 255, dtype=torch.uint8, device=DEV)
    at = ws.data_ptr() + (-ws.data_ptr()) % 256
    for st, out in (call(lib.rmsnorm_block_vjp), call(lib.rmsnorm_block_vjp_ws, at, n)):
        assert st == 0
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    assert (ws[at - ws.data_ptr() + n:] == 255).all()
    rn.rmsnorm_debug_fail_allocs(1)
    for st, out in (call(lib.rmsnorm_block_vjp), call(lib.rmsnorm_block_vjp_ws, at, n - 1),
                    call(lib.rmsnorm_block_vjp_ws, None, n), call(lib.rmsnorm_block_vjp_ws, at + 16, n),
                    call(lib.rmsnorm_block_vjp_ws, p["y"].data_ptr(), rows * D * 2 + n)):
        assert st in (1, 4) and all((t == 5).all() for t in out)
    assert lib.rmsnorm_block_vjp_workspace_size(0, D, 1) == 0 == lib.rmsnorm_block_vjp_workspace_size(4, 0, 1)


@pytest.mark.parametrize("rows,D,groups,pad,off", [(400, 5120, 0, 0, 0), (400, 5120, 400, 0, 0), (333, 5000, 3, 4, 0),
                                                   (305, 5120, 5, 0, 1), (400, 10240, 4, 0, 0), (310, 10250, 310, 0, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_block_wide_ctas(rows, D, groups, pad, off, dt):
    """Rows whose CTAs are just past half or all of an SM's threads."""
    for saved in (False, True):
        p = _problem(rows, D, DT[dt], groups, True, 0.0, pad, off, seed=11 + saved)
        _check_fwd(p, 0.9)
        _check_vjp(p, 0.9, saved=saved)


@pytest.mark.parametrize("rows,D,groups,pad,off", [
    (1300, 1000, 0, 1, 0), (1300, 1025, 5, 0, 3), (2600, 515, 1, 0, 0), (700, 2049, 700, 0, 5), (650, 4098, 10, 0, 2),
    (320, 4104, 2, 0, 0), (320, 4130, 320, 0, 0), (3, 4097, 3, 0, 7), (1, 2050, 0, 0, 1), (330, 8191, 3, 0, 0),
    (310, 10241, 1, 0, 0), (400, 5127, 2, 0, 0), (2500, 1028, 4, 4, 1), (307, 16383, 1, 0, 0), (340, 4090, 0, 6, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_block_rows_off_boundaries(rows, D, groups, pad, off, dt):
    """Rows that all stand alike to 16-byte boundaries, at every distance from one, in
    one or several kinds; and with one tensor standing differently."""
    for i, (post, wb) in enumerate([(True, 0.0), (True, 1.0), (False, 0.0)]):
        p = _problem(rows, D, DT[dt], groups, post, wb, pad, off, seed=31 + i, gate_pad=pad)
        _check_fwd(p, 0.8)
        a = _check_vjp(p, 0.8, g_res=i != 1, saved=i != 1)
        p["y"] = _rand(torch.Generator().manual_seed(i), rows, D, DT[dt], pad + 1, off)
        _check_fwd(p, 0.8)
        _check_vjp(p, 0.8, g_res=i != 1, saved=i != 1)
        del a


def test_block_rows_off_boundaries_leave_their_neighbours_alone():
    """Cut units at a row's ends: what lies between and around the rows stays, whatever
    stands there."""
    rows, D, ld, off = 640, 2043, 2051, 5
    p = _problem(rows, D, torch.bfloat16, 4, True, 0.0, 8, off, seed=41)

    def put(t, fill):
        buf = torch.full((off + rows * ld + 16,), fill, dtype=t.dtype, device=DEV)
        v = buf[off:off + rows * ld].view(rows, ld)[:, :D]
        v.copy_(t)
        return buf, v

    def both(fill):  # the inputs in buffers of `fill`: the same path, so the same bits
        q = {k: put(p[k], fill)[1] for k in ("y", "res", "h", "g", "g_res")}
        outs = [put(torch.zeros_like(p["y"]), 7.0) for _ in range(4)]
        rn.rmsnorm_block_fwd(q["y"], q["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], out=outs[0][1], new_residual=outs[1][1])
        got = rn.rmsnorm_block_vjp(q["y"], q["h"], p["w_post"], p["w_pre"], q["g"], EPS, 0.0, p["gate"], 1.0, q["g_res"],
                                   g_y=outs[2][1], g_h=outs[3][1])
        return outs, [o[1] for o in outs] + list(got[2:])

    keep = torch.ones(off + rows * ld + 16, dtype=torch.bool)
    keep[off:off + rows * ld].view(rows, ld)[:, :D] = False
    (outs, got), (_, want) = both(float("nan")), both(0.0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for buf, _ in outs:
        assert (buf.cpu()[keep] == 7.0).all()


@pytest.mark.parametrize("rows,D,groups,pad,off", [
    (1, 64, 0, 0, 0), (8, 100, 1, 0, 1), (9, 512, 0, 0, 0), (16, 37, 16, 0, 0), (17, 200, 1, 8, 0), (33, 256, 33, 0, 0),
    (61, 511, 1, 0, 0), (64, 512, 0, 0, 0), (64, 128, 2, 0, 0), (65, 512, 1, 0, 0), (2, 5248, 0, 8, 0), (8, 4096, 4, 0, 0),
    (6, 1000, 2, 0, 0), (7, 4097, 7, 0, 0), (8, 8191, 8, 0, 3), (16, 4096, 1, 0, 0), (13, 2048, 0, 0, 0), (11, 4104, 11, 0, 0),
    (16, 4097, 1, 7, 0), (15, 1001, 1, 0, 0), (16, 16384, 1, 0, 0), (12, 2000, 3, 0, 0), (4, 10000, 2, 0, 0), (120, 5248, 3, 0, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_block_few_rows(rows, D, groups, pad, off, dt):
    """Up to 64 rows, on both sides of what one cluster sums by itself."""
    for i, (post, wb) in enumerate([(True, 0.0), (True, 1.0), (False, 0.0)]):
        p = _problem(rows, D, DT[dt], groups, post, wb, pad, off, seed=61 + i, gate_pad=pad)
        a = _check_vjp(p, 0.8, g_res=i != 1, saved=i != 1)
        for _ in range(3):  # the same bits on every run
            b = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, wb, p["gate"], 0.8,
                                     p["g_res"] if i != 1 else None,
                                     rstd=None if i == 1 else torch.stack([1 / torch.sqrt((t.double() ** 2).mean(1) + EPS)
                                                                          for t in (p["y"], p["h"])]).float())
            for s, t in zip(a, b):
                assert (s is None and t is None) or torch.equal(s, t)


@pytest.mark.parametrize("D", [384, 4096, 4099, 20000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("y_std,gate_std,res_std", [(1e12, 1e12, 1e12), (1e-15, 1e-10, 1e-10), (1e-15, 1e-10, 0.0)])
def test_block_fwd_terms_past_fp32(D, dt, y_std, gate_std, res_std):
    """Rows whose norms are in fp32's range while the square of gate * y is not: it
    overflows, or (with no epsilon to hide it) vanishes."""
    g = torch.Generator().manual_seed(D)
    rows = 330
    y, res = (_rand(g, rows, D, DT[dt], std=s) for s in (y_std, res_std))
    gate = _rand(g, 1, D, DT[dt], std=gate_std)
    w_post, w_pre = (_rand(g, 1, D, DT[dt], std=0.2, mean=1.0)[0] for _ in range(2))
    out, h, _ = rn.rmsnorm_block_fwd(y, res, w_post, w_pre, 0.0, 0.0, gate)
    want_out, want_h, _, t_out, t_h, _ = ref.fwd(y, res, w_post, w_pre, 0.0, 0.0, gate, 1.0)
    ref.check("new_residual", h, want_h, t_h)
    ref.check("out", out, want_out, t_out)


def test_block_wait_timeout_is_reported_and_context_survives():
    """A row whose copies are never issued: the wait ends, the status says so, and
    the next calls are right."""
    p = _problem(2000, 4096, torch.bfloat16, 4, True, 0.0, seed=3)
    rn.rmsnorm_device_status(clear=True)
    for backward in (False, True):
        rn.rmsnorm_debug_inject(drop_tile=1501, budget_cycles=2_000_000)
        try:
            if backward:
                rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 1.0, p["g_res"])
            else:
                rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"])
            bits = rn.rmsnorm_device_status(clear=True)
        finally:
            rn.rmsnorm_debug_inject(-1, 0)
        assert bits & rn.DEVSTATUS_WAIT_TIMEOUT
        _check_fwd(p, 1.0)
        _check_vjp(p, 1.0)
        assert rn.rmsnorm_device_status(clear=True) == 0


def test_block_calls_of_two_threads():
    """Two host threads, each with its own stream and problem, at once."""
    import threading
    problems = [_problem(3000, 4096, torch.bfloat16, 5, True, 0.0, seed=21), _problem(2000, 1024, torch.float16, 200, True, 0.0, seed=22)]

    def both(p):
        return rn.rmsnorm_block_fwd(p["y"], p["res"], p["w_post"], p["w_pre"], EPS, 0.0, p["gate"], rstd=True) + \
            rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 1.0, p["g_res"])

    want = [both(p) for p in problems]
    torch.cuda.synchronize()
    same = [True, True]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = both(problems[i])
                same[i] = same[i] and all(torch.equal(a, b) for a, b in zip(got, want[i]))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True, True]


@pytest.mark.parametrize("rows,D,groups", [(1000, 4096, 8), (1400, 1024, 2), (400, 5120, 0), (320, 8192, 320), (3000, 512, 1),
                                           (700, 2041, 7), (330, 12288, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_block_vjp_forms(rows, D, groups, dt):
    """With and without a norm after the block, the gradient of new_residual and saved
    scales, on the tiers that are compiled for some of these."""
    for post in (True, False):
        p = _problem(rows, D, DT[dt], groups, post, 0.0, seed=81)
        for g_res in (True, False):
            for saved in (True, False):
                _check_vjp(p, 1.1, g_res=g_res, saved=saved)


@pytest.mark.parametrize("rows,D,groups", [(5, 4096, 5), (60, 384, 1), (650, 2043, 2), (40, 20000, 4)])
def test_block_replays_with_new_inputs(rows, D, groups):
    """A captured call reads what its buffers hold when it is replayed: on the
    cluster, off-boundary and long-row paths."""
    p, fresh = (_problem(rows, D, torch.bfloat16, groups, True, 0.0, seed=s) for s in (91, 92))

    def both(q):
        return rn.rmsnorm_block_fwd(q["y"], q["res"], q["w_post"], q["w_pre"], EPS, 0.0, q["gate"], 0.6, rstd=True) + \
            rn.rmsnorm_block_vjp(q["y"], q["h"], q["w_post"], q["w_pre"], q["g"], EPS, 0.0, q["gate"], 0.6, q["g_res"])

    want = [both(fresh), both(p)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(p)
    old = {k: v.clone() for k, v in p.items() if torch.is_tensor(v)}
    for source, expected in ((fresh, want[0]), (old, want[1])):
        for k in old:
            p[k].copy_(source[k])
        for _ in range(2):
            for t in got:
                t.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, expected):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dt,widths", [("f32", (4428, 5760, 6400, 6393)), ("bf16", (9600, 11520, 14400, 14377, 10457, 11505))])
def test_block_rings_that_fill_shared_memory(dt, widths):
    """Widths whose ring, table and sums come within bytes of what a CTA may have, with
    more rows than SMs and with every number of row tensors in the ring."""
    for D in widths:
        for groups in (1, 400):
            p = _problem(400, D, DT[dt], groups, True, 0.0, seed=101)
            _check_fwd(p, 0.9)
            for g_res in (True, False):
                _check_vjp(p, 0.9, g_res=g_res, saved=g_res)


@pytest.mark.parametrize("rows,D,groups", [(8, 512, 1), (330, 384, 330), (330, 4096, 3), (330, 4099, 1), (330, 5120, 0), (6, 4096, 6),
                                           (24, 20000, 2)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tiny", ["y", "h"])
def test_block_vjp_of_rows_whose_scale_squared_leaves_fp32(rows, D, groups, dt, tiny):
    """Without an epsilon, rows of 3e-20 have a scale near 3e19, whose square is past
    fp32 while every gradient is in it.  The mean of their squares, 9e-40, is a subnormal:
    a sum and its mean are off by 2^-150 / 2^-130 = 16 u more each, beside the 64 u of a
    sum, so k is 256 * 96 / 64."""
    for post in (True, False):
        for saved in (True, False):
            p = _problem(rows, D, DT[dt], groups, post, 0.0, seed=111)
            p[tiny] = _rand(torch.Generator().manual_seed(5), rows, D, DT[dt], std=3e-20)
            r = [1 / torch.sqrt((t.double() ** 2).mean(1)) for t in (p["y"], p["h"])]
            rstd = torch.stack(r).float() if saved else None
            got = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], 0.0, 0.0, p["gate"], 0.7,
                                       p["g_res"], rstd=rstd)
            want = ref.vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], 0.0, 0.0, p["gate"], 0.7, p["g_res"], rstd)
            for name, t in zip(("g_y", "g_h", "gw_post", "gw_pre", "g_gate"), got):
                if name in want:
                    ref.check(name, t, *want[name], k=384.0 if name in ("g_y", "g_h") else 384.0 + 64.0 + rows / 8)


def test_block_no_rows_and_a_gate_for_each():
    """An empty batch with a gate row per row: no gate rows."""
    for shape in ((0, 64), (2, 0, 64)):
        y = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
        out, nr, _ = rn.rmsnorm_block_fwd(y, y, w, w, EPS, 0.0, y)
        assert out.shape == shape and nr.shape == shape
        got = rn.rmsnorm_block_vjp(y, y, w, w, y, EPS, 0.0, y)
        assert got[4].shape == shape and got[4].dtype == torch.float32
        assert (got[2] == 0).all() and (got[3] == 0).all()
        leaves = [t.clone().requires_grad_() for t in (y, y, w, w, y)]
        out, nr = rn.block_norm(leaves[0], leaves[1], leaves[2], leaves[3], EPS, 0.0, leaves[4])
        grads = torch.autograd.grad([out, nr], leaves, [y, y])
        assert grads[4].shape == shape and (grads[2] == 0).all()
    full = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        rn.rmsnorm_block_fwd(full, full.clone(), w, w, EPS, 0.0, full[:0])


def test_gradients_of_no_rows_through_a_sum():
    """The gradient of a sum is an expanded scalar; with no rows torch counts it as
    contiguous whatever its strides."""
    y, res, gate = (torch.zeros(2, 0, 64, dtype=torch.bfloat16, device=DEV).requires_grad_() for _ in range(3))
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV).requires_grad_()
    for call in (lambda: rn.block_norm(y, res, w, w, EPS, 0.0, gate), lambda: rn.block_norm(y, res, None, w, EPS),
                 lambda: rn.fused_add_rmsnorm(y, res, w, EPS), lambda: (rn.rms_norm(y, w, EPS),)):
        w.grad = None
        sum(t.sum() for t in call()).backward()
        assert (w.grad == 0).all()
    q = torch.zeros(0, 4, 16, dtype=torch.bfloat16, device=DEV).requires_grad_()
    inv, _ = rn.rope_frequencies(8)
    turned, _ = rn.rope(q, None, torch.zeros(0, dtype=torch.int64, device=DEV), inv)
    turned.sum().backward()
    assert q.grad.shape == q.shape


@pytest.mark.parametrize("rows,D,G", [(256, 515, 128), (600, 512, 300), (4096, 96, 2048), (255, 520, 51)])
def test_block_vjp_workspace_holds_the_slices_of_many_gate_rows(rows, D, G):
    """A workspace of just the size asked, with what follows it untouched."""
    lib = rn._native.lib()
    p = _problem(rows, D, torch.float16, G, True, 0.0, seed=121)
    want = rn.rmsnorm_block_vjp(p["y"], p["h"], p["w_post"], p["w_pre"], p["g"], EPS, 0.0, p["gate"], 0.5, p["g_res"])
    n = lib.rmsnorm_block_vjp_workspace_size(rows, D, 0)
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device=DEV)
    at = ws.data_ptr() + (-ws.data_ptr()) % 256
    out = [torch.full_like(t, 5.0) for t in want]
    st = lib.rmsnorm_block_vjp_ws(
        p["y"].data_ptr(), D, p["h"].data_ptr(), D, p["w_post"].data_ptr(), p["w_pre"].data_ptr(), p["gate"].data_ptr(), D, G,
        0.5, p["g"].data_ptr(), D, p["g_res"].data_ptr(), D, None, EPS, 0.0, out[0].data_ptr(), D, out[1].data_ptr(), D,
        out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), rows, D, 0, at, n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    assert (ws[at - ws.data_ptr() + n:] == 255).all()


@pytest.mark.parametrize("rows,D", [(3000, 512), (1400, 1024), (700, 4096), (400, 5120), (330, 8192)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_block_vjp_forms_with_a_gate_row_per_row(rows, D, dt):
    """Every combination of operands, on each tier that is compiled for some of them."""
    for post in (True, False):
        p = _problem(rows, D, DT[dt], rows, post, 0.0, seed=131)
        for g_res in (True, False):
            for saved in (True, False):
                _check_vjp(p, 0.9, g_res=g_res, saved=saved)


@pytest.mark.parametrize("rows,D,groups,dt", [(8, 16384, 8, "bf16"), (8, 16384, 4, "f16"), (8, 16384, 1, "bf16"), (8, 8192, 2, "f32"),
                                              (5, 16383, 5, "bf16"), (153, 16384, 0, "bf16"), (153, 8192, 153, "f32"),
                                              (2560, 4097, 40, "bf16"), (2432, 4097, 38, "bf16"), (640, 8191, 20, "bf16")])
def test_block_vjp_at_the_ends_of_its_tiers(rows, D, groups, dt):
    """The widest rows in a cluster and just past the SMs' count, and the most gate rows off
    16-byte boundaries that keep 16-byte units, with one more."""
    for post in (True, False):
        p = _problem(rows, D, DT[dt], groups, post, 0.0, seed=141)
        for g_res in (True, False):
            _check_vjp(p, 0.9, g_res=g_res, saved=not g_res)
