"""rmsnorm_fwd_q8 against its definition in 64 bits: every tier, ragged groups, strides,
rows off 16-byte boundaries, long rows, in place, values that are not numbers.

Tolerances.  v = h w' is off by 3 u (u = 2^-24: h, w' and the product, each rounded), its
group's a by as much, 448 / a and the last product by u each: a code's argument by 8 u of
itself.  A scale is a r / 448: 3 u from a, 3 u from its products and the constant, and r's:
half the sum of squares' (5 u a term, at most 64 + D / 32768 terms one behind the other and
10 steps of trees, u each) and 4 u from rsqrtf: (64 + D / 65536) u covers them.
"""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn
from q8_reference import FLOOR, U, check_codes, grouped

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def _want(x, res, w, wb, group, eps=EPS):
    """(v / unit, scale) in 64 bits, [rows, groups, ...] and [rows, groups]."""
    h = x.double() + (0 if res is None else res.double())
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    v = grouped(h * (wb + w.double()), group)
    unit = (v.abs().amax(-1) / 448).clamp(min=FLOOR)
    return v / unit[..., None], unit * r


def _check(got, x, res, w, wb, group, eps=EPS):
    out, scale, nr = got
    D = x.shape[-1]
    t, s = _want(x.reshape(-1, D), None if res is None else res.reshape(-1, D), w, wb, group, eps)
    assert out.dtype == E4M3 and out.shape == x.shape and scale.dtype == torch.float32
    assert scale.shape == x.shape[:-1] + ((s.shape[-1],) if group else ())
    assert ((scale.double().reshape(s.shape) - s).abs() <= (64 + D / 65536) * U * s).all()
    check_codes("codes", grouped(out.reshape(-1, D).float(), group).to(E4M3), t, 8 * U * t.abs())
    if res is None:
        assert nr is None
    else:
        assert torch.equal(nr, (x.float() + res.float()).to(x.dtype))


def _rows(g, rows, D, dtype, pad=0, off=0, std=1.0):
    buf = torch.full((rows * (D + pad) + off,), 7.0, dtype=dtype, device=DEV)
    v = buf[off:].view(rows, D + pad)[:, :D]
    v.copy_(std * torch.randn(rows, D, generator=g) * torch.exp(torch.randn(rows, 1, generator=g)))
    return v


SHAPES = [(1, 1), (3, 7), (5, 33), (1, 64), (4, 128), (9, 200), (700, 256), (65, 257), (1000, 512), (3, 1000),
          (33, 1024), (2000, 1024), (4, 4096), (400, 4096), (200, 4104), (300, 4097), (37, 8192), (500, 8192),
          (6, 12288), (400, 16384), (3, 16392), (170, 20001), (2, 40000), (1, 1 << 20),
          # rings, aligned and not, with whole and ragged last units, groups and warps
          (1300, 2048), (1301, 2200), (900, 2049), (700, 4096), (1500, 4097), (3000, 1001), (5000, 263), (470, 5121),
          (310, 8200), (320, 16385), (330, 12296)]


@pytest.mark.parametrize("rows,D", SHAPES, ids=["%dx%d" % s for s in SHAPES])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_shapes(rows, D, group, dt):
    g = torch.Generator().manual_seed(rows + D + group)
    x, res = _rows(g, rows, D, DT[dt]), _rows(g, rows, D, DT[dt], std=2.0)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(DT[dt]).to(DEV)
    _check(rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group), x, res, w, 0.0, group)
    _check(rn.rmsnorm_fwd_q8(x, w - 1, EPS, 1.0, group=group), x, None, w - 1, 1.0, group)


@pytest.mark.parametrize("rows,D", [(50, 96), (40, 1000), (333, 2048), (170, 4096), (300, 4097), (5, 8192), (7, 16384),
                                    (1300, 2048), (640, 4104), (2, 20000)])
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("pads", [(0, 8, 16, 16), (8, 8, 8, 8), (1, 3, 1, 5), (64, 0, 0, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_strides_and_offsets(rows, D, group, pads, dt):
    """Every tensor with a padding and a start of its own; the padding stays as it was."""
    g = torch.Generator().manual_seed(D + group)
    px, pr, pn, po = pads
    x, res = _rows(g, rows, D, DT[dt], px), _rows(g, rows, D, DT[dt], pr, off=pr % 8)
    nr = _rows(g, rows, D, DT[dt], pn, off=pn)
    obuf = torch.full((rows * (D + po) + po + 3,), 77, dtype=torch.uint8, device=DEV)
    out = obuf[po:po + rows * (D + po)].view(rows, D + po)[:, :D].view(E4M3)
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(DT[dt]).to(DEV)
    got = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group, out=out, new_residual=nr)
    assert got[0] is out or got[0].data_ptr() == out.data_ptr()
    _check(got, x, res, w, 0.0, group)
    assert (obuf[:po] == 77).all() and (obuf[po + rows * (D + po):] == 77).all()
    if po:
        assert (obuf[po:po + rows * (D + po)].view(rows, D + po)[:, D:] == 77).all()
    if pn:
        whole = nr.as_strided((rows, D + pn), (D + pn, 1))
        assert (whole[:, D:] == 7).all()


@pytest.mark.parametrize("rows,D", [(3, 64), (6, 4096), (400, 4096), (20, 4097), (300, 1024), (3, 33000), (900, 4096),
                                    (1700, 4097), (5000, 1024)])
@pytest.mark.parametrize("group", [0, 128])
def test_new_residual_in_place(rows, D, group):
    g = torch.Generator().manual_seed(D)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    for which in (0, 1):
        x, res = _rows(g, rows, D, torch.bfloat16), _rows(g, rows, D, torch.bfloat16)
        want = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group)
        into = (x, res)[which]
        got = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group, new_residual=into)
        assert got[2] is into and torch.equal(into, want[2]) and torch.equal(got[1], want[1])
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))


@pytest.mark.parametrize("rows,D", [(6, 256), (5, 4096), (400, 4096), (5, 4097), (4, 40000)])
@pytest.mark.parametrize("group", [0, 128])
def test_zero_rows_and_groups(rows, D, group):
    """A group of zeros has the least scale and zero codes; its neighbours are as ever."""
    g = torch.Generator().manual_seed(D)
    x = _rows(g, rows, D, torch.float32)
    x[1] = 0
    x[2, :200] = 0
    x[3] *= 1e-30  # the sum of squares vanishes beside eps
    w = torch.ones(D, device=DEV)
    w[200:] *= 0.5
    got = rn.rmsnorm_fwd_q8(x, w, EPS, group=group)
    _check(got, x, None, w, 0.0, group)
    assert (got[0][1].float() == 0).all() and torch.isfinite(got[1]).all() and (got[1] > 0).all()


@pytest.mark.parametrize("rows,D", [(6, 256), (5, 4096), (400, 4096), (5, 4097), (3, 40000)])
@pytest.mark.parametrize("group", [0, 128])
def test_values_that_are_not_numbers(rows, D, group):
    """A NaN in a row or an infinite weight takes its groups (its row) along and nothing else."""
    g = torch.Generator().manual_seed(D)
    x = _rows(g, rows, D, torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    clean = rn.rmsnorm_fwd_q8(x, w, EPS, group=group)
    y = x.clone()
    y[1, 5] = float("nan")
    y[2, 130] = float("inf")
    out, scale, _ = rn.rmsnorm_fwd_q8(y, w, EPS, group=group)
    value = grouped(out.float(), group) * scale.view(rows, -1)[..., None]
    assert value[1].isnan().all()
    bad = 130 // (group or D)
    assert value[2, bad].isnan().all() and not scale.view(rows, -1)[2, bad].isfinite()
    other = torch.arange(rows, device=DEV) // 1
    keep = (other != 1) & (other != 2)
    assert torch.equal(out.view(torch.uint8)[keep], clean[0].view(torch.uint8)[keep])
    assert torch.equal(scale[keep], clean[1][keep])
    w2 = w.clone()
    w2[7] = float("inf")
    out, scale, _ = rn.rmsnorm_fwd_q8(x, w2, EPS, group=group)
    value = grouped(out.float(), group) * scale.view(rows, -1)[..., None]
    assert value[:, 0].isnan().all()
    if group:
        assert torch.equal(out.view(torch.uint8)[:, group:], clean[0].view(torch.uint8)[:, group:])
        assert torch.equal(scale[:, 1:], clean[1][:, 1:])


def test_large_offsets():
    """More than 2^31 elements of input, 2^32 bytes; rows are independent."""
    rows, D = 524293, 4096
    x = torch.zeros(rows, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(3)
    at = torch.tensor([0, 1, 262143, 262144, 400001, rows - 1], device=DEV)
    x[at] = torch.randn(6, D, generator=g).to(torch.bfloat16).to(DEV)
    res = torch.zeros_like(x)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    for group in (0, 128):
        out, scale, nr = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group)
        _check((out[at], scale[at], nr[at]), x[at], res[at], w, 0.0, group)
        rest = torch.ones(rows, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert int((out.view(torch.uint8) != 0).any(1)[rest].sum()) == 0
        assert torch.equal(nr, x)
        del out, scale, nr, rest
    del x, res
    torch.cuda.empty_cache()


def test_graph_stream_empty_and_leading_dimensions():
    g = torch.Generator().manual_seed(4)
    x, res = _rows(g, 600, 2048, torch.bfloat16).view(3, 200, 2048), _rows(g, 600, 2048, torch.bfloat16).view(3, 200, 2048)
    w = torch.ones(2048, dtype=torch.bfloat16, device=DEV)
    out, scale, nr = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=64)
    assert out.shape == x.shape and scale.shape == (3, 200, 32) and nr.shape == x.shape
    o2, s2, n2 = torch.empty_like(out), torch.empty_like(scale), torch.empty_like(nr)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=64, out=o2, scale=s2, new_residual=n2)
    for k in range(2):
        x.neg_()
        gr.replay()
        want = rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=64)
        torch.cuda.synchronize()
        for a, b in zip((o2, s2, n2), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        got.append(rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=64, stream=s))
    for s, r in zip(streams, got):
        s.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r, want))
    e = rn.rmsnorm_fwd_q8(x[:0], w, EPS, 0.0, res[:0], group=128)
    assert e[0].shape == (0, 200, 2048) and e[1].shape == (0, 200, 16)
    one = rn.rmsnorm_fwd_q8(x[0, 0], w, EPS)
    assert one[0].shape == (2048,) and one[1].shape == ()


def test_the_same_bits_every_time():
    g = torch.Generator().manual_seed(5)
    for rows, D, group in ((4, 4096, 0), (900, 4096, 128), (3000, 512, 0), (300, 4097, 0), (5, 40000, 32)):
        x = _rows(g, rows, D, torch.float16)
        w = torch.ones(D, dtype=torch.float16, device=DEV)
        a = rn.rmsnorm_fwd_q8(x, w, EPS, group=group)
        for _ in range(3):
            b = rn.rmsnorm_fwd_q8(x, w, EPS, group=group)
            assert torch.equal(a[1], b[1]) and torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))


def test_python_refusals():
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    bad = [dict(group=16), dict(group=-1), dict(group=256), dict(out=x), dict(out=torch.zeros(4, 65, device=DEV).to(E4M3)),
           dict(scale=torch.zeros(4, 1, device=DEV)), dict(scale=torch.zeros(4, device=DEV).half()), dict(new_residual=x),
           dict(residual=x[:2]), dict(residual=x.half()), dict(residual=x, new_residual=x.half()),
           dict(out=torch.zeros(4, 64).to(E4M3)), dict(group=32, scale=torch.zeros(4, device=DEV))]
    for kw in bad:
        with pytest.raises(ValueError):
            rn.rmsnorm_fwd_q8(x, w, EPS, **kw)
    with pytest.raises(ValueError):
        rn.rmsnorm_fwd_q8(x, w[:32], EPS)
    with pytest.raises(ValueError):
        rn.rmsnorm_fwd_q8(x.t(), w, EPS)
    with pytest.raises(TypeError):
        rn.rmsnorm_fwd_q8(x.double(), w.double(), EPS)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_fwd_q8(x, w, -1.0)
    with pytest.raises(rn.RmsnormError):  # the scales in the codes
        buf = torch.zeros(4 * 64, dtype=torch.uint8, device=DEV)
        rn.rmsnorm_fwd_q8(x, w, EPS, out=buf.view(E4M3).view(4, 64), scale=buf.view(torch.float32)[:4])
    with pytest.raises(rn.RmsnormError):  # one row on from the residual
        r = torch.zeros(5, 64, device=DEV)
        rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, r[:4], new_residual=r[1:])


def test_written_tensors_count_as_changed():
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    o, s, n = torch.zeros(4, 64, device=DEV).to(E4M3), torch.zeros(4, device=DEV), torch.zeros(4, 64, device=DEV)
    before = [t._version for t in (o, s, n, x)]
    rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, x, out=o, scale=s, new_residual=n)
    assert [t._version for t in (o, s, n, x)] == [before[0] + 1, before[1] + 1, before[2] + 1, before[3]]


@pytest.mark.parametrize("rows,D", [(4, 4096), (900, 4096), (700, 4104), (1000, 1000), (5, 20000)])
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_all_tensors_at_one_offset(rows, D, group, dt):
    """Rows one element past a 16-byte boundary, codes one byte past a word; and weights
    alone off their boundary."""
    g = torch.Generator().manual_seed(D)
    x, res, nr = (_rows(g, rows, D, DT[dt], off=1) for _ in range(3))
    wide = (1 + 0.2 * torch.randn(D + 1, generator=g)).to(DT[dt]).to(DEV)
    out = torch.empty(rows * D + 1, dtype=torch.uint8, device=DEV)[1:].view(rows, D).view(E4M3)
    _check(rn.rmsnorm_fwd_q8(x, wide[:D], EPS, 0.0, res, group=group, out=out, new_residual=nr), x, res, wide[:D], 0.0, group)
    y = x.contiguous().clone()
    assert y.data_ptr() % 16 == 0
    _check(rn.rmsnorm_fwd_q8(y, wide[1:], EPS, group=group), y, None, wide[1:], 0.0, group)


def test_more_rows_than_a_ring_goes_round():
    """Many rows a CTA, each unlike its neighbours."""
    for rows, D, dt, group in ((5001, 4096, torch.bfloat16, 0), (9999, 2048, torch.float16, 0), (20000, 1536, torch.bfloat16, 0), (9001, 4097, torch.float16, 64), (6000, 2048, torch.float32, 128),
                               (40000, 256, torch.bfloat16, 32)):
        g = torch.Generator().manual_seed(rows)
        x, res = _rows(g, rows, D, dt), _rows(g, rows, D, dt)
        w = (1 + 0.2 * torch.randn(D, generator=g)).to(dt).to(DEV)
        _check(rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group), x, res, w, 0.0, group)


@pytest.mark.parametrize("rows,D,group", [(3000, 4096, 0), (6000, 4096, 0), (3000, 4096, 128), (3000, 4097, 64)])
def test_wait_timeout_is_reported_and_context_survives(rows, D, group):
    """A row whose copies are never issued: the wait ends, the status says so, and the
    next call is right."""
    g = torch.Generator().manual_seed(6)
    x, res = _rows(g, rows, D, torch.bfloat16), _rows(g, rows, D, torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    rn.rmsnorm_device_status(clear=True)
    rn.rmsnorm_debug_inject(drop_tile=1501, budget_cycles=2_000_000)
    try:
        rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group)
        bits = rn.rmsnorm_device_status(clear=True)
    finally:
        rn.rmsnorm_debug_inject(-1, 0)
    assert bits & rn.DEVSTATUS_WAIT_TIMEOUT
    _check(rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, res, group=group), x, res, w, 0.0, group)
    assert rn.rmsnorm_device_status(clear=True) == 0


def test_calls_of_two_threads():
    """Two host threads, each with its own stream and problem, at once."""
    import threading
    g = torch.Generator().manual_seed(7)
    problems = [(_rows(g, 3000, 4096, torch.bfloat16), torch.ones(4096, dtype=torch.bfloat16, device=DEV), 0),
                (_rows(g, 2000, 1001, torch.float32), torch.ones(1001, device=DEV), 32)]
    want = [rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, x, group=gr) for x, w, gr in problems]
    torch.cuda.synchronize()
    same = [False, False]

    def work(i):
        x, w, gr = problems[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [rn.rmsnorm_fwd_q8(x, w, EPS, 0.0, x, group=gr) for _ in range(20)]
        s.synchronize()
        same[i] = all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for r in got for a, b in zip(r, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same)
