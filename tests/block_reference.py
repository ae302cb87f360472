"""The norm pair around a block in 64 bits, with the size of the terms each
result is made of, for the tests' tolerances.

Tolerances.  u = 2^-24.  A sum the kernels form is off by at most 64 u of the
sum of its terms' absolute values: at most 40 additions in a thread, 10 levels
of the trees over lanes and warps, and under ten roundings of the terms.  The
sum of h^2 may be formed from four sums (of res^2, 2 res v, v^2 with v the added
term) as long as their absolute values add up to at most 8 times the result, so
r_h is within 64 * 8 / 2 = 256 u.  Each output is then within 256 u of the terms
it is made of, plus one rounding to its own type: half a step, eps / 2 of the
value, or half the smallest subnormal.  The sums over rows run through at most
rows / grid + 64 additions a column.
"""
import torch

U = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def _gate(gate, rows, D):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64)
    g = gate.double().reshape(-1, D)
    return g.repeat_interleave(rows // g.shape[0], 0)


def fwd(y, res, w_post, w_pre, eps, wb, gate, scale):
    """(out, h, rstd [2, rows]) and the terms of out and h."""
    y, res, w1 = y.double(), res.double(), wb + w_pre.double()
    rows, D = y.shape
    r_y = torch.ones(rows, 1, dtype=torch.float64, device=y.device)
    p = y
    if w_post is not None:
        r_y = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        p = y * r_y * (wb + w_post.double())
    v = scale * _gate(gate, rows, D).to(y.device) * p
    h = res + v
    r_h = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    th = res.abs() + v.abs()
    # a relative error of h's elements moves r_h too
    kappa = 1 + (th * h.abs()).sum(1, keepdim=True) / ((h * h).sum(1, keepdim=True) + eps * D)
    return h * r_h * w1, h, torch.cat([r_y, r_h], 1).t().contiguous(), \
        (th * kappa + h.abs() * kappa) * r_h * w1.abs(), th, kappa.squeeze(1)


def vjp(y, h, w_post, w_pre, g, eps, wb, gate, scale, g_res, rstd=None):
    """Dict of (value, terms) for g_y, g_h, gw_post, gw_pre, g_gate."""
    y, h, g, w1 = y.double(), h.double(), g.double(), wb + w_pre.double()
    rows, D = y.shape
    one = torch.ones(rows, 1, dtype=torch.float64, device=y.device)
    r_h = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    r_y = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if w_post is not None else one
    if rstd is not None:
        r_y = rstd[0].double().reshape(-1, 1) if w_post is not None else one
        r_h = rstd[1].double().reshape(-1, 1)
    a = g * w1
    c = r_h * r_h * (a * h).mean(1, keepdim=True)
    c_t = r_h * r_h * (a * h).abs().mean(1, keepdim=True)
    gr = torch.zeros_like(y) if g_res is None else g_res.double()
    g_h = r_h * (a - h * c) + gr
    t_h = r_h * (a.abs() + h.abs() * c_t) + gr.abs()
    gate64 = _gate(gate, rows, D).to(y.device)
    w2 = wb + w_post.double() if w_post is not None else torch.ones(D, dtype=torch.float64, device=y.device)
    m = scale * gate64 * w2
    n = y * r_y
    out = {"g_h": (g_h, t_h), "gw_pre": ((g * h * r_h).sum(0), (g * h * r_h).abs().sum(0))}
    b, t_b = m * g_h, m.abs() * t_h
    if w_post is not None:
        e = (b * n).mean(1, keepdim=True)
        e_t = (t_b * n.abs()).mean(1, keepdim=True)
        out["g_y"] = (r_y * (b - n * e), r_y * (t_b + n.abs() * e_t))
        out["gw_post"] = ((scale * gate64 * g_h * n).sum(0), (abs(scale) * gate64.abs() * t_h * n.abs()).sum(0))
    else:
        out["g_y"] = (b, t_b)
    if gate is not None:
        G = gate.numel() // D
        out["g_gate"] = tuple(t.view(G, rows // G, D).sum(1) for t in
                              (scale * g_h * n * w2, abs(scale) * t_h * n.abs() * w2.abs()))
    return out


def check(name, got, want, terms, k=256.0):
    """|got - want| <= half a step of want's type + k u terms, element by element."""
    got64 = got.double().reshape(want.shape)
    eps = torch.finfo(got.dtype).eps
    allow = eps / 2 * (want.abs() + k * U * terms) + k * U * terms + TINY[got.dtype]
    assert torch.isfinite(got64).all(), "%s: not finite" % name
    off = (got64 - want).abs() - allow
    assert off.max() <= 0, "%s: off by %.3e more than allowed at %d (want %.6e)" % (
        name, off.max(), off.argmax(), want.flatten()[off.argmax()])
