"""The operators of 8-bit serving and of image and video tokens beside the
norms, the rotary embedding and the cache append, as cases that can be timed
and compared: the fused residual-add norm with an e4m3 output and its scales,
rotary positions with several axes (forward and backward), the append that
quantises the KV cache as it writes it, and the read that brings cached tokens
back into 16 or 32 bits.

`run` computes each in plain torch operations in 32 bits (angles in 64) where
`own` is false, and through the framework's entry points where it is true.
`exact` computes the same from the definitions in 64 bits, the roundings to 8
bits among them.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
TOP = {"e4m3": 448.0, "i8": 127.0}  # the largest code
FLOOR = 2.0 ** -126


def listed():
    return [
        # One decode step of four sequences: the input of the 8-bit q, k and v projection, a scale a token.
        dict(name="norm_q8_decode", op="norm", rows=4, D=4096, dtype="bf16", res=True, group=0, wb=0.0, pad=0),
        # Prefill of the widest model row, a scale a token.
        dict(name="norm_q8_prefill", op="norm", rows=16384, D=8192, dtype="bf16", res=True, group=0, wb=0.0, pad=0),
        # The first norm of a model (nothing to add yet) before a product with scales for 128 elements,
        # (1 + w) weights.
        dict(name="norm_q8_groups", op="norm", rows=8192, D=4096, dtype="f16", res=False, group=128, wb=1.0, pad=0),
        # Rows off 16-byte boundaries, the last group of each a single element.
        dict(name="norm_q8_odd", op="norm", rows=5000, D=4097, dtype="bf16", res=True, group=128, wb=0.0, pad=0),
        # Training on images and video: q and k as views of one projection, pairs in three runs of
        # time, height and width.
        dict(name="axes_train", op="rope", T=16384, Hq=32, Hkv=8, Dh=128, sections="16,24,24", turns=False,
             dtype="bf16", interleaved=False, far=32768, grid=24, fused=True, inverse=False),
        # The backward of an image encoder's attention: two axes that take turns, ragged token count.
        dict(name="axes_backward", op="rope", T=5001, Hq=16, Hkv=16, Dh=80, sections="20,20", turns=True,
             dtype="f32", interleaved=True, far=64, grid=64, fused=False, inverse=True),
        # One decode step of eight sequences into an 8-bit paged cache.
        dict(name="append_q8_decode", op="append", T=8, Hq=32, Hkv=8, Dh=128, sections="64", turns=False,
             dtype="bf16", fmt="e4m3", interleaved=False, far=131072, grid=1, fused=True),
        # The prefill of image and text tokens into an 8-bit cache, positions of three axes.
        dict(name="append_q8_prefill", op="append", T=16384, Hq=32, Hkv=8, Dh=128, sections="24,20,20", turns=True,
             dtype="bf16", fmt="e4m3", interleaved=False, far=32768, grid=32, fused=True),
        # A chunk of a long prompt: appended in whole numbers, heads of 80 of which 32 elements turn, then
        # the context read back for the chunk's attention.
        dict(name="append_read_chunk", op="append_read", T=1000, Hq=32, Hkv=8, Dh=80, sections="16", turns=False,
             dtype="f16", fmt="i8", interleaved=True, far=8192, grid=1, fused=True, context=4000),
        # A short context read back.
        dict(name="read_q8_short", op="read", T=77, Hkv=8, Dh=128, dtype="bf16", fmt="e4m3", holes=0.0),
        # Long contexts of several requests read back, padded as a captured step is.
        dict(name="read_q8_long", op="read", T=65536, Hkv=8, Dh=128, dtype="bf16", fmt="e4m3", holes=0.02),
        # An odd number of tokens, an odd head size, into 32 bits.
        dict(name="read_q8_odd", op="read", T=9999, Hkv=3, Dh=90, dtype="f32", fmt="i8", holes=0.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "rope", "rope", "append", "append", "append_read", "read", "read"])
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        kind = rng.random()
        D = _spread(rng, 64, 8192)
        D = max(64, D // 64 * 64) if kind < 0.6 else D // 8 * 8 if kind < 0.8 else D
        rows = max(1, min(_spread(rng, 1, 16384), 16384 * 8192 * 2 // (SIZE[dtype] * D)))
        return dict(op=op, rows=rows, D=D, dtype=dtype, res=rng.random() < 0.75, group=rng.choice([0, 0, 32, 64, 128]),
                    wb=float(rng.random() < 0.3), pad=rng.choice([0, 0, 64, 8]))
    Dh = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "read":
        dtype = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, T=min(_spread(rng, 1, 65536), 65536 * 1024 * 2 // (Hkv * Dh * SIZE[dtype])), Hkv=Hkv, Dh=Dh,
                    dtype=dtype, fmt=rng.choice(["e4m3", "i8"]), holes=rng.choice([0.0, 0.02]))
    half = rng.choice([Dh, Dh, max(6, Dh // 4 * 2)]) // 2
    axes = rng.choice([1, 2, 3, 3])
    cuts = sorted(rng.sample(range(1, half), axes - 1))
    sections = [b - a for a, b in zip([0] + cuts, cuts + [half])]
    c = dict(op=op, T=_spread(rng, 1, 16384), Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, Dh=Dh,
             sections=",".join(map(str, sections)), turns=rng.random() < 0.5,
             dtype=rng.choice(["bf16", "f16", "f32"]) if op == "rope" else rng.choice(["bf16", "f16"]),
             interleaved=rng.random() < 0.4, far=_spread(rng, 1000, 1000000), grid=_spread(rng, 1, 64),
             fused=rng.random() < 0.6)
    if op == "rope":
        c["inverse"] = rng.random() < 0.4
    else:
        c["fmt"] = "e4m3" if op == "append" else rng.choice(["e4m3", "i8"])
    if op == "append_read":
        c["T"] = min(c["T"], 4096)
        c["context"] = _spread(rng, 1, 32768)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pair_axis(sections, turns):
    """The axis of each pair, [rot / 2] int32 on the host: a run of pairs for each axis, or pairs
    that go round the axes, past those that have all of theirs."""
    if not turns:
        return torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(torch.int32)
    left, order = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                order.append(a)
    return torch.tensor(order, dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=g, device=DEVICE) * std + mean

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    if case["op"] == "norm":
        rows, D, pad = case["rows"], case["D"], case["pad"]

        def tokens(std):  # rows of uneven size with a few large channels, as activations have them
            buf = torch.empty(rows, D + pad, dtype=dt, device=DEVICE)
            wide = 1.0 + 20.0 * (uniform(1, D) < 0.004)
            buf[:, :D].copy_(std * normal(rows, D) * wide * torch.exp(0.5 * normal(rows, 1)))
            return buf[:, :D]

        s["x"] = tokens(1.0)
        s["residual"] = tokens(2.0) if case["res"] else None
        s["w"] = normal(D, mean=1.0 - case["wb"], std=0.1).to(dt)
        s["eps"] = 1e-6
        return s

    T, Hkv, Dh = case["T"], case["Hkv"], case["Dh"]

    def cache(rows):  # what earlier steps left in the pool
        values = normal(rows, Hkv, Dh)
        top = values.abs().amax(-1)
        codes = values * (TOP[case["fmt"]] / top)[..., None]
        codes = codes.round() if case["fmt"] == "i8" else codes
        return codes.to(CODES[case["fmt"]]), top / TOP[case["fmt"]]

    if case["op"] == "read":
        rows = T + T // 8 + 16
        s["k_cache"], s["k_scale"] = cache(rows)
        s["v_cache"], s["v_scale"] = cache(rows)
        # blocks of 16 slots in any order, the last of them in part
        blocks = torch.randperm(rows // 16, generator=g, device=DEVICE)[:(T + 15) // 16]
        slots = (blocks[:, None] * 16 + torch.arange(16, device=DEVICE)).flatten()[:T]
        s["slots"] = torch.where(uniform(T) < case["holes"], torch.full_like(slots, -1), slots)
        return s

    Hq = case["Hq"]
    sections = [int(n) for n in case["sections"].split(",")]
    A, rot = len(sections), 2 * sum(sections)
    s["rot"] = rot
    if case["fused"]:  # heads of one projection's output
        qkv = normal(T, Hq + 2 * Hkv, Dh).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"], s["k"], s["v"] = (normal(T, h, Dh).to(dt) for h in (Hq, Hkv, Hkv))
    # a quarter of text, whose axes agree, then frames of grid x grid tokens
    start = torch.randint(0, max(case["far"] - T, 1), (1,), generator=g, device=DEVICE)
    i, n = torch.arange(T, device=DEVICE), case["grid"]
    axes = {1: [i], 2: [i // n, i % n], 3: [i // (n * n), i // n % n, i % n]}[A]
    text = i < T // 4
    s["positions"] = torch.stack([start + torch.where(text, i, T // 4 + p) for p in axes])
    s["pair_axis"] = _pair_axis(sections, case["turns"])
    s["inv_freq"] = torch.pow(torch.tensor(500000.0, dtype=torch.float64),
                              -2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if case["op"] != "rope":
        rows = 2 * T + 64 + case.get("context", 0)
        s["k_cache"], s["k_scale"] = cache(rows)
        s["v_cache"], s["v_scale"] = cache(rows)
        slots = torch.randperm(rows, generator=g, device=DEVICE)
        s["slots"] = torch.where(uniform(T) < 0.02, torch.full_like(slots[:T], -1), slots[:T])
        if case["op"] == "append_read":  # the tokens before the chunk, then the chunk
            s["context_slots"] = torch.cat([slots[T:T + case["context"]], s["slots"]])
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "rope": _rope, "append": _append, "append_read": _append_read, "read": _read}[s["op"]](s)


def _own(s):
    import rmsnorm_fwd_bwd_add_gb300 as rn
    if s["op"] == "norm":
        return rn.rmsnorm_fwd_q8(s["x"], s["w"], s["eps"], s["wb"], s["residual"], group=s["group"])
    if s["op"] == "rope":
        return rn.rmsnorm_rope_axes(s["q"], s["k"], s["positions"], s["inv_freq"], s["pair_axis"],
                                    interleaved=s["interleaved"], inverse=s["inverse"])
    if s["op"] == "read":
        return rn.rmsnorm_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                                  dtype=DTYPES[s["dtype"]])
    q = rn.rmsnorm_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                             s["inv_freq"], k_scale=s["k_scale"], v_scale=s["v_scale"], pair_axis=s["pair_axis"],
                             interleaved=s["interleaved"])
    if s["op"] == "append":
        return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    k, v = rn.rmsnorm_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["context_slots"],
                              dtype=DTYPES[s["dtype"]])
    return q, k, v, s["k_scale"], s["v_scale"]


def _norm(s):
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    rows, D = h.shape
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"])
    v = h * (s["wb"] + s["w"].float())
    G = s["group"] or D
    n = (D + G - 1) // G
    top = torch.nn.functional.pad(v.abs(), (0, n * G - D)).view(rows, n, G).amax(-1).clamp(min=448.0 * FLOOR)
    by = (448.0 / top).repeat_interleave(G, 1)[:, :D]
    codes = (v * by).to(torch.float8_e4m3fn)
    scale = top * r / 448.0
    new_residual = None if s["residual"] is None else h.to(s["x"].dtype)
    return codes, scale if s["group"] else scale[:, 0], new_residual


def _turned(x, s, sign=1.0):
    """Rotates the first `rot` elements of each head of [T, H, Dh]; 32 bits."""
    rot, half = s["rot"], s["rot"] // 2
    p = s["positions"].double()[s["pair_axis"].long().to(DEVICE)].t()  # [T, rot / 2]
    angle = p * s["inv_freq"].to(DEVICE)
    c, n = angle.cos().float()[:, None, :], (angle.sin() * sign).float()[:, None, :]
    x32 = x.float()
    if s["interleaved"]:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x32[..., :half], x32[..., half:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x32[..., rot:]], -1)


def _rope(s):
    sign = -1.0 if s["inverse"] else 1.0
    return _turned(s["q"], s, sign).to(s["q"].dtype), _turned(s["k"], s, sign).to(s["k"].dtype)


def _in_8_bits(x, fmt):
    """(codes, scales) of the heads of [T, H, Dh]."""
    top = x.abs().amax(-1).clamp(min=TOP[fmt] * FLOOR)
    codes = x * (TOP[fmt] / top)[..., None]
    return (codes.round() if fmt == "i8" else codes).to(CODES[fmt]), top / TOP[fmt]


def _append(s):
    rows = s["k_cache"].shape[0]
    at = torch.where(s["slots"] < 0, torch.full_like(s["slots"], rows), s["slots"])
    caches, scales = [], []
    for cache, scale, t in ((s["k_cache"], s["k_scale"], _turned(s["k"], s)), (s["v_cache"], s["v_scale"], s["v"].float())):
        codes, by = _in_8_bits(t, s["fmt"])
        bits = cache.view(torch.uint8)
        longer = torch.cat([bits, bits[:1]])  # one row more, for the tokens that are not kept
        longer[at] = codes.view(torch.uint8)
        caches.append(longer[:rows].view(cache.dtype))
        longer = torch.cat([scale, scale[:1]])
        longer[at] = by
        scales.append(longer[:rows])
    return _turned(s["q"], s).to(s["q"].dtype), *caches, *scales


def _values(cache, scale, slots, dtype):
    at = slots.clamp(min=0)
    x = cache.view(torch.uint8)[at].view(cache.dtype).float() * scale[at][..., None]
    return torch.where((slots < 0)[:, None, None], torch.zeros_like(x), x).to(dtype)


def _append_read(s):
    q, k_cache, v_cache, k_scale, v_scale = _append(s)
    return (q, _values(k_cache, k_scale, s["context_slots"], q.dtype),
            _values(v_cache, v_scale, s["context_slots"], q.dtype), k_scale, v_scale)


def _read(s):
    dt = DTYPES[s["dtype"]]
    return _values(s["k_cache"], s["k_scale"], s["slots"], dt), _values(s["v_cache"], s["v_scale"], s["slots"], dt)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, z = case, SIZE[case["dtype"]]
    if c["op"] == "norm":  # x (and residual) in; codes, scales (and new_residual) out
        n = c["rows"] * c["D"]
        groups = -(-c["D"] // c["group"]) if c["group"] else 1
        return {"bytes": n * (z * (3 if c["res"] else 1) + 1) + c["D"] * z + 4 * groups * c["rows"], "flops": 9 * n}
    read = lambda tokens: tokens * (2 * c["Hkv"] * (c["Dh"] * (1 + z) + 4) + 8)  # noqa: E731
    if c["op"] == "read":
        return {"bytes": read(c["T"]), "flops": 2 * c["T"] * c["Hkv"] * c["Dh"]}
    axes = len(c["sections"].split(","))
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["Dh"]
        return {"bytes": 2 * n * z + 8 * axes * c["T"], "flops": 3 * n}
    n = c["T"] * (2 * c["Hq"] * z + 2 * c["Hkv"] * (z + 1)) * c["Dh"] + c["T"] * (8 * axes + 8 + 8 * c["Hkv"])
    flops = c["T"] * (3 * c["Hq"] + 8 * c["Hkv"]) * c["Dh"]
    if c["op"] == "append":
        return {"bytes": n, "flops": flops}
    tokens = c["T"] + c["context"]
    return {"bytes": n + read(tokens), "flops": flops + 2 * tokens * c["Hkv"] * c["Dh"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest(x, fmt):
    """x (in units of its scale, 64 bits) at the nearest code, ties to even."""
    if fmt == "i8":
        return torch.round(x)
    exponent = torch.frexp(x)[1].double() - 1.0  # of 1.f x 2^e
    step = torch.exp2(torch.clamp(exponent, min=-6.0) - 3.0)  # four significant bits, three below 2^-6
    return torch.clamp(torch.round(x / step) * step, -448.0, 448.0)


def _unit(x, fmt):
    """The scale that takes the largest of x's last dimension to the largest code."""
    largest = torch.max(torch.abs(x), dim=-1, keepdim=True).values / TOP[fmt]
    return torch.where(largest < FLOOR, torch.full_like(largest, FLOOR), largest)


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda t: None if t is None else t.double().contiguous()  # noqa: E731
    if case["op"] == "norm":
        h = wide(s["x"])
        if s["residual"] is not None:
            h = h + wide(s["residual"])
        r = 1.0 / torch.sqrt(torch.mean(h * h, -1) + s["eps"])
        v = h * (wide(s["w"]) + s["wb"])
        parts = v.split(s["group"] or case["D"], dim=1)
        units = [_unit(p, "e4m3") for p in parts]
        codes = torch.cat([_nearest(p / u, "e4m3") for p, u in zip(parts, units)], 1)
        scale = torch.cat(units, 1) * r[:, None]
        return codes, scale if s["group"] else scale.squeeze(1), None if s["residual"] is None else h

    def values(codes, unit, slots):
        kept = slots >= 0
        out = torch.zeros(slots.shape[0], case["Hkv"], case["Dh"], dtype=torch.float64, device=DEVICE)
        out[kept] = codes[slots[kept]] * unit[slots[kept]].unsqueeze(-1)
        return out

    if case["op"] == "read":
        return tuple(values(wide(s[c]), wide(s[u]), s["slots"]) for c, u in (("k_cache", "k_scale"), ("v_cache", "v_scale")))

    def turned(x, sign):  # pairs as complex numbers
        x, rot = wide(x), s["rot"]
        axis = s["pair_axis"].tolist()
        angle = torch.stack([sign * s["positions"][a].double() * f for a, f in zip(axis, s["inv_freq"].tolist())], 1)
        by = torch.polar(torch.ones_like(angle), angle)[:, None, :]
        if s["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * by
            first = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * by
            first = torch.cat([z.real, z.imag], -1)
        return torch.cat([first, x[..., rot:]], -1)

    if case["op"] == "rope":
        sign = -1.0 if s["inverse"] else 1.0
        return turned(s["q"], sign), turned(s["k"], sign)
    kept = s["slots"] >= 0
    q = turned(s["q"], 1.0)
    caches = []
    for cache, unit, t in (("k_cache", "k_scale", turned(s["k"], 1.0)), ("v_cache", "v_scale", wide(s["v"]))):
        codes, units = wide(s[cache]), wide(s[unit])
        u = _unit(t, s["fmt"])
        codes[s["slots"][kept]] = _nearest(t / u, s["fmt"])[kept]
        units[s["slots"][kept]] = u.squeeze(-1)[kept]
        caches.append((codes, units))
    (k, k_unit), (v, v_unit) = caches
    if case["op"] == "append":
        return q, k, v, k_unit, v_unit
    return q, values(k, k_unit, s["context_slots"]), values(v, v_unit, s["context_slots"]), k_unit, v_unit
