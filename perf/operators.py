"""The operators between the matrix products of a decoder block, as cases that
can be timed and compared: the norms before and after a block fused with its
gate and residual scale (forward and VJP), rotary positions (half and
interleaved pairs, part of the head, scaled for long contexts; forward,
backward and the append to the KV cache), and the block tables and slot maps
that a serving step builds from its requests' lengths.

`run` computes each in plain torch operations in 32 bits (angles in 64) where
`own` is false, and through the framework's entry points where it is true.
`exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # One decode step of four sequences: the latency of the norm pair around a block,
        # with the (1 + w) weights of a sandwich-normed model.
        dict(name="block_fwd_decode", op="block_fwd", rows=4, D=4096, dtype="bf16", groups=0,
             post=True, wb=1.0, scale=1.0, pad=0),
        # Prefill of eight conditioned sequences: a gate row per sequence, the widest model row.
        dict(name="block_fwd_prefill", op="block_fwd", rows=16384, D=8192, dtype="bf16", groups=8,
             post=True, wb=0.0, scale=0.5, pad=0),
        # A row length off 16-byte boundaries, a learned gate per channel, no norm after the block
        # (a scaled residual).
        dict(name="block_fwd_odd", op="block_fwd", rows=5000, D=4097, dtype="f16", groups=1,
             post=False, wb=0.0, scale=0.22, pad=0),
        # The training backward of the prefill step, the forward's per-row scales at hand.
        dict(name="block_vjp_train", op="block_vjp", rows=16384, D=4096, dtype="bf16", groups=8,
             post=True, wb=0.0, scale=1.0, pad=0, rstd=True, gres=True),
        # The small fp16 problem of the tests, nothing saved by the forward.
        dict(name="block_vjp_small", op="block_vjp", rows=64, D=512, dtype="f16", groups=1,
             post=True, wb=0.0, scale=1.0, pad=0, rstd=False, gres=True),
        # fp32 training rows of a wider buffer, an odd number of them, one gate row for each row.
        dict(name="block_vjp_f32_rows", op="block_vjp", rows=4095, D=2048, dtype="f32", groups=4095,
             post=True, wb=0.0, scale=1.0, pad=64, rstd=True, gres=False),
        # Training: q and k as views of one fused projection, scaled for a long context.
        dict(name="rope_train", op="rope", T=16384, Hq=32, Hkv=8, Dh=128, rot=128, dtype="bf16",
             interleaved=False, scaling="yarn", far=131072, fused=True, inverse=False),
        # Its backward: half of each head rotated, interleaved pairs, ragged token count.
        dict(name="rope_backward", op="rope", T=5001, Hq=16, Hkv=4, Dh=128, rot=64, dtype="f32",
             interleaved=True, scaling="linear", far=32768, fused=False, inverse=True),
        # One decode step of eight sequences into a paged cache.
        dict(name="append_decode", op="append", T=8, Hq=32, Hkv=8, Dh=128, rot=128, dtype="bf16",
             interleaved=False, scaling="llama3", far=131072, fused=True),
        # A prefill chunk with an odd head size of which a part is rotated.
        dict(name="append_prefill", op="append", T=4096, Hq=32, Hkv=8, Dh=80, rot=32, dtype="f16",
             interleaved=False, scaling="none", far=4096, fused=True),
        # The bookkeeping of a decode step: 250 requests, one token each, some finished.
        dict(name="plan_decode", op="plan", B=250, new=1, block=16, far=8192, done=0.04),
        # The bookkeeping of a chunked step: many requests, chunks of up to 64 tokens.
        dict(name="plan_chunked", op="plan", B=4000, new=64, block=64, far=16384, done=0.02),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_fwd", "block_fwd", "block_vjp", "block_vjp", "rope", "append", "plan"])
    if op in ("block_fwd", "block_vjp"):
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        kind = rng.random()
        D = _spread(rng, 64, 8192)
        D = max(64, D // 64 * 64) if kind < 0.6 else D // 8 * 8 if kind < 0.8 else D
        most = 16384 * 8192 * 2 // (SIZE[dtype] * D * (2 if op == "block_vjp" else 1))
        rows = max(1, min(_spread(rng, 1, 16384), most))
        per = rng.choice([1, rows, _spread(rng, 1, rows)])
        rows = rows // per * per  # whole groups
        groups = rng.choice([0, 1, rows // per])
        c = dict(op=op, rows=rows, D=D, dtype=dtype, groups=groups, post=rng.random() < 0.75,
                 wb=float(rng.random() < 0.3), scale=round(rng.uniform(0.1, 1.5), 3),
                 pad=rng.choice([0, 0, 64, 8]))
        if op == "block_vjp":
            c.update(rstd=rng.random() < 0.6, gres=rng.random() < 0.75)
        return c
    if op in ("rope", "append"):
        Dh = rng.choice([64, 80, 96, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
        Hkv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, T=_spread(rng, 1, 16384), Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, Dh=Dh,
                 rot=rng.choice([Dh, Dh, max(2, Dh // 4 * 2)]),
                 dtype=rng.choice(["bf16", "f16", "f32"]) if op == "rope" else rng.choice(["bf16", "f16"]),
                 interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "ntk", "yarn", "llama3"]),
                 far=_spread(rng, 1000, 1000000), fused=rng.random() < 0.6)
        if op == "rope":
            c["inverse"] = rng.random() < 0.4
        return c
    return dict(op="plan", B=_spread(rng, 1, 4000), new=rng.choice([1, 1, _spread(rng, 2, 64)]),
                block=rng.choice([1, 16, 16, 64, 100]), far=_spread(rng, 100, 16384),
                done=round(rng.uniform(0, 0.1), 3))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inv_freq(rot, base, scaling, far):
    """(inverse frequencies in radians a position, [rot / 2] float64 on the host; the factor on
    cosine and sine) of a rotary embedding stretched from 8192 positions to `far`."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    inv = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    factor, trained = max(1.0, far / 8192.0), 8192.0
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling == "ntk":
        grown = base * factor ** (rot / (rot - 2.0)) if rot > 2 else base
        return torch.pow(torch.tensor(grown, dtype=torch.float64), -2.0 * i / rot), 1.0
    if scaling == "yarn":
        at = [rot * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return inv * (1 - ramp) + inv / factor * ramp, 0.1 * math.log(factor) + 1.0
    if scaling == "llama3":
        turns = trained * inv / (2 * math.pi)  # turns within the trained context
        smooth = ((turns - 1.0) / 3.0).clamp(0, 1)
        return inv * smooth + inv / factor * (1 - smooth), 1.0
    return inv, 1.0


def _wide(shape, pad, dtype, fill, g):
    """A [rows, D] tensor whose rows lie D + pad elements apart."""
    rows, D = shape
    buf = torch.empty(rows, D + pad, dtype=dtype, device=DEVICE)
    buf[:, :D].copy_(fill(rows, D, g))
    return buf[:, :D]


def _tokens(case):
    """The token budget of a step, which a captured step is padded to: near what the requests
    bring on average, so that now and then the last of them wait."""
    mean = 1.0 if case["new"] == 1 else 0.67 * (case["new"] + 1) / 2 + 0.33
    return (int(case["B"] * mean * 1.01) + 63) // 64 * 64


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case)

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=g, device=DEVICE) * std + mean

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEVICE)

    def ints(lo, hi, n):  # lo .. hi, both included
        return torch.randint(lo, hi + 1, (n,), generator=g, device=DEVICE)

    if case["op"] in ("block_fwd", "block_vjp"):
        rows, D, pad, dt = case["rows"], case["D"], case["pad"], DTYPES[case["dtype"]]
        # rows of uneven size, as tokens have them
        act = lambda r, d, _: normal(r, d) * torch.exp(0.5 * normal(r, 1))  # noqa: E731
        s["y"] = _wide((rows, D), pad, dt, act, g)
        s["w_post"] = normal(D, mean=1.0 - case["wb"], std=0.05).to(dt) if case["post"] else None
        s["w_pre"] = normal(D, mean=1.0 - case["wb"], std=0.05).to(dt)
        s["gate"] = None
        if case["groups"]:  # a slice of a wider modulation, as conditioning makes it
            G = case["groups"]
            s["gate"] = normal(G, 2 * D, mean=0.3, std=0.4).to(dt)[:, :D] if G > 1 else \
                normal(1, D, mean=0.3, std=0.4).to(dt)
        s["eps"] = 1e-6
        if case["op"] == "block_fwd":
            s["residual"] = _wide((rows, D), pad, dt, lambda r, d, _: 2.0 * normal(r, d), g)
        else:
            s["h"] = _wide((rows, D), pad, dt, lambda r, d, _: 2.0 * normal(r, d), g)
            s["g_out"] = _wide((rows, D), pad, dt, lambda r, d, _: normal(r, d), g)
            s["g_res"] = _wide((rows, D), pad, dt, lambda r, d, _: normal(r, d), g) if case["gres"] else None
            s["saved"] = None
            if case["rstd"]:  # what the forward wrote for these rows
                ms = [t.double().square().mean(-1) for t in (s["y"], s["h"])]
                s["saved"] = torch.stack([torch.rsqrt(m + s["eps"]) for m in ms]).float()
                if not case["post"]:
                    s["saved"][0] = 1.0
        return s

    if case["op"] in ("rope", "append"):
        T, Hq, Hkv, Dh, dt = case["T"], case["Hq"], case["Hkv"], case["Dh"], DTYPES[case["dtype"]]
        if case["fused"]:  # heads of one projection's output
            qkv = normal(T, Hq + 2 * Hkv, Dh).to(dt)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (normal(T, h, Dh).to(dt) for h in (Hq, Hkv, Hkv))
        start = ints(0, max(case["far"] - T, 0), 1)
        s["positions"] = start + torch.arange(T, device=DEVICE) if case["op"] == "rope" or T > 64 else \
            ints(0, case["far"] - 1, T)
        s["inv_freq"], s["attn_scale"] = _inv_freq(case["rot"], 500000.0, case["scaling"], case["far"])
        if case["op"] == "append":  # a paged pool with room around what this step writes
            rows = 2 * T + 64
            s["k_cache"] = normal(rows, Hkv, Dh).to(dt)
            s["v_cache"] = normal(rows, Hkv, Dh).to(dt)
            slots = torch.randperm(rows, generator=g, device=DEVICE)[:T]
            s["slots"] = torch.where(uniform(T) < 0.02, torch.full_like(slots, -1), slots)
        return s

    # plan: lengths, tables and a pool of free blocks in the middle of a run
    B, bs = case["B"], case["block"]
    lens = ints(0, case["far"], B)
    done = uniform(B) < case["done"]
    new = ints(1, case["new"], B)
    if case["new"] > 1:  # a third of the requests only decode
        new = torch.where(uniform(B) < 0.33, torch.ones_like(new), new)
    new = torch.where(done, torch.zeros_like(new), new)  # a freed row is given out in the next step
    have = (lens + bs - 1) // bs
    s["W"] = (case["far"] + case["new"] + bs - 1) // bs + 1
    held = int(have.sum())
    want = int(((lens + new + bs - 1) // bs - have).sum())
    spare = max(1, int(want * 0.98)) + 8  # now and then the last requests go without
    pool = B * s["W"]
    ids = torch.randperm(pool, generator=g, device=DEVICE).to(torch.int32)
    taken = torch.arange(s["W"], device=DEVICE)[None, :] < have[:, None]
    table = torch.full((B, s["W"]), -1, dtype=torch.int32, device=DEVICE)
    table[taken] = ids[:held]
    free = torch.full((pool,), -1, dtype=torch.int32, device=DEVICE)
    free[:spare] = ids[held:held + spare]
    s.update(lens=lens.to(torch.int32), new_lens=new.to(torch.int32), finished=done, block_table=table,
             free_blocks=free, free_count=torch.tensor([spare], dtype=torch.int32, device=DEVICE))
    s["T"] = _tokens(case)
    s["lens_kept"] = torch.empty_like(s["lens"])
    s["count_kept"] = torch.empty_like(s["free_count"])
    s["lens_out"] = torch.empty_like(s["lens"])
    s["count_out"] = torch.empty_like(s["free_count"])
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"block_fwd": _block_fwd, "block_vjp": _block_vjp, "rope": _rope, "append": _append,
            "plan": _plan}[s["op"]](s)


def _own(s):
    import rmsnorm_fwd_bwd_add_gb300 as rn
    if s["op"] == "block_fwd":
        return rn.rmsnorm_block_fwd(s["y"], s["residual"], s["w_post"], s["w_pre"], s["eps"], s["wb"],
                                    s["gate"], s["scale"], rstd=True)
    if s["op"] == "block_vjp":
        return rn.rmsnorm_block_vjp(s["y"], s["h"], s["w_post"], s["w_pre"], s["g_out"], s["eps"], s["wb"],
                                    s["gate"], s["scale"], s["g_res"], rstd=s["saved"])
    if s["op"] == "rope":
        return rn.rmsnorm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], attn_scale=s["attn_scale"],
                               interleaved=s["interleaved"], inverse=s["inverse"])
    if s["op"] == "append":
        q = rn.rmsnorm_rope_kv_append_ex(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"],
                                         s["v_cache"], s["inv_freq"], attn_scale=s["attn_scale"],
                                         interleaved=s["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    rn.rmsnorm_kv_release(s["lens"], s["finished"], s["block_table"], s["block"], s["free_blocks"],
                          s["free_count"], lens_out=s["lens_kept"], free_count_out=s["count_kept"])
    plan = rn.rmsnorm_kv_plan(s["lens_kept"], s["new_lens"], s["block_table"], s["block"], s["T"],
                              free_blocks=s["free_blocks"], free_count=s["count_kept"],
                              lens_out=s["lens_out"], free_count_out=s["count_out"])
    return (plan.positions, plan.slots, plan.requests, plan.starts, plan.granted, s["block_table"],
            s["free_blocks"], s["lens_out"], s["count_out"])


def _gate_rows(s, rows, dtype):
    """The gate of each row, [1 or rows, D]."""
    if s["gate"] is None:
        return torch.ones(1, 1, dtype=dtype, device=DEVICE)
    g = s["gate"].to(dtype)
    return g if g.shape[0] in (1, rows) else g.repeat_interleave(rows // g.shape[0], 0, output_size=rows)


def _block_fwd(s):
    y, res = s["y"].float(), s["residual"].float()
    rows, dt = y.shape[0], s["y"].dtype
    if s["w_post"] is not None:
        r_y = torch.rsqrt(y.square().mean(-1) + s["eps"])
        p = y * r_y[:, None] * (s["wb"] + s["w_post"].float())
    else:
        r_y, p = torch.ones(rows, device=DEVICE), y
    h = res + s["scale"] * _gate_rows(s, rows, torch.float32) * p
    r_h = torch.rsqrt(h.square().mean(-1) + s["eps"])
    out = h * r_h[:, None] * (s["wb"] + s["w_pre"].float())
    return out.to(dt), h.to(dt), torch.stack([r_y, r_h])


def _block_vjp(s):
    y, h, g = s["y"].float(), s["h"].float(), s["g_out"].float()
    rows, dt, D = y.shape[0], s["y"].dtype, y.shape[1]
    post = s["w_post"] is not None
    if s["saved"] is not None:
        r_y, r_h = s["saved"][0], s["saved"][1]
    else:
        r_y = torch.rsqrt(y.square().mean(-1) + s["eps"]) if post else torch.ones(rows, device=DEVICE)
        r_h = torch.rsqrt(h.square().mean(-1) + s["eps"])
    r_y, r_h = r_y[:, None], r_h[:, None]
    a = g * (s["wb"] + s["w_pre"].float())
    gw_pre = (g * h * r_h).sum(0)
    g_h = r_h * (a - h * r_h.square() * (a * h).mean(-1, keepdim=True))
    if s["g_res"] is not None:
        g_h = g_h + s["g_res"].float()
    n = y * r_y                                         # the block's output, normed, before its weight
    gate = s["scale"] * _gate_rows(s, rows, torch.float32)
    g_p = gate * g_h                                    # gradient of the normed output
    w2 = s["wb"] + s["w_post"].float() if post else torch.ones(D, device=DEVICE)
    g_gate = None
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        g_gate = (s["scale"] * g_h * n * w2).view(G, rows // G, D).sum(1)
    if not post:
        return g_p.to(dt), g_h.to(dt), None, gw_pre, g_gate
    gw_post = (g_p * n).sum(0)
    b = g_p * w2
    g_y = r_y * (b - n * (b * n).mean(-1, keepdim=True))
    return g_y.to(dt), g_h.to(dt), gw_post, gw_pre, g_gate


def _rotate(x, s, sign=1.0):
    """Rotates the first `rot` elements of each head of [T, H, Dh]."""
    rot, half = s["rot"], s["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].to(DEVICE)[None, :]
    c = (angle.cos() * s["attn_scale"]).float()[:, None, :]
    n = (angle.sin() * (s["attn_scale"] * sign)).float()[:, None, :]
    x32 = x.float()
    if s["interleaved"]:
        a, b = x32[..., 0:rot:2], x32[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x32[..., :half], x32[..., half:rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x32[..., rot:]], -1).to(x.dtype)


def _rope(s):
    sign = -1.0 if s["inverse"] else 1.0
    return _rotate(s["q"], s, sign), _rotate(s["k"], s, sign)


def _append(s):
    rows = s["k_cache"].shape[0]
    at = torch.where(s["slots"] < 0, torch.full_like(s["slots"], rows), s["slots"])
    caches = []
    for cache, t in ((s["k_cache"], _rotate(s["k"], s)), (s["v_cache"], s["v"])):
        longer = torch.cat([cache, cache[:1]])  # one row more, for the tokens that are not kept
        longer[at] = t
        caches.append(longer[:rows])
    return _rotate(s["q"], s), caches[0], caches[1]


def _plan(s):
    bs, T, W = s["block"], s["T"], s["W"]
    table, free = s["block_table"].clone(), s["free_blocks"].clone()
    lens, new, done = s["lens"].long(), s["new_lens"].long(), s["finished"]
    B, n = lens.shape[0], free.shape[0]
    col = torch.arange(W, device=DEVICE)
    # release: the finished requests' blocks go back on the stack, in order
    gone = (col[None, :] < ((lens + bs - 1) // bs)[:, None]) & done[:, None]
    rank = gone.flatten().long().cumsum(0).view(B, W) - 1 + s["free_count"].long()
    longer = torch.cat([free, free[:1]])
    longer[torch.where(gone, rank, torch.full_like(rank, n))] = table
    free = longer[:n]
    count = s["free_count"].long() + gone.sum()
    lens = torch.where(done, torch.zeros_like(lens), lens)
    # plan: new blocks off the top of the stack, for the requests that get theirs
    have, want = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
    ends = new.cumsum(0)
    fits = (want <= W) & (ends <= T)
    need = torch.where(fits, want - have, torch.zeros_like(have))
    cum = need.cumsum(0)
    granted = fits & ((need == 0) | (cum <= count))
    fresh = (col[None, :] >= have[:, None]) & (col[None, :] < want[:, None]) & granted[:, None]
    top = count - 1 - (cum - need)[:, None] - (col[None, :] - have[:, None])
    table = torch.where(fresh, free[top.clamp(0, n - 1)], table)
    popped = torch.where(granted, need, torch.zeros_like(need)).sum()
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEVICE), ends])
    t = torch.arange(T, device=DEVICE)
    req = torch.searchsorted(ends, t, right=True)
    live = req < B
    req0 = req.clamp(max=B - 1)
    pos = torch.where(live, lens[req0] + t - starts[req0], torch.zeros_like(t))
    block = table.flatten()[req0 * W + (pos // bs).clamp(max=W - 1)].long()
    slots = torch.where(live & granted[req0], block * bs + pos % bs, torch.full_like(t, -1))
    requests = torch.where(live, req, torch.full_like(t, -1)).to(torch.int32)
    lens_out = torch.where(granted, lens + new, lens).to(torch.int32)
    return (pos, slots, requests, starts, granted, table, free, lens_out,
            (count - popped).to(torch.int32))


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("block_fwd", "block_vjp"):
        n, z = c["rows"] * c["D"], SIZE[c["dtype"]]
        G, D = c["groups"], c["D"]
        small = (1 + c["post"]) * D * z + G * D * z
        if c["op"] == "block_fwd":  # y, residual in; out, new_residual and both scales out
            return {"bytes": 4 * n * z + small + 8 * c["rows"], "flops": 14 * n}
        # y, h, g_out (and g_residual) in; g_y, g_h and the weights' and gate's gradients out
        tensors = 5 + c["gres"]
        return {"bytes": tensors * n * z + small + (1 + c["post"] + G) * D * 4 + 8 * c["rows"] * c["rstd"],
                "flops": 30 * n}
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["Dh"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 8 * c["T"], "flops": 3 * n}
    if c["op"] == "append":
        n = c["T"] * (c["Hq"] + 2 * c["Hkv"]) * c["Dh"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 16 * c["T"], "flops": 3 * n}
    tokens = _tokens(c)
    blocks = tokens / c["block"] + c["done"] * c["B"] * c["far"] / 2 / c["block"]
    return {"bytes": tokens * 20 + c["B"] * (3 * 4 + 8 + 1) + blocks * 8, "flops": tokens * 8.0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _norm64(x, w, wb, eps):
    return x / torch.sqrt(torch.mean(x * x, dim=-1, keepdim=True) + eps) * (w + wb)


def _joined64(y, res, w_post, gate, s):
    """residual + scale * gate * norm(y): the residual stream after the block."""
    p = y if w_post is None else _norm64(y, w_post, s["wb"], s["eps"])
    if gate is None:
        return res + s["scale"] * p
    G, (rows, D) = gate.shape[0], y.shape
    return (res.view(G, -1, D) + s["scale"] * gate[:, None, :] * p.view(G, -1, D)).view(rows, D)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    wide = lambda t: None if t is None else t.double().contiguous()  # noqa: E731
    if case["op"] == "block_fwd":
        y, w2 = wide(s["y"]), wide(s["w_post"])
        h = _joined64(y, wide(s["residual"]), w2, wide(s["gate"]), s)
        scales = [1.0 / torch.sqrt(torch.mean(t * t, -1) + s["eps"]) for t in (y, h)]
        if w2 is None:
            scales[0] = torch.ones_like(scales[0])
        return _norm64(h, wide(s["w_pre"]), s["wb"], s["eps"]), h, torch.stack(scales)
    if case["op"] == "block_vjp":  # by differentiation of the definition
        leaf = lambda t: None if t is None else wide(t).requires_grad_()  # noqa: E731
        y, h, w2, w1, gate = (leaf(s[k]) for k in ("y", "h", "w_post", "w_pre", "gate"))
        value = (_norm64(h, w1, s["wb"], s["eps"]) * wide(s["g_out"])).sum()
        if s["g_res"] is not None:
            value = value + (h * wide(s["g_res"])).sum()
        g_h, gw_pre = torch.autograd.grad(value, [h, w1])
        joined = _joined64(y, torch.zeros_like(g_h), w2, gate, s)
        leaves = [t for t in (y, w2, gate) if t is not None]
        grads = list(torch.autograd.grad((joined * g_h).sum(), leaves))
        g_y = grads.pop(0)
        gw_post = grads.pop(0) if w2 is not None else None
        return g_y, g_h, gw_post, gw_pre, grads.pop(0) if gate is not None else None

    def turned(x, sign):  # pairs as complex numbers
        x, rot = wide(x), s["rot"]
        angle = sign * s["positions"].double()[:, None] * s["inv_freq"].to(DEVICE)[None, :]
        by = torch.polar(torch.full_like(angle, s["attn_scale"]), angle)[:, None, :]
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
    k_cache, v_cache = wide(s["k_cache"]), wide(s["v_cache"])
    k_cache[s["slots"][kept]] = turned(s["k"], 1.0)[kept]
    v_cache[s["slots"][kept]] = wide(s["v"])[kept]
    return turned(s["q"], 1.0), k_cache, v_cache
