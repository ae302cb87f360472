"""Values in 8 bits against their definitions in 64 bits, shared by the tests of the
8-bit norm and cache.

A code c of a value t (64 bits, in units of the scale) may be off by half a step of the
code's grid at t, and by what the kernel's fp32 t is off: each test says how much.
"""
import torch

U = 2.0 ** -24  # half a step of fp32
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
FLOOR = 2.0 ** -126


def half_step(t, fmt):
    """Half the distance between the codes around |t|."""
    if fmt == torch.int8:
        return torch.full_like(t, 0.5)
    e = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))  # three bits of fraction
    return torch.exp2(e - 4.0)


def check_codes(name, codes, t, off):
    """codes [.., n] of the values t, off their kernel's error in t's units."""
    fmt = codes.dtype
    c = codes.double()
    assert torch.isfinite(c).all() and c.abs().max() <= TOP[fmt] if c.numel() else True
    allow = half_step(t.abs() + off, fmt) + off
    far = (c - t).abs() - allow
    assert not c.numel() or far.max() <= 0, (name, far.max())


def units(x, fmt):
    """The scale of x's last dimension, 64 bits."""
    return (x.abs().amax(-1) / TOP[fmt]).clamp(min=FLOOR)


def grouped(x, group):
    """[rows, D] -> [rows, groups, group or D], the last group filled up with zeros."""
    G = group or x.shape[-1]
    n = -(-x.shape[-1] // G)
    return torch.nn.functional.pad(x, (0, n * G - x.shape[-1])).view(*x.shape[:-1], n, G)
