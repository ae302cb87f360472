"""rope_frequencies against hand-worked values, and the refusals of the rotary
and cache entry points that come before any CUDA call."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
A = 1 << 36


@pytest.fixture(scope="module", autouse=True)
def lib():
    from rmsnorm_fwd_bwd_add_gb300 import _native, build
    build.build()
    return _native.lib()


def test_plain_linear_and_ntk():
    f, s = rn.rope_frequencies(8, 10000.0)
    assert s == 1.0 and np.allclose(f.numpy(), [1, 0.1, 0.01, 0.001], rtol=1e-15)
    g, s = rn.rope_frequencies(8, 10000.0, "linear", factor=4.0)
    assert s == 1.0 and np.allclose(g.numpy(), f.numpy() / 4, rtol=1e-15)
    g, s = rn.rope_frequencies(8, 10000.0, "ntk", factor=8.0)
    # base 10000 * 8^(8/6) = 160000: the slowest pair is stretched 8 times, the fastest not
    assert s == 1.0 and np.allclose(g.numpy(), [1, 0.05, 0.0025, 0.000125], rtol=1e-13)
    assert rn.rope_frequencies(2, 10000.0, "ntk", factor=8.0)[0].tolist() == [1.0]


def test_yarn_ramp():
    r, base, n = 64, 10000.0, 4096.0
    g, s = rn.rope_frequencies(r, base, "yarn", factor=16.0, trained_length=n)
    f = base ** (-2.0 * np.arange(r // 2) / r)
    assert s == np.float32(0.1 * math.log(16.0) + 1)
    # pairs that turn more than 32 times over 4096 positions keep their frequency: index
    # below floor(64 ln(4096 / (64 pi)) / (2 ln 10000)) = floor(10.47) = 10; those beyond
    # ceil(64 ln(4096 / (2 pi)) / (2 ln 10000)) = ceil(22.51) = 23 are divided by 16
    ramp = np.clip((np.arange(r // 2) - 10.0) / 13.0, 0, 1)
    assert np.allclose(g.numpy(), f * (1 - ramp) + f / 16 * ramp, rtol=1e-14)
    same = rn.rope_frequencies(r, base)[0].numpy()  # the host's own powers, bit for bit
    assert np.array_equal(g.numpy()[:11], same[:11]) and np.allclose(g.numpy()[23:], same[23:] / 16, rtol=1e-15)


def test_llama3_ramp():
    g, s = rn.rope_frequencies(128, 500000.0, "llama3", factor=8.0, trained_length=8192.0)
    f = 500000.0 ** (-2.0 * np.arange(64) / 128)
    assert s == 1.0
    for i in range(64):
        turns = 8192.0 * f[i] / (2 * math.pi)
        want = f[i] if turns >= 4 else f[i] / 8 if turns <= 1 else \
            (1 - (turns - 1) / 3) * f[i] / 8 + (turns - 1) / 3 * f[i]
        assert abs(g[i].item() - want) <= 1e-14 * want
    assert 0 < sum(1 for i in range(64) if f[i] / 8 < g[i] < f[i]) < 64


def test_frequency_refusals():
    for kw in (dict(scaling="other"), dict(rot_dim=7), dict(rot_dim=0)):
        with pytest.raises(ValueError):
            rn.rope_frequencies(**{"rot_dim": 8, **kw})
    for kw in (dict(base=0.0), dict(base=float("nan")), dict(scaling="linear", factor=0.0),
               dict(scaling="yarn", factor=2.0), dict(scaling="llama3", factor=2.0, trained_length=100, low=4.0, high=4.0),
               dict(scaling="yarn", factor=2.0, trained_length=100, low=40.0), dict(rot_dim=2048),
               dict(scaling="yarn", factor=2.0, trained_length=100, base=1.0)):
        with pytest.raises(rn.RmsnormError):
            rn.rope_frequencies(**{"rot_dim": 8, **kw})


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def rope(lib, q=A, qs=(0, 128, 16), k=2 * A, ks=(0, 64, 16), pos=3 * A, qo=4 * A, qos=(0, 128, 16), ko=5 * A,
         kos=(0, 64, 16), inv=(1.0, 0.5), scale=1.0, B=1, S=10, Hq=8, Hkv=4, Dh=16, rot=4, dtype=1):
    f = (ctypes.c_double * len(inv))(*inv) if inv is not None else None
    return lib.rmsnorm_rope(q, strides(*qs), k, strides(*ks), pos, qo, strides(*qos), ko, strides(*kos), f, scale,
                            0, 0, B, S, Hq, Hkv, Dh, rot, dtype, None)


def test_rope_refusals(lib):
    import torch
    bad = [dict(dtype=3), dict(B=-1), dict(S=-1), dict(Hq=-1), dict(Dh=0), dict(rot=0), dict(rot=3), dict(rot=18),
           dict(inv=None), dict(inv=(1.0, float("nan"))), dict(inv=(1e7, 1.0)), dict(scale=float("inf")), dict(pos=None),
           dict(q=None), dict(ko=None), dict(q=A + 1), dict(qs=(0, -1, 16)),
           dict(qos=(0, 128, 8)), dict(qos=(0, 64, 16)), dict(kos=(0, 0, 16)), dict(qos=(0, 16, 0)),  # q_out on itself
           dict(qo=A + 64), dict(qo=2 * A), dict(ko=4 * A), dict(ko=A), dict(qo=3 * A), dict(ko=3 * A - 64),
           # heads of one projection, in place, but q_out one head too far on
           dict(q=A, qs=(0, 192, 16), k=A + 256, ks=(0, 192, 16), qo=A + 32, qos=(0, 192, 16), ko=A + 256,
                kos=(0, 192, 16)),
           dict(qo=A, qos=(0, 192, 16))]
    for kw in bad:
        assert rope(lib, **kw) == 1, kw
    assert rope(lib, Dh=2048) == 2 and rope(lib, S=1 << 50) == 2 and rope(lib, Hq=1 << 20) == 2
    assert rope(lib, qs=(0, 1 << 60, 16)) == 2
    assert rope(lib, S=0, q=None, qo=None) == 0
    if torch.cuda.is_available():
        return  # what follows is accepted and would launch on made-up addresses
    fused = dict(q=A, qs=(0, 192, 16), k=A + 256, ks=(0, 192, 16))
    ok = [dict(), dict(qo=A, ko=2 * A), dict(Hkv=0, k=None, ko=None), dict(Hq=0, q=None, qo=None), dict(qs=(0, 0, 0)),
          dict(**fused), dict(**fused, qo=A, qos=(0, 192, 16), ko=A + 256, kos=(0, 192, 16)),
          # heads before tokens, two batches of one buffer, in place
          dict(B=2, q=A, qs=(2400, 16, 160), k=A + 2 * 1280, ks=(2400, 16, 160), qo=A, qos=(2400, 16, 160),
               ko=A + 2 * 1280, kos=(2400, 16, 160))]
    for kw in ok:
        assert rope(lib, **kw) == 3, kw  # reaches the device query


def append(lib, q=A, k=2 * A, v=3 * A, pos=4 * A, slots=5 * A, qo=6 * A, kc=7 * A, kcs=(64, 16), vc=8 * A,
           vcs=(64, 16), T=10, N=100, Hkv=4, dtype=0):
    f = (ctypes.c_double * 8)(*[1.0] * 8)
    return lib.rmsnorm_rope_kv_append_ex(q, strides(128, 16), k, strides(64, 16), v, strides(64, 16), pos, slots, qo,
                                         strides(128, 16), kc, strides(*kcs), vc, strides(*vcs), f, 1.0, 0, T, 8,
                                         Hkv, 16, 16, N, dtype, None)


def test_append_refusals(lib):
    import torch
    for kw in (dict(v=None), dict(slots=None), dict(kc=None), dict(N=-1), dict(vc=7 * A), dict(vc=7 * A + 128),
               dict(kc=2 * A), dict(kc=A - 64), dict(vc=3 * A + 1280 - 2), dict(kc=6 * A), dict(kc=4 * A), dict(vc=5 * A),
               dict(kcs=(60, 16)), dict(kcs=(64, 8)), dict(qo=2 * A)):
        assert append(lib, **kw) == 1, kw
    assert append(lib, T=0, q=None) == 0
    if not torch.cuda.is_available():
        assert append(lib) == 3
        assert append(lib, kcs=(128, 16), vcs=(128, 16), vc=7 * A + 128) == 3  # K and V rows interleaved


def plan(lib, lens=A, new=2 * A, table=3 * A, ld=10, W=10, bs=16, free=4 * A, fc=5 * A, N=100, lo=6 * A, fo=7 * A,
         st=8 * A, pos=9 * A, slots=10 * A, req=11 * A, gr=12 * A, B=8, T=64):
    return lib.rmsnorm_kv_plan(lens, new, table, ld, W, bs, free, fc, N, lo, fo, st, pos, slots, req, gr, B, T, None)


def release(lib, lens=A, fin=2 * A, table=3 * A, ld=10, W=10, bs=16, free=4 * A, fc=5 * A, N=100, lo=6 * A, fo=7 * A,
            B=8):
    return lib.rmsnorm_kv_release(lens, fin, table, ld, W, bs, free, fc, N, lo, fo, B, None)


def test_plan_and_release_refusals(lib):
    import torch
    for kw in (dict(B=-1), dict(T=-1), dict(bs=0), dict(ld=9), dict(W=-1), dict(N=-1), dict(fc=None), dict(fo=None),
               dict(free=None), dict(st=None), dict(pos=None), dict(slots=None), dict(req=None), dict(gr=None),
               dict(lens=None), dict(new=None), dict(lo=None), dict(table=None), dict(lens=A + 2), dict(st=8 * A + 4),
               dict(lo=2 * A), dict(lo=A + 4), dict(table=4 * A), dict(fo=4 * A), dict(pos=10 * A), dict(req=9 * A + 8),
               dict(gr=8 * A), dict(slots=3 * A - 8)):
        assert plan(lib, **kw) == 1, kw
    for kw in (dict(B=-1), dict(bs=-3), dict(ld=9), dict(fc=None), dict(free=None), dict(fin=None), dict(lo=3 * A),
               dict(lo=A + 4), dict(fo=4 * A + 16), dict(lo=2 * A), dict(free=3 * A), dict(fo=5 * A + 1)):
        assert release(lib, **kw) == 1, kw
    assert plan(lib, T=1 << 31) == 2 and plan(lib, B=1 << 31) == 2 and release(lib, N=1 << 31) == 2
    if not torch.cuda.is_available():
        assert plan(lib) == 3 and plan(lib, lo=A, fo=5 * A) == 3 and release(lib, lo=A, fo=5 * A) == 3
        assert plan(lib, free=None, fc=None, fo=None, N=0) == 3


def test_python_refuses_cpu_tensors():
    import torch
    q = torch.zeros(2, 2, 8)
    inv, _ = rn.rope_frequencies(8)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_rope(q, None, torch.zeros(2, dtype=torch.int64), inv)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_kv_plan(lens, lens, torch.zeros(2, 2, dtype=torch.int32), 16, 4)


PLAN = r"""
#include <cstdio>
#include "rope_plan.h"
using namespace rmsn;
// Every head length has a plan of its own choosing: a power of two of warps a token, and
// at most 12 steps a head, or as few as a warp's 32 lanes allow.
int main() {
    for (int lanes = 1; lanes <= 520; ++lanes)
        for (long T : {1, 7, 300, 2432, 2433, 4096, 5001, 100000})
            for (int heads : {1, 3, 40, 130})
                for (int in_flight : {4, 8}) {
                    const RopePlan p = make_rope_plan(T, lanes, heads, in_flight, 304, 8);
                    const int least = (lanes + 31) / 32, steps = p.cw > 0 ? (lanes + p.cw - 1) / p.cw : 0;
                    const long rest = T - p.whole;
                    if (p.cw < 1 || p.cw > 32 || steps > (least > 12 ? least : 12) || p.wpt < 1 || p.wpt > 16 ||
                        (p.wpt & (p.wpt - 1)) || p.whole < 0 || rest < 0 || rest >= 2432 || p.grid < 1 || p.grid > 304) {
                        printf("lanes %d T %ld heads %d in flight %d: %d units a step, %d warps a token, grid %d", lanes, T,
                               heads, in_flight, p.cw, p.wpt, p.grid);
                        return 1;
                    }
                }
    return 0;
}
"""


def test_every_head_length_has_a_plan(tmp_path):
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PLAN)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-std=c++17", "-O2", "-I" + os.path.join(root, "rmsnorm_fwd_bwd_add_gb300", "csrc"), "-o",
                    str(exe), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
