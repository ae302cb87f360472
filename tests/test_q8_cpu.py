"""The axes of pairs, and the refusals of the 8-bit norm, the rotary axes and the 8-bit
cache that come before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

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


def on_gpu():
    import torch
    return torch.cuda.is_available()  # accepted calls would launch on made-up addresses


def test_sections():
    import torch
    assert rn.rope_sections((2, 3, 1)).tolist() == [0, 0, 1, 1, 1, 2]
    assert rn.rope_sections([2, 3, 1], in_turn=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert rn.rope_sections((24, 20, 20), in_turn=True).tolist() == [0, 1, 2] * 20 + [0] * 4
    assert rn.rope_sections((0, 2)).tolist() == [1, 1] and rn.rope_sections((3,)).dtype == torch.int32
    for bad in ((), (0, 0), (1, -1), (1, 1, 1, 1, 1)):
        with pytest.raises(ValueError):
            rn.rope_sections(bad)


def q8(lib, x=A, ld_x=64, res=2 * A, ld_r=64, w=3 * A, eps=1e-6, wb=0.0, out=4 * A, ld_o=64, scale=5 * A, group=0,
       nr=6 * A, ld_n=64, rows=10, D=64, dtype=1):
    return lib.rmsnorm_fwd_q8(x, ld_x, res, ld_r, w, eps, wb, out, ld_o, scale, group, nr, ld_n, rows, D, dtype, None)


def test_norm_refusals(lib):
    for kw in (dict(dtype=3), dict(D=0), dict(rows=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(wb=float("inf")),
               dict(group=1), dict(group=-32), dict(group=256), dict(w=None), dict(x=None), dict(out=None), dict(scale=None),
               dict(res=None), dict(nr=None), dict(ld_x=63), dict(ld_r=63), dict(ld_o=63), dict(ld_n=0), dict(x=A + 1),
               dict(w=3 * A + 1), dict(scale=5 * A + 2), dict(nr=6 * A + 1),
               dict(out=A), dict(out=A + 1279), dict(out=2 * A), dict(out=3 * A), dict(out=6 * A), dict(scale=A),
               dict(scale=4 * A + 636), dict(scale=6 * A), dict(scale=3 * A), dict(nr=A + 128), dict(nr=2 * A - 128),
               dict(nr=3 * A), dict(scale=2 * A + 1276), dict(group=32, scale=6 * A - 76)):
        assert q8(lib, **kw) == 1, kw
    assert q8(lib, D=(1 << 24) + 1) == 2 and q8(lib, rows=1 << 62) == 2 and q8(lib, ld_o=1 << 62, rows=1 << 40) == 2
    assert q8(lib, rows=0, x=None, out=None, scale=None) == 0
    if on_gpu():
        return
    for kw in (dict(), dict(nr=A), dict(nr=2 * A), dict(res=None, nr=None), dict(out=4 * A + 1, ld_o=65), dict(group=32),
               dict(rows=1, ld_x=0, ld_o=0, ld_r=0, ld_n=0), dict(ld_x=100, ld_n=100, nr=A), dict(scale=4 * A + 640),
               # x and residual side by side in one buffer, updated in place
               dict(ld_x=128, ld_r=128, res=A + 128, nr=A + 128, ld_n=128)):
        assert q8(lib, **kw) == 3, kw


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def axes_of(of):
    return None if of is None else (ctypes.c_int32 * len(of))(*of)


def rope(lib, q=A, qs=(0, 128, 16), k=2 * A, ks=(0, 64, 16), pos=3 * A, axes=2, of=(0, 1), qo=4 * A, qos=(0, 128, 16),
         ko=5 * A, kos=(0, 64, 16), inv=(1.0, 0.5), scale=1.0, B=1, S=10, Hq=8, Hkv=4, Dh=16, rot=4, dtype=1):
    f = (ctypes.c_double * len(inv))(*inv) if inv is not None else None
    return lib.rmsnorm_rope_axes(q, strides(*qs), k, strides(*ks), pos, axes, axes_of(of), qo, strides(*qos), ko,
                                 strides(*kos), f, scale, 0, 0, B, S, Hq, Hkv, Dh, rot, dtype, None)


def test_rope_axes_refusals(lib):
    for kw in (dict(axes=0), dict(axes=-1), dict(of=None), dict(of=(0, 2)), dict(of=(-1, 0)), dict(dtype=3), dict(rot=3),
               dict(inv=None), dict(pos=None), dict(q=None), dict(qo=3 * A + 88), dict(qo=3 * A), dict(ko=A), dict(B=-1),
               # the second axis' positions in an output
               dict(ko=3 * A + 120), dict(axes=1, of=(0, 1))):
        assert rope(lib, **kw) == 1, kw
    assert rope(lib, axes=5) == 2 and rope(lib, Dh=2048) == 2
    assert rope(lib, S=0, q=None, qo=None) == 0
    if on_gpu():
        return
    for kw in (dict(), dict(axes=1, of=None), dict(axes=1, of=(0, 0)), dict(axes=4, of=(3, 0)), dict(qo=A, ko=2 * A),
               dict(Hkv=0, k=None, ko=None), dict(ko=3 * A + 160)):
        assert rope(lib, **kw) == 3, kw


def append(lib, q=A, qs=(128, 16), k=2 * A, ks=(64, 16), v=3 * A, vs=(64, 16), pos=4 * A, axes=1, of=None, slots=5 * A,
           qo=6 * A, qos=(128, 16), kc=7 * A, kcs=(64, 16), vc=8 * A, vcs=(64, 16), ksc=9 * A, kss=(4, 1), vsc=10 * A,
           vss=(4, 1), T=10, Hq=8, Hkv=4, N=100, fmt=1, dtype=1):
    return lib.rmsnorm_kv_append(q, strides(*qs), k, strides(*ks), v, strides(*vs), pos, axes, axes_of(of), slots, qo,
                                 strides(*qos), kc, strides(*kcs), vc, strides(*vcs), ksc, strides(*kss), vsc,
                                 strides(*vss), (ctypes.c_double * 2)(1.0, 0.5), 1.0, 0, T, Hq, Hkv, 16, 4, N, fmt, dtype,
                                 None)


PACKED = dict(kcs=(160, 16), vc=7 * A + 64, vcs=(160, 16), ksc=7 * A + 128, kss=(40, 1), vsc=7 * A + 144, vss=(40, 1))


def test_append_refusals(lib):
    for kw in (dict(fmt=3), dict(fmt=-1), dict(dtype=3), dict(N=-1), dict(axes=0), dict(axes=2), dict(pos=None),
               dict(slots=None), dict(kc=None), dict(vc=None), dict(ksc=None), dict(vsc=None), dict(v=None), dict(qo=None),
               dict(kcs=(60, 16)), dict(kcs=(64, 8)), dict(kss=(3, 1)), dict(kss=(4, 0)), dict(ksc=9 * A + 2),
               dict(vc=7 * A), dict(vc=7 * A + 6399), dict(vsc=9 * A), dict(ksc=7 * A), dict(ksc=8 * A + 6396),
               dict(kc=A), dict(kc=2 * A + 1279), dict(vc=3 * A), dict(kc=6 * A), dict(ksc=A), dict(vsc=6 * A),
               dict(kc=4 * A), dict(ksc=5 * A - 1596), dict(qo=4 * A), dict(qo=2 * A), dict(qo=A + 32),
               dict(axes=2, of=(0, 1), ksc=4 * A + 156), dict(**{**PACKED, "ksc": 7 * A + 124}),
               dict(**{**PACKED, "vsc": 7 * A + 140}), dict(fmt=0), dict(fmt=0, ksc=None)):
        assert append(lib, **kw) == 1, kw
    assert append(lib, axes=5, of=(0, 0)) == 2
    assert append(lib, T=0, q=None) == 0
    if on_gpu():
        return
    for kw in (dict(), dict(fmt=2), dict(fmt=0, ksc=None, vsc=None), PACKED, dict(N=0, kc=None, vc=None, ksc=None, vsc=None),
               dict(qo=A), dict(axes=2, of=(0, 1), ksc=4 * A + 160), dict(Hkv=0, k=None, v=None),
               dict(kcs=(16, 1600), kss=(1, 100)), dict(vc=7 * A + 6400), dict(vsc=9 * A + 1600)):
        assert append(lib, **kw) == 3, kw


def read(lib, kc=A, kcs=(64, 16), vc=2 * A, vcs=(64, 16), ksc=3 * A, kss=(4, 1), vsc=4 * A, vss=(4, 1), slots=5 * A,
         ko=6 * A, kos=(64, 16), vo=7 * A, vos=(64, 16), T=10, Hkv=4, Dh=16, N=100, fmt=1, dtype=1):
    return lib.rmsnorm_kv_read(kc, strides(*kcs), vc, strides(*vcs), ksc, strides(*kss), vsc, strides(*vss), slots, ko,
                               strides(*kos), vo, strides(*vos), T, Hkv, Dh, N, fmt, dtype, None)


def test_read_refusals(lib):
    for kw in (dict(fmt=0), dict(fmt=3), dict(dtype=3), dict(T=-1), dict(Hkv=-1), dict(Dh=0), dict(N=-1), dict(kc=None),
               dict(vsc=None), dict(slots=None), dict(ko=None), dict(vo=None), dict(kos=(63, 16)), dict(kos=(64, 15)),
               dict(kcs=(-1, 16)), dict(ksc=3 * A + 1), dict(ko=6 * A + 1), dict(vo=6 * A), dict(ko=7 * A + 1278),
               dict(ko=A + 6398), dict(vo=2 * A), dict(ko=3 * A), dict(vo=4 * A + 1596), dict(ko=5 * A)):
        assert read(lib, **kw) == 1, kw
    assert read(lib, Dh=2000) == 2 and read(lib, T=1 << 50) == 2 and read(lib, Hkv=1 << 20) == 2
    assert read(lib, T=0, kc=None) == 0 and read(lib, Hkv=0, ko=None) == 0
    if on_gpu():
        return
    for kw in (dict(), dict(fmt=2), dict(N=0, kc=None, vc=None, ksc=None, vsc=None), dict(kcs=(0, 0), kss=(0, 0)),
               dict(vc=A, vsc=3 * A), dict(kos=(128, 16), vos=(128, 16), vo=6 * A + 128)):
        assert read(lib, **kw) == 3, kw


def test_python_refuses_cpu_tensors():
    import torch
    q = torch.zeros(2, 2, 8)
    inv, _ = rn.rope_frequencies(8)
    i64 = torch.zeros(2, dtype=torch.int64)
    c, s = torch.zeros(4, 2, 8, dtype=torch.int8), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_fwd_q8(torch.zeros(2, 8), torch.ones(8), 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_rope_axes(q, None, i64.view(2, 1).expand(2, 2), inv, rn.rope_sections((2, 2)))
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_kv_append(q, q, q, i64, i64, c, c, inv, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rmsnorm_kv_read(c, c, s, s, i64)


def run_host(tmp_path, text):
    """Compiles and runs a host program against the plans' headers."""
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(text)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O1", "-I" + os.path.join(root, "include"),
                    "-I" + os.path.join(root, "rmsnorm_fwd_bwd_add_gb300", "csrc"), "-o", str(exe), str(src)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_norm_plans(tmp_path):
    """Every plan is one that the kernels take: a row's units have threads, its single
    columns too, rings fit an SM's shared memory beside the static sums, a CTA's rows
    stand alike."""
    run_host(tmp_path, r"""
#include <cstdio>
#include "norm_q8.h"
using namespace rmsn;
int main() {
    const long lengths[] = {1, 7, 8, 15, 16, 17, 63, 64, 255, 256, 257, 1000, 1024, 1032, 2047, 2048, 2056, 4096, 4097, 4104, 5120,
                            8192, 8193, 8200, 12288, 16384, 16385, 16392, 20000, 1L << 20, 1L << 24};
    for (long D : lengths)
        for (long rows : {1, 2, 5, 152, 153, 303, 304, 305, 607, 609, 1216, 1217, 4000, 100000})
            for (int es : {2, 4})
                for (int res = 0; res < 4; ++res)  // bit 1: in groups
                    for (int classes : {0, 1, 2, 4, 8})
                        for (int aligned = 0; aligned < 2; ++aligned) {
                            if (aligned && classes != 1) continue;
                            const Q8Plan p = make_q8_plan(rows, D, es, res & 1, res & 2 ? 64 : 0, classes, aligned, 152);
                            const long E = 16 / es, units = D / E;
                            bool ok = q8_plan_ok(p) && p.grid <= rows;
                            const bool held = p.kind == Q8_DIRECT || p.kind == Q8_STAGED;
                            if (p.kind == Q8_WARP) ok = ok && !p.shift && D % E == 0 && units <= 32 * p.units && aligned;
                            if (held) ok = ok && units >= 2 && units <= (long)p.threads * p.units && classes > 0;
                            // up to E - 1 columns before the units and as many behind
                            if (held && p.shift) ok = ok && p.threads >= 2 * (E - 1);
                            if (held && !p.shift) ok = ok && aligned && D % E == 0;
                            if (p.kind == Q8_DIRECT) ok = ok && p.grid == rows;
                            if (p.kind == Q8_LONG) ok = ok && aligned && D % E == 0;
                            if (p.kind == Q8_STAGED) {
                                const long need = (p.shift ? D * es + 30 : D * es + 15) / 16 * 16;
                                const int cap = p.threads <= 128 ? 128 : p.threads <= 256 ? 256 : 512;
                                const long groups = p.shift ? 3 * 4 * (cap * p.units * E / 32 + 2) : 12;
                                const long fixed = groups + 2 * 8 * (cap / 32);
                                ok = ok && (long)p.stage_bytes >= need && p.stage_bytes % 16 == 0;
                                ok = ok && (long)p.smem == Q8_HEADER + (long)p.stages * (res & 1 ? 2 : 1) * p.stage_bytes;
                                ok = ok && (long)p.smem + fixed <= 227 * 1024 && p.stages * 8 <= Q8_HEADER;
                                const int per_sm = (p.grid + 151) / 152;
                                ok = ok && per_sm * ((long)p.smem + fixed + 1024) <= 228 * 1024 && per_sm * p.threads <= 512;
                                if (p.shift) ok = ok && p.grid % classes == 0;
                            }
                            if (!ok) {
                                printf("D %ld rows %ld es %d res %d classes %d aligned %d: kind %d threads %d units %d stages %d grid %d smem %zu",
                                       D, rows, es, res, classes, aligned, p.kind, p.threads, p.units, p.stages, p.grid, p.smem);
                                return 1;
                            }
                        }
    return 0;
}
""")


def test_cache_plans(tmp_path):
    """Every part of a token has heads, a head's lanes are a warp's, rings fit shared memory
    and hold what a step copies."""
    run_host(tmp_path, r"""
#include <cstdio>
#include "kv_append8.h"
using namespace rmsn;
template <int VB, int UPL> bool append_ok(long T, int Dh, int lanes, int Hq, int Hkv, int pairs, int es) {
    const int cw = (lanes + UPL - 1) / UPL;
    const Append8Plan p = make_append8_plan(T, cw, Hq, Hkv, 2, pairs, UPL, 152 * C8_CTAS_PER_SM, C8_NT / 32);
    const int hpi = 32 / cw, most = Hq > Hkv ? Hq : Hkv;
    bool ok = p.cw == cw && cw >= 1 && cw <= 32 && p.wpt >= 1 && (p.wpt & (p.wpt - 1)) == 0 && (p.wpt - 1) * hpi < most;
    ok = ok && p.grid >= 1 && p.grid <= 152 * C8_CTAS_PER_SM && p.whole >= 0 && p.whole <= T && T - p.whole < 152 * C8_CTAS_PER_SM * 8;
    const long step = append8_step_bytes<VB, UPL>(Dh * es, cw);
    if (VB < 16) ok = ok && step >= (long)hpi * ((Dh * es + 30) / 16 * 16);
    const long smem = (C8_NT / 32) * (append8_ring<VB, UPL, RMSNORM_CACHE_E4M3>() * step + 2 * append8_plane(2 * pairs) * 4);
    return ok && step % 16 == 0 && smem + 4608 <= 227 * 1024;
}
int main() {
    for (int Dh = 2; Dh <= 1024; ++Dh)
        for (long T : {1, 8, 300, 2432, 2433, 4096, 100000})
            for (int Hq : {0, 1, 5, 32, 130})
                for (int Hkv : {0, 1, 3, 8, 70}) {
                    if (Hq + Hkv == 0) continue;
                    const int pairs = Dh / 2, odd = (Dh + 1) / 2;
                    bool ok = true;
                    if (Dh % 16 == 0 && Dh / 16 <= 32) ok = ok && append_ok<16, 1>(T, Dh, Dh / 16, Hq, Hkv, pairs, 2);
                    if (Dh % 16 == 0) ok = ok && append_ok<16, 2>(T, Dh, Dh / 16, Hq, Hkv, pairs, 2);
                    if (Dh % 8 == 0 && Dh / 8 <= 64) ok = ok && append_ok<16, 2>(T, Dh, Dh / 8, Hq, Hkv, pairs, 4);
                    if (Dh % 8 == 0) ok = ok && append_ok<16, 4>(T, Dh, Dh / 8, Hq, Hkv, pairs, 4);
                    if ((Dh + 3) / 4 <= 128) ok = ok && append_ok<4, 4>(T, Dh, (Dh + 3) / 4, Hq, Hkv, pairs, 2);
                    if (odd <= 128) ok = ok && append_ok<2, 4>(T, Dh, odd, Hq, Hkv, pairs, 2) && append_ok<4, 4>(T, Dh, odd, Hq, Hkv, pairs, 4);
                    if (odd <= 256) ok = ok && append_ok<2, 8>(T, Dh, odd, Hq, Hkv, pairs, 2) && append_ok<4, 8>(T, Dh, odd, Hq, Hkv, pairs, 4);
                    if (Hkv)
                        for (int C : {1, 2, 4, 8}) {
                            if (Dh % C) continue;
                            const Read8Plan p = make_read8_plan(T, Dh / C, Hkv, 152, 4, 3, C8_NT / 32);
                            const int hpi = p.cw > 0 ? 32 / p.cw : 0;
                            ok = ok && p.cw >= 1 && p.cw <= 32 && p.cw <= Dh / C && p.wpt >= 1 && (p.wpt & (p.wpt - 1)) == 0 && p.grid >= 1;
                            ok = ok && (p.wpt == 1 || (p.wpt / 2) * hpi < Hkv) && (p.tokens == 1 || p.tokens * Hkv <= hpi);
                        }
                    if (!ok) {
                        printf("Dh %d T %ld heads %d + %d", Dh, T, Hq, Hkv);
                        return 1;
                    }
                }
    return 0;
}
""")


def test_every_head_has_lanes(tmp_path):
    """A head that is sent to an instance fits its lanes, whatever part of it turns."""
    run_host(tmp_path, r"""
#include <cstdio>
#include "kv_append8.h"
using namespace rmsn;
template <typename T, bool I> bool ok(int Dh, int rot) {
    constexpr int E = 16 / (int)sizeof(T);
    const int lanes = head_lanes<E, I>(Dh, rot);
    // whole vectors, as the dispatch asks for
    if (Dh % E || (I ? rot : rot / 2) % E) return true;
    if (!append8_vectors_fit<T, I>(Dh, rot)) return Dh > 1000;  // smaller units
    const int upl = lanes <= 32 * (8 / E) ? 8 / E : 16 / E, cw = (lanes + upl - 1) / upl;
    return cw >= 1 && cw <= 32;
}
int main() {
    int left = 0;
    for (int Dh = 2; Dh <= 1024; ++Dh)
        for (int rot = 2; rot <= Dh; rot += 2) {
            if (!(ok<__half, false>(Dh, rot) && ok<__half, true>(Dh, rot) && ok<float, false>(Dh, rot) && ok<float, true>(Dh, rot))) {
                printf("Dh %d rot %d", Dh, rot);
                return 1;
            }
            left += Dh == 1024 && rot % 8 == 0 && !append8_vectors_fit<__half, true>(Dh, rot);
        }
    printf("no head of 1024 with odd parts met");
    return left > 0 ? 0 : 1;
}
""")
