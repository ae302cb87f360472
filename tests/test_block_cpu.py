"""Host-side answers of rmsnorm_block_fwd and rmsnorm_block_vjp, and the row
split and partial-sum slots their kernels share, without a GPU."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 32  # made-up addresses, far apart


@pytest.fixture(scope="module")
def lib():
    from rmsnorm_fwd_bwd_add_gb300 import _native, build
    build.build()
    return _native.lib()


def fwd(lib, y=A, ld=64, res=2 * A, w_post=3 * A, w_pre=4 * A, gate=None, ld_gate=64, G=0, scale=1.0, eps=1e-6,
        wb=0.0, out=5 * A, ld_out=64, nr=6 * A, rstd=None, rows=8, D=64, dtype=1):
    return lib.rmsnorm_block_fwd(y, ld, res, ld, w_post, w_pre, gate, ld_gate, G, scale, eps, wb, out, ld_out, nr,
                                 ld, rstd, rows, D, dtype, None)


def vjp(lib, y=A, h=2 * A, w_post=3 * A, w_pre=4 * A, gate=None, ld_gate=64, G=0, scale=1.0, g=5 * A, gr=6 * A,
        rstd=None, eps=1e-6, gy=7 * A, gh=8 * A, gw_post=9 * A, gw_pre=10 * A, g_gate=None, rows=8, D=64, ld=64):
    return lib.rmsnorm_block_vjp(y, ld, h, ld, w_post, w_pre, gate, ld_gate, G, scale, g, ld, gr, ld, rstd, eps,
                                 0.0, gy, ld, gh, ld, gw_post, gw_pre, g_gate, rows, D, 1, None)


def test_block_fwd_refusals(lib):
    for kw in (dict(dtype=3), dict(D=0), dict(rows=-1), dict(eps=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(wb=float("inf")), dict(w_pre=None), dict(y=None), dict(res=None),
               dict(out=None), dict(nr=None), dict(ld=63), dict(ld_out=63),
               dict(gate=11 * A, G=0), dict(gate=11 * A, G=3), dict(gate=11 * A, G=-1),
               dict(gate=11 * A, G=2, ld_gate=63), dict(y=A + 1), dict(w_pre=4 * A + 1), dict(rstd=7 * A + 2),
               dict(nr=5 * A), dict(out=A + 2), dict(nr=2 * A + 128), dict(out=3 * A), dict(out=4 * A + 64),
               dict(gate=11 * A, G=1, out=11 * A), dict(rstd=A + 64), dict(rstd=5 * A + 128), dict(rstd=3 * A),
               dict(gate=11 * A, G=8, rstd=11 * A + 512)):
        assert fwd(lib, **kw) == 1, kw
    assert fwd(lib, D=(1 << 24) + 1, ld=1 << 25, ld_out=1 << 25) == 2
    assert fwd(lib, rows=1 << 40, ld=1 << 40, D=1 << 20) == 2
    assert fwd(lib, rows=0, y=None, out=None) == 0


def test_block_vjp_refusals(lib):
    for kw in (dict(gw_pre=None), dict(gw_post=None), dict(w_post=None), dict(g_gate=11 * A),
               dict(gate=12 * A, G=1), dict(g=None), dict(h=None), dict(gy=None), dict(gh=7 * A),
               dict(gy=A + 2), dict(gh=6 * A + 128), dict(gy=3 * A), dict(gw_pre=9 * A + 64),
               dict(gw_pre=A + 64), dict(gw_post=4 * A), dict(rstd=9 * A), dict(gw_pre=10 * A + 2),
               dict(gate=12 * A, G=2, g_gate=12 * A), dict(gate=12 * A, G=8, g_gate=8 * A + 256),
               dict(ld=60)):
        assert vjp(lib, **kw) == 1, kw
    assert vjp(lib, rows=0, gate=12 * A, G=1 << 58, g_gate=13 * A) == 2


SPLIT = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "block.h"
using namespace rmsn;
int main() {
    srand(1);
    for (int it = 0; it < 20000; ++it) {
        const int64_t G = 1 + rand() % 40, rpg = 1 + rand() % 50, rows = G * rpg;
        const int64_t grid = 1 + rand() % (rows < 60 ? rows : 60), q = rows / grid, r = rows % grid;
        std::vector<int> written(2 * grid, -1);
        if (first_row(0, q, r) != 0 || first_row(grid, q, r) != rows) return 1;
        // the second stage's own arithmetic: the CTA that takes row i
        auto cta_of = [&](int64_t i) { return i < r * (q + 1) ? i / (q + 1) : r + (i - r * (q + 1)) / q; };
        for (int64_t c = 0; c < grid; ++c) {
            const int64_t r0 = first_row(c, q, r), r1 = first_row(c + 1, q, r);
            if (r1 <= r0) return 2;
            for (int64_t i = r0; i < r1; ++i) {
                if (cta_of(i) != c || gate_row(i, rpg) != i / rpg) return 3;
                const int64_t gr = i / rpg;
                if (gr * rpg >= r0 && (gr + 1) * rpg <= r1) continue;  // whole
                const int64_t s = mid_slot(c, gr, q, r, rpg);
                if (s < 0 || s >= 2 * grid || (written[s] != -1 && written[s] != gr)) return 4;
                written[s] = (int)gr;
            }
        }
        for (int64_t gr = 0; gr < G; ++gr) {  // the second stage finds every part
            const int64_t c0 = cta_of(gr * rpg), c1 = cta_of((gr + 1) * rpg - 1);
            if (c0 == c1) continue;
            if (written[mid_slot(c0, gr, q, r, rpg)] != gr) return 5;
            for (int64_t c = c0 + 1; c <= c1; ++c) {
                if (written[2 * c] != gr) return 6;
                written[2 * c] = -1;
            }
            written[mid_slot(c0, gr, q, r, rpg)] = -1;
        }
        for (int w : written) if (w != -1) return 7;  // and no part is left over
        const int64_t big = ((int64_t)1 << 40) + rand(), per = 1 + rand();
        if (gate_row(big, per) != big / per) return 8;
    }
    return 0;
}
"""


def test_row_split_and_partial_slots(tmp_path):
    src, exe = tmp_path / "split.cu", tmp_path / "split"
    src.write_text(SPLIT)
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-std=c++17", "-I" + os.path.join(ROOT, "rmsnorm_fwd_bwd_add_gb300", "csrc"), "-o",
                    str(exe), str(src)], check=True, capture_output=True)
    assert subprocess.run([str(exe)]).returncode == 0
