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


def test_block_fwd_takes_no_gate_rows_for_no_rows(lib):
    assert fwd(lib, rows=0, gate=11 * A, G=0) == 0 and fwd(lib, rows=0, gate=11 * A, G=3) == 0
    assert fwd(lib, rows=8, gate=11 * A, G=0) == 1 and fwd(lib, rows=0, gate=11 * A, G=-1) == 1


SPLIT = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "block_plan.h"
using namespace rmsn;

// Every row is one CTA's, and the second stage finds every part of every gate row.
int check(const BlockArgs &a, int64_t grid, int64_t G) {
    const int64_t rpg = a.rows_per_gate, q = a.split_q, r = a.split_r;
    std::vector<int> seen(a.rows, 0), written(2 * grid, -1);
    for (int64_t c = 0; c < grid; ++c) {
        const RowDeal d = vjp_rows(a, c);
        if (d.n < 1) return 1;
        for (int64_t seg = 0; seg < d.n;) {
            const int64_t gr = gate_row(d.row(seg), rpg);
            int64_t end = seg;
            for (; end < d.n && gate_row(d.row(end), rpg) == gr; ++end) ++seen[d.row(end)];
            if (end - seg != rpg) {
                const int64_t s = mid_slot(c, seg == 0);
                if (s < 0 || s >= 2 * grid || written[s] != -1) return 2;
                written[s] = (int)gr;
            }
            seg = end;
        }
        if (a.team && gate_row(d.row(0), rpg) != gate_row(d.row(d.n - 1), rpg)) return 3;
    }
    for (int n : seen) if (n != 1) return 4;
    for (int64_t gr = 0; gr < G; ++gr) {
        int64_t c0, c1;
        if (a.team) {
            c0 = split_first(gr, q, r);
            c1 = split_first(gr + 1, q, r) - 1;
        } else {
            c0 = split_part<int64_t>(gr * rpg, q, r);
            c1 = split_part<int64_t>(gr * rpg + rpg - 1, q, r);
        }
        if (c0 == c1) continue;
        for (int64_t c = c0; c <= c1; ++c) {
            const int64_t s = mid_slot(c, c > c0 || a.team || split_first(c0, q, r) / rpg == gr);
            if (written[s] != gr) return 5;
            written[s] = -1;
        }
    }
    for (int w : written) if (w != -1) return 6;  // and no part is left over
    return 0;
}

int main() {
    srand(1);
    for (int it = 0; it < 20000; ++it) {
        BlockArgs a{};
        const int64_t G = 1 + rand() % 40;
        a.rows_per_gate = 1 + rand() % 50;
        a.rows = G * a.rows_per_gate;
        const int64_t grid = 1 + rand() % (a.rows < 60 ? a.rows : 60);
        a.team = grid >= 8 * G && rand() % 2;
        a.rows_per_team = a.rows / G;
        a.split_q = a.team ? grid / G : a.rows / grid;
        a.split_r = a.team ? grid % G : a.rows % grid;
        if (split_first(0, a.split_q, a.split_r) != 0) return 10;
        auto runs = [&](int64_t rows, int64_t size) {  // rows of a team in runs of a.run CTAs
            a.run = 0;
            for (int k = 8; k > 1 && !a.run; k /= 2)
                if (size % k == 0 && rand() % 2) a.run = k;
            if (a.run) a.run_q = rows / (size / a.run), a.run_r = rows % (size / a.run);
        };
        if (a.team && grid % G == 0) runs(a.rows_per_team, grid / G);
        if (const int e = check(a, grid, G)) return 20 + e;
        // the forward's deal, in chunks
        a.team = rand() % 2;
        a.chunk_shift = rand() % 4;
        a.split_q = a.rows / grid;
        a.split_r = a.rows % grid;
        a.run = 0;
        if (a.team) runs(a.rows, grid);
        std::vector<int> seen(a.rows, 0);
        for (int64_t c = 0; c < grid; ++c) {
            const RowDeal d = fwd_rows(a, c, grid);
            for (int64_t i = 0; i < d.n; ++i) {
                if (d.row(i) < 0 || d.row(i) >= a.rows) return 30;
                if (a.run && (d.row(i) - d.row(0)) % a.run) return 33;  // alike rows only
                ++seen[d.row(i)];
            }
        }
        for (int n : seen) if (n != 1) return 31;
        const int64_t big = ((int64_t)1 << 40) + rand(), per = 1 + rand();
        if (gate_row(big, per) != big / per) return 32;
    }
    return 0;
}
"""

PLAN = r"""
#include <cstdio>
#include "block_plan.h"
using namespace rmsn;
int64_t lanes_units(const BlockPlan &p) { return (int64_t)p.threads * (p.half ? 1 : 2); }
int main() {
    const int sms[] = {1, 2, 132, 152};
    for (int64_t D = 1; D <= 40000; D += D < 1100 ? 1 : D < 9000 ? 7 : 61)
        for (int64_t rows : {1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 151, 300, 305, 1217, 5000, 16384, 1000000})
            for (int es : {2, 4})
                for (int vjp = 0; vjp < 2; ++vjp)
                    for (int sm : sms) {
                        const int asked = std::max(make_block_plan(rows, D, es, 16, 3, true, 2, sm, 0).grid,
                                                   make_block_plan(rows, D, es, es, 3, true, 2, sm, 1).grid);
                        for (int tensors = vjp ? 3 : 2; tensors <= (vjp ? 5 : 3); ++tensors)
                            for (int how = 0; how < 12; ++how)
                                for (int64_t gates : {(int64_t)1, (int64_t)5, rows}) {
                                    const int unit = 16 >> how / 3, classes = how % 3 == 0 ? 0 : how % 3 == 1 ? 1 : 8;
                                    if (unit < es || rows % gates) continue;
                                    const BlockPlan p =
                                        make_block_plan(rows, D, es, unit, tensors, vjp, gates, sm, classes);
                                    const char *why = nullptr;
                                    if (p.grid < 1 || p.grid > rows) why = "grid";
                                    if (vjp && !p.cluster && p.grid > asked) why = "more scratch than the size asked beforehand";
                                    if (p.kind != BLOCK_GENERIC) {
                                        const int64_t lanes = p.kind == BLOCK_WARP ? 32 : p.threads;
                                        const int per = p.half ? 16 : 32;
                                        if (p.threads < 32 || p.threads > 1024 || p.threads % 32) why = "threads";
                                        const int64_t width = p.shift ? D * es / 16 * 16 - 64 : D * es;
                                        if (lanes * per < width) why = "a row does not fit its threads";
                                        if ((D * es % p.ub && !p.shift) || (p.ub != 16 && p.ub != 4 && p.ub != 2)) why = "unit";
                                        if (p.half && (!vjp || p.kind != BLOCK_STAGED)) why = "half";
                                        if (p.half && p.threads > 640) why = "half's threads";
                                    }
                                    if (p.kind == BLOCK_STAGED) {
                                        if (p.stages < 1 || p.stages > 8) why = "stages";
                                        if (p.smem < 128 + (size_t)D * 4 +
                                                     (size_t)p.stages * tensors * p.stage_bytes) why = "ring";
                                        if (p.smem > 227 * 1024) why = "shared memory";
                                        if (p.stage_bytes % 16 || p.stage_bytes < D * es + (unit == 16 && D * es % 16 == 0 ? 0 : 15)) why = "stage";
                                        if (8 * p.stages > 128) why = "barriers";
                                    }
                                    if (p.kind == BLOCK_WARP && vjp &&
                                        p.smem != ((size_t)p.threads / 32 + (p.cluster ? 2 : 0)) * block_sum_bytes(D))
                                        why = "warps' rows";
                                    if (p.cluster) {
                                        if (!vjp || p.cluster > 8 || p.grid != p.cluster || p.team || p.smem > 227 * 1024)
                                            why = "cluster";
                                        if (p.kind == BLOCK_DIRECT && p.smem != 2 * block_sum_bytes(D)) why = "cluster's sums";
                                        if (p.kind != BLOCK_DIRECT && p.kind != BLOCK_WARP) why = "cluster's tier";
                                        // several gate rows, or rows that stand differently: a row a CTA
                                        if ((gates > 1 || (p.shift && classes > 1)) && p.grid != rows) why = "cluster's rows";
                                        if (p.kind == BLOCK_WARP && (rows + p.grid - 1) / p.grid > p.threads / 32) why = "cluster's warps";
                                    }
                                    if (p.kind != BLOCK_GENERIC && p.kind != BLOCK_WARP && p.shift &&
                                        D - std::min(D * es / 16 - 1, lanes_units(p)) * (16 / es) > p.threads)
                                        why = "threads for the ends";
                                    if (p.shift) {
                                        const int64_t teams = vjp ? gates : 1;
                                        if (p.ub != 16 || classes == 0 || p.kind == BLOCK_WARP || p.kind == BLOCK_GENERIC)
                                            why = "shift";
                                        if (p.kind == BLOCK_STAGED && classes > 1 && (!p.team || p.chunk_shift || p.grid % teams ||
                                                                       p.grid / teams % classes || p.grid / teams > rows / teams ||
                                                                       (p.run && p.run != classes)))
                                            why = "shift's teams";
                                    } else if (p.team && vjp && gates * 8 > p.grid) why = "team";
                                    if (p.kind == BLOCK_DIRECT && p.grid != rows && !p.cluster) why = "direct";
                                    if (p.kind == BLOCK_GENERIC && p.team) why = "generic team";
                                    if (p.chunk_shift && ((int64_t)p.grid << p.chunk_shift) > rows) why = "chunk";
                                    if (why) {
                                        printf("%s: rows %ld D %ld es %d vjp %d unit %d tensors %d gates %ld sm %d classes %d: kind %d grid %d "
                                               "threads %d stages %d\n", why, (long)rows, (long)D, es, vjp, unit, tensors,
                                               (long)gates, sm, classes, p.kind, p.grid, p.threads, p.stages);
                                        return 1;
                                    }
                                }
                    }
    return 0;
}
"""

LIMITS = r"""
#include <cstdio>
#include "block_plan.h"
using namespace rmsn;
// The widest CTA of the instance that a plan takes: its sums are two buffers of eight
// floats a warp in static shared memory, beside the ring and table asked for at launch.
int widest(const BlockPlan &p, bool vjp) {
    for (int t : {256, 320, 512, 640})
        if (p.threads <= t && (t % 320 || (vjp ? t == 640 && p.half : true))) return t;
    return 1024;
}
int main() {
    for (int es : {2, 4})
        for (int64_t D = 1; D <= 32768 / es; ++D)
            for (int64_t rows : {153, 400, 4000})
                for (int vjp = 0; vjp < 2; ++vjp)
                    for (int tensors = vjp ? 3 : 2; tensors <= (vjp ? 5 : 3); ++tensors)
                        for (int classes : {0, 1, 2, 4, 8})
                            for (int unit : {16, es}) {
                                const BlockPlan p = make_block_plan(rows, D, es, unit, tensors, vjp, 1, 152, classes);
                                if (p.kind == BLOCK_GENERIC) continue;
                                const size_t sums = p.kind == BLOCK_WARP ? 64 : 64 * widest(p, vjp) / 32;
                                if (p.smem + sums > 227 * 1024) {
                                    printf("rows %ld D %ld es %d vjp %d tensors %d unit %d classes %d: %zu + %zu bytes\n", (long)rows,
                                           (long)D, es, vjp, tensors, unit, classes, p.smem, sums);
                                    return 1;
                                }
                            }
    return 0;
}
"""

GUARD = r"""
#include <cstdio>
#include "block_plan.h"
using namespace rmsn;
int main() {
    auto refuses = [](BlockPlan p, void (*spoil)(BlockPlan &)) {
        if (!block_plan_ok(p)) return false;
        spoil(p);
        return !block_plan_ok(p);
    };
    const BlockPlan staged = make_block_plan(5000, 4096, 2, 16, 4, true, 1, 152, 1);
    const BlockPlan half = make_block_plan(5000, 5120, 2, 16, 4, true, 1, 152, 1);
    const BlockPlan shift = make_block_plan(5000, 4097, 2, 2, 4, true, 1, 152, 8);
    const BlockPlan warp = make_block_plan(5000, 512, 2, 16, 4, true, 1, 152, 1);
    const BlockPlan cluster = make_block_plan(8, 4096, 2, 16, 4, true, 1, 152, 1);
    const BlockPlan generic = make_block_plan(5000, 20000, 2, 16, 4, true, 1, 152, 1);
    if (staged.kind != BLOCK_STAGED || !half.half || !shift.shift || warp.kind != BLOCK_WARP || !cluster.cluster ||
        generic.kind != BLOCK_GENERIC) return 1;
    if (!refuses(staged, [](BlockPlan &p) { p.stages = 0; })) return 2;
    if (!refuses(staged, [](BlockPlan &p) { p.stages = 9; })) return 3;
    if (!refuses(staged, [](BlockPlan &p) { p.stage_bytes = 0; })) return 4;
    if (!refuses(staged, [](BlockPlan &p) { p.threads = 1056; })) return 5;
    if (!refuses(staged, [](BlockPlan &p) { p.grid = 0; })) return 6;
    if (!refuses(half, [](BlockPlan &p) { p.threads = 672; })) return 7;
    if (!refuses(shift, [](BlockPlan &p) { p.kind = BLOCK_WARP, p.threads = 32; })) return 8;
    if (!refuses(shift, [](BlockPlan &p) { p.kind = BLOCK_GENERIC; })) return 9;
    if (!refuses(warp, [](BlockPlan &p) { p.threads = 512; })) return 10;
    if (!refuses(cluster, [](BlockPlan &p) { p.cluster = 9; })) return 11;
    if (!refuses(generic, [](BlockPlan &p) { p.cluster = 2; })) return 12;
    for (int64_t D = 1; D < 33000; D += D < 300 ? 1 : 13)  // and every plan that is made passes
        for (int64_t rows : {1, 8, 64, 153, 400, 5000})
            for (int vjp = 0; vjp < 2; ++vjp)
                for (int how = 0; how < 8; ++how)
                    if (!block_plan_ok(make_block_plan(rows, D, how % 2 ? 4 : 2, how / 2 % 2 ? 16 : 4, vjp ? 5 : 2, vjp, 1, 152,
                                                       how / 4 ? 8 : 0))) {
                        printf("rows %ld D %ld vjp %d how %d", (long)rows, (long)D, vjp, how);
                        return 13;
                    }
    return 0;
}
"""

SCRATCH = r"""
#include <cstdio>
#include "block_plan.h"
using namespace rmsn;
// What the size asked beforehand allows: 320 MB of long rows, or the 12 bytes an element
// of eight CTAs, or of the rows, and never less than a call takes.
int main() {
    for (int64_t D = 1; D <= (int64_t)1 << 24; D += D < 100 ? 1 : D / 37 + 1)
        for (int64_t rows : {1, 2, 9, 127, 128, 256, 300, 1000, 4096, 8192, 100000})
            for (int es : {2, 4})
                for (int sm : {2, 152}) {
                    const size_t asked = block_workspace_bytes(rows, D, es, sm);
                    const size_t cap = 12 * (size_t)D * (rows < 8 ? rows : 8) + 256;
                    if (D > 32768 && asked > cap + ((size_t)64 << 20) && asked > ((size_t)320 << 20) + 256) {
                        printf("rows %ld D %ld: %zu bytes", (long)rows, (long)D, asked);
                        return 1;
                    }
                    if (asked > 12 * (size_t)D * rows + 4 * (size_t)D * (rows / 128) + 256) return 2;
                    for (int64_t gates : {(int64_t)1, rows / 3, rows / 2})
                        for (int unit : {16, es})
                            for (int classes : {0, 1, 2, 4, 8}) {
                                if (gates < 1 || rows % gates) continue;
                                const BlockPlan p = make_block_plan(rows, D, es, unit, 3, true, gates, sm, classes);
                                const size_t need = block_scratch_bytes(p.cluster ? 1 : p.grid, rows, D);
                                const int slices = block_slices(p.team ? 1 : gates, D);
                                if (need > asked || need < ((size_t)(p.cluster ? 0 : p.grid) * 3 + (slices > 1 ? slices : 0)) * D * 4) {
                                    printf("rows %ld D %ld gates %ld unit %d classes %d: %zu of %zu bytes", (long)rows, (long)D,
                                           (long)gates, unit, classes, need, asked);
                                    return 3;
                                }
                            }
                }
    return 0;
}
"""


def _run(tmp_path, name, text):
    src, exe = tmp_path / (name + ".cu"), tmp_path / name
    src.write_text(text)
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    subprocess.run([nvcc, "-std=c++17", "-O2", "-I" + os.path.join(ROOT, "rmsnorm_fwd_bwd_add_gb300", "csrc"), "-o",
                    str(exe), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


def test_row_split_and_partial_slots(tmp_path):
    _run(tmp_path, "split", SPLIT)


def test_plans_stay_within_the_chip_and_the_workspace(tmp_path):
    """Every plan fits its threads, ring and shared memory, and the VJP's never has
    more CTAs than the workspace query counted on."""
    _run(tmp_path, "plan", PLAN)


def test_plans_leave_room_for_the_kernels_static_sums(tmp_path):
    """What a launch asks for and what its kernel holds anyway fit a CTA's shared
    memory together, at every row length that has a plan on chip."""
    _run(tmp_path, "limits", LIMITS)


def test_plans_that_no_kernel_can_run_are_refused(tmp_path):
    _run(tmp_path, "guard", GUARD)


def test_scratch_of_long_rows_is_bounded(tmp_path):
    _run(tmp_path, "scratch", SCRATCH)
