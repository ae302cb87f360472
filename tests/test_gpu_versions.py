"""Calls that write into a tensor they were given count as in-place changes of
it: autograd refuses a backward pass through what they overwrote, as it does
after a torch operation in place."""
import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()


def _mk(*s, dtype=torch.bfloat16):
    return torch.randn(*s, device=DEV).to(dtype)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _calls():
    """name: (call, the tensors it writes)"""
    y, r, w, g = _mk(6, 64), _mk(6, 64), _mk(64), _mk(6, 64)
    o = [_mk(6, 64) for _ in range(2)]
    f = [torch.zeros(64, device=DEV) for _ in range(3)]
    rstd = torch.zeros(2, 6, device=DEV)
    rs1 = torch.zeros(6, device=DEV)
    gate = _mk(64)
    q, k, v = _mk(6, 4, 16), _mk(6, 2, 16), _mk(6, 2, 16)
    pos, slots = torch.arange(6, device=DEV), torch.arange(6, device=DEV)
    kc, vc, qo, ko = _mk(8, 2, 16), _mk(8, 2, 16), _mk(6, 4, 16), _mk(6, 2, 16)
    inv, _ = rn.rope_frequencies(16)
    lens, new, fin = _i32(1, 2), _i32(1, 1), torch.zeros(2, dtype=torch.bool, device=DEV)
    table, free, count = _i32(0, 1, 2, 3).view(2, 2), _i32(4, 5, 6, 7), _i32(4)
    lo, co = _i32(0, 0), _i32(0)
    plan = rn.rmsnorm_kv_plan(lens.clone(), new, table.clone(), 4, 6)
    ws = torch.empty(max(256, rn.rmsnorm_vjp_workspace_size(6, 64, torch.bfloat16)), dtype=torch.uint8, device=DEV)
    x2, half = _mk(6, 128), _mk(6, 64)
    return {
        "block_fwd": (lambda: rn.rmsnorm_block_fwd(y, r, w, w, EPS, out=o[0], new_residual=o[1], rstd=rstd), [*o, rstd]),
        "block_fwd in place": (lambda: rn.rmsnorm_block_fwd(y, r, w, w, EPS, out=y, new_residual=r), [y, r]),
        "block_vjp": (lambda: rn.rmsnorm_block_vjp(y, r, w, w, g, EPS, 0.0, gate, g_y=o[0], g_h=o[1], gw_post=f[0],
                                                   gw_pre=f[1], g_gate=f[2]), [*o, *f]),
        "rope": (lambda: rn.rmsnorm_rope(q, k, pos, inv, q_out=qo, k_out=ko), [qo, ko]),
        "rope in place": (lambda: rn.rmsnorm_rope(q, k, pos, inv, q_out=q, k_out=k), [q, k]),
        "append_ex": (lambda: rn.rmsnorm_rope_kv_append_ex(q, k, v, pos, slots, kc, vc, inv, q_out=qo), [qo, kc, vc]),
        "kv_release": (lambda: rn.rmsnorm_kv_release(lens, fin, table, 4, free, count), [lens, count, free]),
        "kv_release out": (lambda: rn.rmsnorm_kv_release(lens, fin, table, 4, free, count, lens_out=lo, free_count_out=co),
                           [lo, co, free]),
        "kv_plan": (lambda: rn.rmsnorm_kv_plan(lens, new, table, 4, 6, free_blocks=free, free_count=count),
                    [lens, count, table]),
        "kv_plan out": (lambda: rn.rmsnorm_kv_plan(
            lens, new, table, 4, 6, free_blocks=free, free_count=count, lens_out=lo, free_count_out=co,
            positions=plan.positions, slots=plan.slots, requests=plan.requests, starts=plan.starts, granted=plan.granted),
            [lo, co, table, plan.positions, plan.slots, plan.requests, plan.starts, plan.granted]),
        "fwd": (lambda: rn.rmsnorm_fwd(y, w, EPS, residual=r, out=o[0], new_residual=o[1]), o),
        "fwd without residual": (lambda: rn.rmsnorm_fwd(y, w, EPS, out=o[0]), o[:1]),
        "vjp": (lambda: rn.rmsnorm_vjp(y, w, g, EPS, gx=o[0], gw=f[0]), [o[0], f[0]]),
        "fused_vjp": (lambda: rn.rmsnorm_fused_vjp(y, w, g, EPS, 0.0, r, g_h=o[0], gw=f[0]), [o[0], f[0]]),
        "bound fwd": (rn.rmsnorm_fwd_bind(y, w, EPS, residual=r, out=o[0], new_residual=o[1]), o),
        "bound vjp": (rn.rmsnorm_vjp_bind(y, w, g, EPS, gx=o[0], gw=f[0]), [o[0], f[0]]),
        "fwd_ex": (lambda: rn.rmsnorm_fwd_ex(y, w, EPS, 0.0, r, out=o[0], new_residual=o[1], rstd=rs1), [*o, rs1]),
        "vjp_ex": (lambda: rn.rmsnorm_vjp_ex(y, w, g, EPS, 0.0, gx=o[0], gw=f[0]), [o[0], f[0]]),
        "vjp_ws": (lambda: rn.rmsnorm_vjp_ws(y, w, g, EPS, workspace=ws, gx=o[0], gw=f[0]), [o[0], f[0], ws]),
        "vjp_noalloc": (lambda: rn.rmsnorm_vjp_noalloc(y, w, g, EPS, gx=o[0], gw=f[0]), [o[0], f[0]]),
        "gated_silu": (lambda: rn.rmsnorm_gated_silu(x2, out=half), [half]),
        "rope_kv_append": (lambda: rn.rmsnorm_rope_kv_append(q, k, v, pos, slots, kc, vc, q_out=qo), [qo, kc, vc]),
    }


@pytest.mark.parametrize("name", [
    "block_fwd", "block_fwd in place", "block_vjp", "rope", "rope in place", "append_ex", "kv_release", "kv_release out",
    "kv_plan", "kv_plan out", "fwd", "fwd without residual", "vjp", "fused_vjp", "bound fwd", "bound vjp", "fwd_ex",
    "vjp_ex", "vjp_ws", "vjp_noalloc", "gated_silu", "rope_kv_append"])
def test_tensors_written_count_as_changed(name):
    call, written = _calls()[name]
    for _ in range(2):
        before = [t._version for t in written]
        got = call()
        assert all(t._version > b for t, b in zip(written, before)), [t._version - b for t, b in zip(written, before)]
    got = got if isinstance(got, tuple) else (got,)
    given = {t.data_ptr() for t in written}
    for t in got:  # what the call allocated is new
        assert t is None or t.data_ptr() in given or t._version == 0


def test_inputs_do_not_count_as_changed():
    y, r, w = _mk(6, 64), _mk(6, 64), _mk(64)
    before = [t._version for t in (y, r, w)]
    rn.rmsnorm_block_fwd(y, r, w, w, EPS)
    rn.rmsnorm_fwd(y, w, EPS, residual=r)
    q, pos = _mk(6, 4, 16), torch.arange(6, device=DEV)
    rn.rmsnorm_rope(q, None, pos, rn.rope_frequencies(16)[0])
    assert [t._version for t in (y, r, w)] == before and q._version == 0 and pos._version == 0


def test_backward_through_overwritten_tensors_is_refused():
    inv, _ = rn.rope_frequencies(16)
    for overwrite in (lambda nr, pos: rn.rmsnorm_block_fwd(_mk(6, 64), nr, None, _mk(64), EPS, new_residual=nr),
                      lambda nr, pos: rn.rmsnorm_fwd(_mk(6, 64), _mk(64), EPS, residual=nr, new_residual=nr),
                      lambda nr, pos: rn.rmsnorm_rope(nr.view(6, 4, 16), None, pos, inv, q_out=nr.view(6, 4, 16))):
        y, r, w = (_mk(*s).requires_grad_() for s in ((6, 64), (6, 64), (64,)))
        out, nr = rn.block_norm(y, r, w, w, EPS)
        overwrite(nr.detach(), torch.arange(6, device=DEV))
        with pytest.raises(RuntimeError, match="inplace"):
            out.float().sum().backward()
    # positions that a step's plan writes again
    lens, new, table = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in ([0, 0], [3, 3], [[0], [1]]))
    plan = rn.rmsnorm_kv_plan(lens, new, table, 16, 6)
    q = _mk(6, 4, 16).requires_grad_()
    turned, _ = rn.rope(q, None, plan.positions, inv)
    rn.rmsnorm_kv_plan(lens, new, table, 16, 6, positions=plan.positions)
    with pytest.raises(RuntimeError, match="inplace"):
        turned.float().sum().backward()


def test_inference_tensors_are_written():
    with torch.inference_mode():
        y, r, w = _mk(6, 64), _mk(6, 64), _mk(64)
        q, pos = _mk(6, 4, 16), torch.arange(6, device=DEV)
        inv, _ = rn.rope_frequencies(16)
        want = rn.rmsnorm_block_fwd(y, r, w, w, EPS)[0]
        turned = rn.rmsnorm_rope(q, None, pos, inv)[0]
    for mode in (True, False):
        with torch.inference_mode(mode):
            out = y.clone()
            res, qo = r.clone(), q.clone()
            rn.rmsnorm_block_fwd(y, r, w, w, EPS, out=out, new_residual=res)
            rn.rmsnorm_rope(q, None, pos, inv, q_out=qo)
            assert torch.equal(out, want) and torch.equal(qo, turned)
            rn.rmsnorm_fwd(y, w, EPS, out=out)
    rn.rmsnorm_block_fwd(y, r, w, w, EPS, out=y, new_residual=r)  # tensors made in inference mode, outside of it
    assert torch.equal(y, want)
