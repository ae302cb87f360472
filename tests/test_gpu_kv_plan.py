"""rmsnorm_kv_plan and rmsnorm_kv_release against a step-by-step Python model of
the pool, over many steps of a random serving run, and at the edges: no
requests, no room, padded steps, bad lengths and ids."""
import random

import pytest
import torch

import rmsnorm_fwd_bwd_add_gb300 as rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_add_gb300 import build
    build.build()
    rn.rmsnorm_device_status(clear=True)
    yield
    assert rn.rmsnorm_device_status(clear=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The pool, one request and one block at a time."""

    def __init__(self, B, W, bs, blocks, seed):
        self.B, self.W, self.bs, self.rng = B, W, bs, random.Random(seed)
        self.lens, self.table = [0] * B, [[-1] * W for _ in range(B)]
        self.stack = list(range(blocks))
        self.rng.shuffle(self.stack)

    def release(self, finished):
        for b, done in enumerate(finished):
            if done:
                self.stack += self.table[b][:-(-self.lens[b] // self.bs)]
                self.lens[b] = 0

    def plan(self, new, T):
        starts, cum, top = [0], 0, len(self.stack)
        out = dict(pos=[], slots=[], req=[], granted=[])
        taken = 0
        for b, n in enumerate(new):
            starts.append(starts[-1] + n)
            have, want = -(-self.lens[b] // self.bs), -(-(self.lens[b] + n) // self.bs)
            ok = want <= self.W and starts[-1] <= T
            if ok:
                cum += want - have
                ok = want == have or cum <= top
            if ok:
                for i in range(have, want):
                    self.table[b][i] = self.stack[top - 1 - taken]
                    taken += 1
            for j in range(n):
                p = self.lens[b] + j
                out["pos"].append(p)
                out["slots"].append(self.table[b][p // self.bs] * self.bs + p % self.bs if ok else -1)
                out["req"].append(b)
            if ok:
                self.lens[b] += n
            out["granted"].append(ok)
        self.stack = self.stack[:top - taken]
        pad = T - len(out["pos"])
        for key, fill in (("pos", 0), ("slots", -1), ("req", -1)):
            out[key] = (out[key] + [fill] * max(pad, 0))[:T]
        out["starts"] = starts
        return out


@pytest.mark.parametrize("B,W,bs,blocks,most,T", [
    (1, 4, 16, 4, 1, 1), (5, 8, 4, 30, 9, 40), (33, 20, 1, 300, 5, 100), (250, 16, 16, 2500, 1, 256),
    (1000, 6, 7, 4000, 12, 6000), (3000, 5, 64, 9000, 64, 60000), (1025, 3, 16, 2000, 2, 4097),
    (34, 3, 1, 60, 5, 70), (64, 50, 2, 300, 40, 700), (200, 4, 4, 300, 9, 500)],
    ids=lambda v: str(v))
def test_serving_run(B, W, bs, blocks, most, T):
    m = Model(B, W, bs, blocks, B + W)
    rng = random.Random(7)
    lens, table = i32([0] * B), torch.full((B, W + 3), -1, dtype=torch.int32, device=DEV)[:, :W]
    free, count = i32(m.stack), i32([blocks])
    denied = 0
    for step in range(12):
        done = [rng.random() < 0.2 for _ in range(B)]
        rn.rmsnorm_kv_release(lens, torch.tensor(done, device=DEV), table, bs, free, count)
        m.release(done)
        assert lens.tolist() == m.lens and count.item() == len(m.stack)
        assert free[:len(m.stack)].tolist() == m.stack
        new = [rng.choice([0, 1, 1, rng.randint(0, most)]) for _ in range(B)]
        got = rn.rmsnorm_kv_plan(lens, i32(new), table, bs, T, free_blocks=free, free_count=count)
        want = m.plan(new, T)
        assert got.starts.tolist() == want["starts"]
        assert got.granted.tolist() == want["granted"]
        assert got.positions.tolist() == want["pos"]
        assert got.slots.tolist() == want["slots"]
        assert got.requests.tolist() == want["req"]
        assert lens.tolist() == m.lens and got.lens is lens and count.item() == len(m.stack)
        denied += want["granted"].count(False)
        for b in rng.sample(range(B), min(B, 40)):
            n = -(-m.lens[b] // bs)
            assert table[b, :n].tolist() == m.table[b][:n]
    held = sum((table[b, :-(-m.lens[b] // bs)].tolist() for b in range(B)), [])
    assert sorted(held + m.stack) == list(range(blocks))  # every block in one place
    # by the model alone: the tight pools, tables and budgets turn requests away
    assert (denied > 0) == (B in (34, 64, 200, 1000))


def test_long_prompts():
    """A prefill of many blocks, a table without a pool, and slots past 2^31."""
    B, bs, W = 3, 16, 8192
    lens, new = i32([0, 5, 100000]), i32([130000, 0, 7])
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    table[1, :1], table[2, :6250] = 9000, torch.arange(10000, 16250, dtype=torch.int32, device=DEV)
    free = torch.arange(20000, dtype=torch.int32, device=DEV)
    got = rn.rmsnorm_kv_plan(lens, new, table, bs, 130007, free_blocks=free, free_count=i32([9000]))
    assert got.granted.tolist() == [True] * 3 and got.lens.tolist() == [130000, 5, 100007]
    assert got.free_count.tolist() == [9000 - 8125 - 1]
    p = torch.arange(130000, device=DEV)
    assert torch.equal(got.slots[:130000], (8999 - p // 16) * 16 + p % 16)
    assert torch.equal(got.positions[:130000], p)
    assert got.slots[130000:].tolist() == [(8999 - 8125) * 16 + i for i in range(7)]
    t = i32([[2000000, 2000001], [7, -1]])
    got = rn.rmsnorm_kv_plan(i32([4094, 1]), i32([5, 1]), t, 4096, 8)
    assert got.slots.tolist() == [2000000 * 4096 + 4094, 2000000 * 4096 + 4095] + \
        [2000001 * 4096 + i for i in range(3)] + [7 * 4096 + 1, -1, -1]
    assert got.free_count is None and got.granted.all()


def test_edges():
    t0 = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    got = rn.rmsnorm_kv_plan(i32([]), i32([]), t0, 16, 5, free_blocks=i32([3, 1]), free_count=i32([2]))
    assert got.starts.tolist() == [0] and got.slots.tolist() == [-1] * 5 and got.free_count.tolist() == [2]
    assert got.positions.tolist() == [0] * 5 and got.requests.tolist() == [-1] * 5
    # no tokens at all: only requests that ask for none are granted
    t = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    got = rn.rmsnorm_kv_plan(i32([0, 0, 0]), i32([0, 1, 0]), t, 16, 0, free_blocks=i32([0, 1]), free_count=i32([2]))
    assert got.granted.tolist() == [True, False, False] and got.slots.numel() == 0
    assert got.free_count.tolist() == [2]
    # an empty pool, a table without columns
    got = rn.rmsnorm_kv_plan(i32([4]), i32([1]), i32([[0]]), 4, 1, free_blocks=i32([]), free_count=i32([0]))
    assert got.granted.tolist() == [False] and got.lens.tolist() == [4] and got.slots.tolist() == [-1]
    got = rn.rmsnorm_kv_plan(i32([0, 0]), i32([0, 1]), torch.zeros((2, 0), dtype=torch.int32, device=DEV), 4, 1,
                             free_blocks=i32([0]), free_count=i32([1]))
    assert got.granted.tolist() == [True, False]
    # out of place: the old state stays
    lens, count = i32([3, 3]), i32([2])
    lo, co = torch.empty_like(lens), torch.empty_like(count)
    got = rn.rmsnorm_kv_plan(lens, i32([2, 1]), i32([[0, -1], [1, -1]]), 4, 3, free_blocks=i32([2, 3, -1, -1]), free_count=count,
                             lens_out=lo, free_count_out=co)
    assert lens.tolist() == [3, 3] and count.tolist() == [2] and lo.tolist() == [5, 4] and co.tolist() == [1]
    assert got.slots.tolist() == [3, 3 * 4, 7]


def test_bad_state_is_flagged():
    rn.rmsnorm_device_status(clear=True)
    free = i32([0, 1, 2, 3])
    t = i32([[0, -1], [1, -1], [9, -1]])
    got = rn.rmsnorm_kv_plan(i32([2, -5, 2]), i32([1, 1, 1]), t, 4, 4, free_blocks=free, free_count=i32([1]))
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert got.granted.tolist() == [True, False, True] and got.slots.tolist() == [2, -1, -1, -1]
    assert got.lens.tolist() == [3, -5, 3] and got.starts.tolist() == [0, 1, 1, 2]
    got = rn.rmsnorm_kv_plan(i32([0]), i32([1]), t[:1], 4, 1, free_blocks=i32([77, 78]), free_count=i32([99]))
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert got.slots.tolist() == [-1] and got.free_count.tolist() == [1]
    got = rn.rmsnorm_kv_plan(i32([0, 3]), i32([-2, 1]), t[:2], 4, 1)
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX and got.granted.tolist() == [False, True]
    # a length near the type's end does not wrap
    got = rn.rmsnorm_kv_plan(i32([2 ** 31 - 1]), i32([2 ** 31 - 1]), i32([[0]]), 2 ** 31 - 1, 3)
    assert got.granted.tolist() == [False] and got.lens.tolist() == [2 ** 31 - 1]
    assert rn.rmsnorm_device_status(clear=True) == 0
    # a stack that would run over; a request that claims more blocks than its row has
    stack, count = i32([5, 5, 5]), i32([2])
    lens = i32([8, 100, 4])
    rn.rmsnorm_kv_release(lens, torch.tensor([True, True, True], device=DEV), i32([[0, 1], [2, 2], [2, -1]]), 4, stack,
                          count)
    assert rn.rmsnorm_device_status(clear=True) == rn.DEVSTATUS_BAD_INDEX
    assert count.tolist() == [3] and stack.tolist() == [5, 5, 0] and lens.tolist() == [0, 0, 0]


def test_graph_replay_advances_the_state():
    """A captured step that updates its lengths and pool in place, replayed."""
    B, W, bs, blocks = 40, 10, 4, 500
    m = Model(B, W, bs, blocks, 3)
    lens, new = i32([0] * B), i32([1] * B)
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    free, count = i32(m.stack), i32([blocks])
    done = torch.zeros(B, dtype=torch.bool, device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        rn.rmsnorm_kv_release(lens, done, table, bs, free, count)
        got = rn.rmsnorm_kv_plan(lens, new, table, bs, 64, free_blocks=free, free_count=count)
    rng = random.Random(1)
    for _ in range(30):
        d, n = [rng.random() < 0.1 for _ in range(B)], [rng.randint(0, 2) for _ in range(B)]
        done.copy_(torch.tensor(d)), new.copy_(torch.tensor(n))
        gr.replay()
        m.release(d)
        want = m.plan(n, 64)
        assert got.slots.tolist() == want["slots"] and got.positions.tolist() == want["pos"]
        assert lens.tolist() == m.lens and count.item() == len(m.stack)


def test_a_serving_step_from_lengths_to_the_next_norm():
    """Lengths -> plan -> rotary append -> attention over the paged cache (plain
    torch here) -> the norms around the block: against the same step on dense
    per-request tensors in 64 bits."""
    import block_reference as ref
    g = torch.Generator().manual_seed(4)
    B, W, bs, Hq, Hkv, Dh = 5, 6, 8, 4, 2, 32
    D = Hq * Dh
    m = Model(B, W, bs, 40, 1)
    kc = torch.zeros(40 * bs, Hkv, Dh, device=DEV)
    vc = torch.zeros(40 * bs, Hkv, Dh, device=DEV)
    lens, table = i32([0] * B), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    free, count = i32(m.stack), i32([40])
    inv, scale = rn.rope_frequencies(16, 10000.0, "yarn", factor=4.0, trained_length=512.0)
    w_post, w_pre = torch.rand(D, generator=g).to(DEV) + 0.5, torch.rand(D, generator=g).to(DEV) + 0.5
    gate = torch.randn(D, generator=g).to(DEV)
    seqs = [[] for _ in range(B)]  # (k, v) in 64 bits, rotated

    def turn(x, p):
        ang = p.double()[:, None] * inv.to(DEV)
        z = torch.complex(x[..., :8].double(), x[..., 8:16].double()) * torch.polar(torch.full_like(ang, scale), ang)[:, None]
        return torch.cat([z.real, z.imag, x[..., 16:].double()], -1)
    for new in ([7, 3, 1, 0, 9], [1, 1, 1, 5, 1], [1, 1, 1, 1, 1]):
        T = sum(new) + 3  # padded
        plan = rn.rmsnorm_kv_plan(lens, i32(new), table, bs, T, free_blocks=free, free_count=count)
        qkv = torch.randn(T, Hq + 2 * Hkv, Dh, generator=g).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        qo = rn.rmsnorm_rope_kv_append_ex(q, k, v, plan.positions, plan.slots, kc, vc, inv, attn_scale=scale)
        y, want_y = torch.zeros(T, D, device=DEV), torch.zeros(T, D, dtype=torch.float64, device=DEV)
        q64, k64 = turn(q, plan.positions), turn(k, plan.positions)
        for t in range(sum(new)):
            b, p = plan.requests[t].item(), plan.positions[t].item()
            rows = torch.arange(p + 1, device=DEV)
            at = table[b, rows // bs].long() * bs + rows % bs
            seqs[b].append((k64[t], v[t].double()))
            for kk, vv, qq, dst in ((kc[at].double(), vc[at].double(), qo[t].double(), y),
                                    (torch.stack([s[0] for s in seqs[b][:p + 1]]),
                                     torch.stack([s[1] for s in seqs[b][:p + 1]]), q64[t], want_y)):
                s = torch.einsum("hd,nhd->hn", qq, kk.repeat_interleave(2, 1)) / Dh ** 0.5
                dst[t] = torch.einsum("hn,nhd->hd", s.softmax(-1), vv.repeat_interleave(2, 1)).reshape(-1)
        res = torch.randn(T, D, generator=g).to(DEV)
        out, nr, _ = rn.rmsnorm_block_fwd(y, res, w_post, w_pre, 1e-6, 0.0, gate, 0.5)
        want = ref.fwd(want_y, res, w_post, w_pre, 1e-6, 0.0, gate.view(1, D), 0.5)
        # rotated q and k are within 4e-7 of their pairs, scores of up to 10 move by 1e-5 and
        # the softmax by as much: 1e-4 of the values' size covers it with room
        n = sum(new)
        assert (out[:n] - want[0][:n]).abs().max() <= 1e-4 * want[0].abs().max()
        assert (nr[:n] - want[1][:n]).abs().max() <= 1e-4 * want[1].abs().max()


def test_python_refusals():
    lens, table = i32([0, 0]), torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    free, count = i32([0, 1]), i32([2])
    for a, kw in (((lens.long(), lens, table, 16, 4), {}), ((lens, lens[:1], table, 16, 4), {}),
                  ((lens, lens, table.long(), 16, 4), {}), ((lens, lens, table[:1], 16, 4), {}),
                  ((lens, lens, table.t(), 16, 4), {}), ((lens, lens, table, 16, -1), {}),
                  ((lens, lens, table[:1].expand(2, 4), 16, 4), {}),
                  ((lens, lens, table, 16, 4), dict(free_blocks=free)), ((lens, lens, table, 16, 4), dict(free_count=count)),
                  ((lens, lens, table, 16, 4), dict(free_count_out=count)),
                  ((lens, lens, table, 16, 4), dict(positions=lens)),
                  ((lens, lens, table, 16, 4), dict(free_blocks=free, free_count=i32([1, 1])))):
        with pytest.raises(ValueError):
            rn.rmsnorm_kv_plan(*a, **kw)
    with pytest.raises(ValueError):
        rn.rmsnorm_kv_release(lens, lens, table, 16, free, count)
    with pytest.raises(rn.RmsnormError):
        rn.rmsnorm_kv_plan(lens, lens.clone(), table, 0, 4)
    with pytest.raises(rn.RmsnormError):  # new_lens is the output too
        rn.rmsnorm_kv_plan(lens, lens, table, 16, 4)


@pytest.mark.parametrize("B,every,T", [(9001, 1, 12000), (9001, 1, 3000), (13000, 2500, 40), (13000, 2500, 9000),
                                       (4097, 4096, 8)])
def test_more_requests_than_a_pass(B, every, T):
    """Several passes of the scan, with tokens in all requests, or in one of
    `every`, whose neighbours lie further apart than the tokens' table holds."""
    W, bs, blocks = 3, 4, 2 * B
    m = Model(B, W, bs, blocks, B)
    rng = random.Random(every)
    lens, table = i32([0] * B), torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    free, count = i32(m.stack), i32([blocks])
    for step in range(4):
        done = [rng.random() < 0.4 for _ in range(B)]
        rn.rmsnorm_kv_release(lens, torch.tensor(done, device=DEV), table, bs, free, count)
        m.release(done)
        assert lens.tolist() == m.lens and free[:len(m.stack)].tolist() == m.stack
        new = [rng.choice([0, 1, 1, 6]) if b % every == 0 else 0 for b in range(B)]
        got = rn.rmsnorm_kv_plan(lens, i32(new), table, bs, T, free_blocks=free, free_count=count)
        want = m.plan(new, T)
        assert got.starts.tolist() == want["starts"]
        assert got.granted.tolist() == want["granted"]
        assert got.positions.tolist() == want["pos"]
        assert got.slots.tolist() == want["slots"]
        assert got.requests.tolist() == want["req"]
        assert lens.tolist() == m.lens and count.item() == len(m.stack)
