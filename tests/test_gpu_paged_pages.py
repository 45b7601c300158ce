"""Where the pages of the paged cache are, step after step: held by a request, or free in the ring, each exactly once."""
import numpy as np
import pytest

import paged_ref as ref
from test_gpu_paged import PAGE, Server, i32, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


class Pool:
    """Tables, ring and lengths on the device, beside a list of pages for each request and one of the free ones."""

    def __init__(self, api, R, T, nb, n_pages, seed, held=True):
        import torch
        self.api, self.rng = api, np.random.default_rng(seed)
        self.sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=2, Hkv=2, d=64, d_idx=64, topk=2)
        ids = self.rng.permutation(n_pages)
        head = int(self.rng.integers(n_pages))
        self.ring, self.free = i32(np.roll(ids, head)), i32([head, n_pages])
        self.table = torch.full((R, nb), -1, dtype=torch.int32, device="cuda")
        self.lens, self.held = i32([0] * R), i32([0] * R) if held else None
        self.ws = api.new_paged_workspace(self.sh, api.OP_PAGED_PLAN)
        self.pages, self.left, self.n = [[] for _ in range(R)], list(ids), np.zeros(R, int)

    def step(self, new, ended=None):
        p = self.api.paged_plan(self.sh, i32(new), self.lens, self.table, self.ring, self.free, held=self.held,
                                ended=None if ended is None else i32(ended), workspace=self.ws)
        self.lens, self.free = p.lens, p.free_state
        back = []
        for r in range(self.sh.R):
            if ended is not None and ended[r]:
                back += self.pages[r]
                self.pages[r], self.n[r] = [], 0
        for r in range(self.sh.R):
            self.n[r] += new[r]
            while len(self.pages[r]) * PAGE < self.n[r]:
                self.pages[r].append(self.left.pop(0))
        self.left += back
        return p

    def check(self, p, new):
        status_ok(self.api, self.ws)
        table, ring, (head, count) = self.table.cpu().numpy(), self.ring.cpu().numpy(), self.free.tolist()
        assert p.lens.tolist() == self.n.tolist()
        assert [int(ring[(head + i) % len(ring)]) for i in range(count)] == self.left
        for r, pages in enumerate(self.pages):
            assert table[r, :len(pages)].tolist() == pages
        if self.held is not None:
            assert self.held.tolist() == [len(x) for x in self.pages]
        assert sorted(self.left + sum(self.pages, [])) == list(range(len(ring)))
        starts, req, pos, slots, segs = (t.cpu().numpy() for t in (p.q_starts, p.row_req, p.row_pos, p.slots, p.segs))
        assert starts.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
        want = [(r, at, self.pages[r][at // PAGE] * PAGE + at % PAGE) for r in range(self.sh.R) for at in range(self.n[r] - new[r], self.n[r])]
        n = len(want)
        assert list(zip(req[:n], pos[:n], slots[:n])) == want and np.all(req[n:] == -1) and np.all(slots[n:] == -1)
        first = [i for i in range(n) if i in starts or pos[i] % PAGE == 0]
        assert segs.tolist() == first + [n] * (len(segs) - len(first))


@pytest.mark.parametrize("R,T,nb,most", [(1, 16, 9, 8), (6, 400, 5, 60), (40, 3000, 6, 70), (1100, 9000, 3, 8)])
def test_lengths_that_are_lowered_lose_no_page(api, R, T, nb, most):
    """A hundred steps of rows accepted and rejected, also over page borders, some requests ending: held and free pages stay the pool."""
    pool = Pool(api, R, T, nb, R * nb + 3, seed=R)
    rng = pool.rng
    for step in range(100 if R < 1000 else 12):
        ended = (rng.random(R) < 0.05).astype(int) if step % 3 else None
        have = pool.n if ended is None else np.where(ended, 0, pool.n)
        new = np.minimum(rng.integers(0, most + 1, R), nb * PAGE - have)
        p = pool.step(new, ended)
        pool.check(p, new)
        drop = np.minimum(np.where(rng.random(R) < 0.5, rng.integers(0, most + 1, R), 0), pool.n)
        if step % 7 == 3:
            drop = np.where(rng.random(R) < 0.3, np.minimum(pool.n, 300), drop)
        pool.n -= drop
        pool.lens = pool.lens - i32(drop)


@pytest.mark.parametrize("held", [[1, 2, 0], [2, 9, 0], [2, -1, 0], [2, 2, 5]])
def test_held_pages_out_of_range_make_no_step(api, held):
    """Fewer than the length takes, or more than the table's columns."""
    pool = Pool(api, 3, 20, 4, 20, seed=2)
    p = pool.step([10, 4, 0])
    pool.lens, pool.held = i32([200, 250, 0]), i32(held)
    before = [t.clone() for t in (pool.table, pool.ring, pool.free, pool.lens, pool.held)]
    p = api.paged_plan(pool.sh, i32([1, 1, 1]), pool.lens, pool.table, pool.ring, pool.free, held=pool.held, workspace=pool.ws)
    with pytest.raises(api.MsaError, match="MSA_ERR_DEVICE"):
        api.check_device_status(pool.ws)
    for a, b in zip(before, (pool.table, pool.ring, p.free_state, p.lens, pool.held)):
        assert a.tolist() == b.tolist()
    assert not p.q_starts.any() and (p.slots == -1).all()


def test_speculative_rows_are_dropped_and_written_again(api):
    """Four rows a step, some of them rejected afterwards, through the plan, the append and the attention: the cache is that of
    the tokens kept, and the attention's rows see those alone."""
    import torch
    sv = Server(api, R=3, nb=4, n_pages=13, Hq=4, Hkv=1, d=64, di=64, k=4, T=500, seed=4)
    held, rng = i32([0, 0, 0]), np.random.default_rng(11)
    kept = [np.zeros((0, 64)) for _ in range(3)]
    for step in range(25):
        new = [120, 126, 250] if step == 0 else [4, 4, 4]
        x = sv.rows()
        plan = api.paged_plan(sv.sh, i32(new), sv.lens, sv.table, sv.ring, sv.free, held=held, workspace=sv.ws[16])
        sv.lens, sv.free = plan.lens, plan.free_state
        api.paged_append(sv.sh, x["k"][0], x["v"][0], x["ki"][0], plan.slots, plan.segs, sv.k8, sv.v8, sv.ks, sv.vs, sv.ki, workspace=sv.ws[17])
        o, lse = api.paged_attn(sv.sh, x["q"][0], sv.k8, sv.v8, sv.ks, sv.vs, sv.table, plan.row_req, plan.row_pos, workspace=sv.ws[20])
        for ws in sv.ws.values():
            status_ok(api, ws)
        st, req, pos = (t.cpu().numpy() for t in (plan.q_starts, plan.row_req, plan.row_pos))
        kept = [np.concatenate([kept[r], x["ki"][1][st[r]:st[r + 1]]]) for r in range(3)]
        table, ki = sv.table.cpu().numpy(), sv.ki.double().cpu().numpy()
        for r in range(3):
            assert np.array_equal(ki[table[r, :(len(kept[r]) + 127) // PAGE]].reshape(-1, 64)[:len(kept[r])], kept[r])
        n = st[-1]
        ow, lw, do, dl = ref.attn(x["q"][1], *(c.view(torch.uint8).cpu().numpy() for c in (sv.k8, sv.v8)), sv.ks.cpu().numpy(), sv.vs.cpu().numpy(),
                                  table, req, pos, None, 0.125)
        assert np.all(np.abs(o.double().cpu().numpy()[:n] - ow[:n]) <= do[:n])
        drop = rng.integers(0, 4, 3) if step else np.array([0, 3, 0])
        kept = [kept[r][:len(kept[r]) - drop[r]] for r in range(3)]
        sv.lens = sv.lens - i32(drop)
    free = int(sv.free[1])
    assert free + int(held.sum()) == 13 and (held >= (sv.lens + 127) // PAGE).all()


@pytest.mark.parametrize("R,T,nb", [(3, 8, 70), (40, 2000, 20), (1100, 1200, 3)])
@pytest.mark.parametrize("held", [False, True])
def test_entries_that_are_no_pages_do_not_enter_the_ring(api, R, T, nb, held):
    """Ended requests whose table has entries out of range: recorded, the other pages free in their order."""
    rng = np.random.default_rng(R + held)
    lens = rng.integers(1, nb * PAGE + 1, R)
    lens[0] = nb * PAGE
    m = (lens + 127) // PAGE
    n_pages = int(m.sum()) + R + 4
    ids = rng.permutation(n_pages).astype(np.int32)
    table, at = np.full((R, nb), -1, np.int32), 0
    for r in range(R):
        table[r, :m[r]] = ids[at:at + m[r]]
        at += m[r]
    ended = (rng.random(R) < 0.6).astype(int)
    ended[0] = 1
    hurt = (rng.random((R, nb)) < 0.3) & (np.arange(nb) < m[:, None]) & (ended == 1)[:, None]
    hurt[0, 0] = True
    table[hurt] = rng.choice([-1, n_pages, -2 ** 31, 2 ** 31 - 1], hurt.sum())
    new = np.where(rng.random(R) < 0.5, 1, 0)
    have = np.where(ended, 0, lens)
    new = np.where(have + new > nb * PAGE, 0, new)
    head, count = n_pages - 2, n_pages - at                     # the ring's end is passed
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(count)) % n_pages] = ids[at:]
    sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=2, Hkv=2, d=64, d_idx=64, topk=2)
    ws, dt, dr, h = api.new_paged_workspace(sh, api.OP_PAGED_PLAN), i32(table), i32(ring), i32(m) if held else None
    p = api.paged_plan(sh, i32(new), i32(lens), dt, dr, i32([head, count]), ended=i32(ended), held=h, workspace=ws)
    with pytest.raises(api.MsaError, match="site 103"):
        api.check_device_status(ws)
    taken = (have + new + 127) // PAGE - (have + 127) // PAGE
    back = [table[r, j] for r in range(R) if ended[r] for j in range(m[r]) if not hurt[r, j]]
    left = list(ids[at:])[taken.sum():] + back
    got, (head2, count2) = dr.cpu().numpy(), p.free_state.tolist()
    assert head2 == (head + taken.sum()) % n_pages and count2 == len(left)
    assert [got[(head2 + i) % n_pages] for i in range(count2)] == left
    assert p.lens.tolist() == (have + new).tolist() and (p.slots[:int(new.sum())] >= 0).all()


def test_a_ring_entry_that_is_no_page_stays_out_of_the_table(api):
    """Its rows have no slot and its column is -1, in the step that takes it and in the next; when the request has ended
    it does not come back."""
    import torch
    for T in (4, 1500):
        sh = api.PagedShape(R=2, T=T, max_blocks=2, n_pages=4, Hq=2, Hkv=1, d=64, d_idx=64, topk=2)
        table, ring, ws = torch.full((2, 2), 7, dtype=torch.int32, device="cuda"), i32([9, 3, 0, 1]), api.new_paged_workspace(sh, api.OP_PAGED_PLAN)
        lens, free = i32([0, 0]), i32([0, 4])
        for new, slots in (([2, 2], [-1, -1, 3 * PAGE, 3 * PAGE + 1]), ([1, 1], [-1, 3 * PAGE + 2])):
            p = api.paged_plan(sh, i32(new), lens, table, ring, free, workspace=ws)
            lens, free = p.lens, p.free_state
            with pytest.raises(api.MsaError, match="site 102"):
                api.check_device_status(ws)
            assert p.slots[:len(slots)].tolist() == slots and table.tolist() == [[-1, 7], [3, 7]]
        p = api.paged_plan(sh, i32([0, 0]), lens, table, ring, free, ended=i32([1, 1]), workspace=ws)
        with pytest.raises(api.MsaError, match="site 103"):
            api.check_device_status(ws)
        assert p.free_state.tolist() == [2, 3] and [int(ring[(2 + i) % 4]) for i in range(3)] == [0, 1, 3]


def test_pages_that_go_back_are_free_from_the_next_step_on(api):
    """A full pool in which one request ends and another starts in its slot: refused in that step, made after one that only
    gives the pages back."""
    pool = Pool(api, 2, 700, 3, 6, seed=1)
    new = [300, 384]
    pool.check(pool.step(new), new)
    assert pool.free.tolist()[1] == 0
    before = [t.clone() for t in (pool.table, pool.ring, pool.free, pool.lens, pool.held)]
    p = api.paged_plan(pool.sh, i32([200, 0]), pool.lens, pool.table, pool.ring, pool.free, held=pool.held, ended=i32([1, 0]), workspace=pool.ws)
    with pytest.raises(api.MsaError, match="site 101, info 4"):
        api.check_device_status(pool.ws)
    for a, b in zip(before, (pool.table, pool.ring, p.free_state, p.lens, pool.held)):
        assert a.tolist() == b.tolist()
    for new, ended in (([0, 0], [1, 0]), ([200, 0], None)):
        pool.check(pool.step(new, ended), new)
    assert pool.lens.tolist() == [200, 384] and pool.free.tolist()[1] == 1
