"""Forking, compaction and copies of cache pages against their definitions."""
import numpy as np
import pytest

import chunk_ref as ref
import paged_ref
from test_gpu_paged import dev, i32

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def state(rng, R, nb, families, spare, extra_held=False):
    """Tables of R requests, the rows of a family sharing their first pages: (lens, held or None, table, ring, free, shares)."""
    lens = rng.integers(0, nb * PAGE + 1, R)
    lens[rng.random(R) < 0.1] = 0
    lens[rng.random(R) < 0.2] //= PAGE
    lens = np.where(rng.random(R) < 0.2, lens // PAGE * PAGE, lens)
    held = -(-lens // PAGE)
    if extra_held:
        held = np.minimum(nb, held + rng.integers(0, 3, R))
    fam = rng.integers(0, families, R)
    common = {f: int(rng.integers(0, 1 + min(int(x) for x in lens[fam == f] // PAGE))) for f in set(fam.tolist())}
    n_pages = int(held.sum() + spare)
    ids = rng.permutation(n_pages)
    table = np.full((R, nb), -5, np.int32)
    shares = np.zeros(n_pages, np.int32)
    at = 0
    first = {}
    for r in range(R):
        f, c = int(fam[r]), common[int(fam[r])]
        if f not in first:
            first[f] = ids[at:at + c]
            at += c
        else:
            shares[first[f]] += 1
        table[r, :c] = first[f]
        table[r, c:held[r]] = ids[at:at + held[r] - c]
        at += held[r] - c
    head, count = int(rng.integers(n_pages)), n_pages - at
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(count)) % n_pages] = ids[at:]
    return lens.astype(np.int32), held.astype(np.int32) if extra_held else None, table, ring, np.array([head, count], np.int32), shares


def shape(api, table, n_pages, **kw):
    return api.PagedShape(**{**dict(R=table.shape[0], T=4, max_blocks=table.shape[1], n_pages=n_pages, Hq=8, Hkv=2, d=64, d_idx=64, topk=4), **kw})


def run_fork(api, src, fl, s, ws=None):
    lens, held, table, ring, free, shares = s
    sh = shape(api, table, len(ring))
    t = [None if x is None else i32(x) for x in (src, fl, lens, held, table, ring, free, shares)]
    if ws is None:
        ws = api.new_paged_workspace(sh, api.OP_PAGED_FORK)
        ws[4096:].fill_(0xFF)
    moves = api.paged_fork(sh, t[0], t[2], t[4], t[5], t[6], t[7], fork_lens=t[1], held=t[3], workspace=ws)
    n = lambda x: None if x is None else x.cpu().numpy()
    return ws, (n(t[2]), n(t[3]), n(t[4]), n(t[5]), n(t[6]), n(t[7]), n(moves))


@pytest.mark.parametrize("R,nb,families", [(1, 1, 1), (2, 3, 1), (8, 9, 2), (64, 40, 3), (300, 5, 300), (1500, 3, 4), (33, 200, 1)])
@pytest.mark.parametrize("kind", ["all", "some", "swap", "end", "one"])
@pytest.mark.parametrize("more", [False, True])
def test_fork(api, R, nb, families, kind, more):
    rng = np.random.default_rng(R * 7 + nb)
    s = state(rng, R, nb, families, spare=R + 5, extra_held=more)
    src = {"all": rng.integers(-1, R, R), "some": np.where(rng.random(R) < 0.5, np.arange(R), rng.integers(-1, R, R)), "swap": rng.permutation(R),
           "end": np.full(R, -1), "one": np.full(R, R // 2)}[kind]
    fl = None if more else np.array([rng.integers(0, s[0][x] + 1) if x >= 0 else 0 for x in src])
    ws, got = run_fork(api, src, fl, s)
    api.check_device_status(ws)
    want = ref.fork(src, s[0], s[2], s[3], s[4], s[5], fl, s[1])
    for name, g, w in zip(("lens", "held", "table", "ring", "free", "shares", "moves"), got, want):
        if g is not None:
            assert np.array_equal(g, w), name
    # what is held and what is free make up the pool
    lens, held, table, ring, free, shares, _ = want
    held_pages = [table[r, b] for r in range(R) for b in range(held[r])]
    pool = set(held_pages) | {ring[(free[0] + i) % len(ring)] for i in range(free[1])}
    assert len(pool) == len(ring) and len(held_pages) == len(set(held_pages)) + shares.sum()


@pytest.mark.parametrize("change", ["source", "below", "long", "negative", "fork length", "ring head", "ring count", "pages", "held"])
def test_fork_that_does_not_fit_changes_nothing(api, change):
    rng = np.random.default_rng(4)
    lens, held, table, ring, free, shares = state(rng, 6, 4, 2, spare=9, extra_held=change == "held")
    lens[1] = 3 * PAGE + 5
    src, fl = np.array([1, 1, 1, 3, -1, 5]), None
    if change == "source":
        src[3] = 6
    elif change == "below":
        src[3] = -2
    elif change == "long":
        lens[5] = 4 * PAGE + 1
    elif change == "negative":
        lens[5] = -1
    elif change == "fork length":
        fl = np.array([lens[1] + 1, 0, 0, 0, 0, 0])
    elif change == "ring head":
        free[0] = len(ring)
    elif change == "ring count":
        free[1] = len(ring) + 1
    elif change == "pages":
        free[1] = 1
    else:
        held[1] = 3
    s = (lens, held, table, ring, free, shares)
    ws, got = run_fork(api, src, fl, s)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    for g, w in zip(got, s):
        assert g is None or np.array_equal(g, w)
    assert np.array_equal(got[6], np.tile([-1, -1, 0], (6, 1)))


def test_fork_passes_over_entries_that_are_no_pages(api):
    lens, table = np.array([300, 200], np.int32), np.array([[0, 99, 2, -1], [3, 4, -1, -1]], np.int32)
    ring, free, shares = np.array([5, 6, 7, -1, -1, -1, -1, -1], np.int32), np.array([0, 3], np.int32), np.zeros(8, np.int32)
    ws, got = run_fork(api, np.array([-1, 0]), None, (lens, None, table, ring, free, shares))
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert list(got[2][1]) == [0, 99, 5, -1] and list(got[6][1]) == [2, 5, 44]
    assert list(got[4]) == [1, 5] and list(got[3][3:6]) == [2, 3, 4]         # page 0 stays: the other slot holds it
    ring[0] = 8                                                              # a ring entry that is no page
    ws, got = run_fork(api, np.array([0, 0]), None, (lens, None, np.array([[0, 1, 2, -1], [3, 4, -1, -1]], np.int32), ring, free, shares))
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert list(got[2][1]) == [0, 1, -1, -1] and list(got[6][1]) == [-1, -1, 0]


@pytest.mark.parametrize("R,nb,live", [(1, 1, 1.0), (3, 5, 0.3), (40, 30, 0.9), (200, 9, 0.5), (70, 400, 0.2), (5, 3, 0.01)])
@pytest.mark.parametrize("counted", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(api, R, nb, live, counted, in_place):
    rng = np.random.default_rng(R + nb)
    lens, held, table, ring, free, shares = state(rng, R, nb, max(1, R // 3), spare=int(R * nb * (1 / live - 1) / 2) + 1, extra_held=counted)
    n_pages = len(ring)
    sh = shape(api, table, n_pages)
    lt, ht, tt, st = (None if x is None else i32(x) for x in (lens, held, table, shares if counted else None))
    ws = api.new_paged_workspace(sh, api.OP_PAGED_COMPACT)
    ws[4096:].fill_(0xFF)
    z = lambda *n: i32(np.full(n, 77))
    out = api.PagedCompact(tt, z(n_pages), z(2), st, z(max(1, n_pages // 2), 3)) if in_place else None
    p = api.paged_compact(sh, lt, tt, st, held=ht, out=out, workspace=ws)
    api.check_device_status(ws)
    for name, g, w in zip(p._fields, p, ref.compact(lens, table, n_pages, shares if counted else None, held)):
        assert (g is None) == (w is None), name
        assert w is None or np.array_equal(g.cpu().numpy(), w), name
    if not in_place:
        assert np.array_equal(tt.cpu().numpy(), table)


def test_compact_of_bad_lengths_and_entries(api):
    table = np.array([[7, 9, 1], [3, 2, 5]], np.int32)
    sh = shape(api, table, 8)
    for lens in ([400, 0], [128 * 3 + 1, -4]):
        ws = api.new_paged_workspace(sh, api.OP_PAGED_COMPACT)
        p = api.paged_compact(sh, i32(lens), i32(table), workspace=ws)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert p.block_table.cpu().numpy().tolist() == [[0, 9, 1], [3, 2, 5]]
        assert p.free_state.tolist() == [0, 6] and p.moves[0].tolist() == [7, 0, 128]


def caches(rng, n_pages, Hkv, d, di):
    import torch
    k8, v8 = (torch.from_numpy(rng.integers(0, 256, (n_pages, Hkv, PAGE, d), dtype=np.uint8)).cuda().view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (dev(rng.standard_normal((n_pages, Hkv)).astype(np.float32)) for _ in range(2))
    ki = torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, (n_pages, PAGE, di)).astype(np.int16)).cuda().view(torch.bfloat16)
    return k8, v8, ks, vs, ki


def raw(x):
    import torch
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()]).cpu().numpy().copy()


@pytest.mark.parametrize("Hkv,d,di", [(8, 128, 128), (2, 64, 64), (1, 64, 128), (300, 64, 64)])
@pytest.mark.parametrize("which", ["all", "kv", "k_idx"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_copy(api, Hkv, d, di, which, n):
    rng = np.random.default_rng(n + Hkv)
    n_pages = 2 * n + 3
    c = list(caches(rng, n_pages, Hkv, d, di))
    if which == "kv":
        c[4] = None
    elif which == "k_idx":
        c[:4] = [None] * 4
    ids = rng.permutation(n_pages)
    moves = np.stack([ids[:n], ids[n:2 * n], rng.integers(0, PAGE + 1, n)], 1)
    moves[rng.random(n) < 0.3, 0] = -1
    if n > 2:
        moves[:3] = [[ids[0], ids[n], 128], [ids[0], ids[n + 1], 1], [ids[2], ids[n + 2], 0]]     # one page to two, and scales alone
    sh = api.PagedShape(R=1, T=1, max_blocks=1, n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=d, d_idx=di, topk=1)
    want = [None if x is None else raw(x) for x in c]
    for a, b, rows in moves:
        if a < 0:
            continue
        if which != "k_idx":
            for i in (0, 1):
                want[i][b, :, :rows] = want[i][a, :, :rows]
            for i in (2, 3):
                want[i][b] = want[i][a]
        if which != "kv":
            want[4][b, :rows] = want[4][a, :rows]
    ws = api.new_paged_workspace(sh, api.OP_PAGED_COPY)
    api.paged_copy(sh, i32(moves), *c, workspace=ws)
    api.check_device_status(ws)
    for x, w in zip(c, want):
        assert x is None or np.array_equal(raw(x), w)


@pytest.mark.parametrize("bad", [[9, 1, 5], [0, 9, 5], [0, -1, 5], [0, 1, 129], [0, 1, -1]])
def test_copy_leaves_out_bad_moves(api, bad):
    rng = np.random.default_rng(1)
    c = caches(rng, 9, 2, 64, 64)
    sh = api.PagedShape(R=1, T=1, max_blocks=1, n_pages=9, Hq=2, Hkv=2, d=64, d_idx=64, topk=1)
    want = [raw(x) for x in c]
    ws = api.new_paged_workspace(sh, api.OP_PAGED_COPY)
    api.paged_copy(sh, i32([bad]), *c, workspace=ws)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    for x, w in zip(c, want):
        assert np.array_equal(raw(x), w)


@pytest.mark.parametrize("R,nb,families", [(3, 300, 2), (5, 1100, 2), (40, 513, 3), (2, 257, 1)])
@pytest.mark.parametrize("kind", ["swap", "one", "end", "half"])
def test_fork_of_long_rows(api, R, nb, families, kind):
    """Rows of more entries than a warp takes at a time; of `half`, some requests go on from a part of another's."""
    rng = np.random.default_rng(R + nb)
    s = state(rng, R, nb, families, spare=R + 5)
    src = {"swap": rng.permutation(R), "one": np.full(R, R // 2), "end": np.full(R, -1), "half": rng.integers(0, R, R)}[kind]
    fl = np.array([s[0][x] // 2 if x >= 0 else 0 for x in src]) if kind == "half" else None
    ws, got = run_fork(api, src, fl, s)
    api.check_device_status(ws)
    want = ref.fork(src, s[0], s[2], s[3], s[4], s[5], fl, s[1])
    for name, g, w in zip(("lens", "held", "table", "ring", "free", "shares", "moves"), got, want):
        if g is not None:
            assert np.array_equal(g, w), name


def test_forks_on_two_streams_at_once(api):
    """Two pools, each with its tables and its workspace; the calls of both overlap."""
    import torch
    rng = np.random.default_rng(3)
    jobs = [state(rng, 200, 40, 5, spare=205), state(rng, 64, 300, 4, spare=70)]
    want, got = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in jobs:
        R = len(s[0])
        s_src = rng.integers(-1, R, R)
        want.append(ref.fork(s_src, s[0], s[2], s[3], s[4], s[5], None, None))
        got.append((s_src, [i32(x) for x in (s_src, s[0], s[2], s[3], s[4], s[5])], shape(api, s[2], len(s[3]))))
    spaces = [api.new_paged_workspace(g[2], api.OP_PAGED_FORK) for g in got]
    torch.cuda.synchronize()
    moves = [api.paged_fork(g[2], *g[1], workspace=ws, stream=st) for g, ws, st in zip(got, spaces, streams)]
    torch.cuda.synchronize()
    for g, w, m, ws in zip(got, want, moves, spaces):
        api.check_device_status(ws)
        lens, _, table, ring, free, shares, wm = w
        for a, b in zip(g[1][1:] + [m], (lens, table, ring, free, shares, wm)):
            assert np.array_equal(a.cpu().numpy(), b)
