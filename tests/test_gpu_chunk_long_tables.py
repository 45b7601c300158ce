"""Tables of more blocks than a union is taken of in one go, forks and compactions over large tables."""
import numpy as np
import pytest

import chunk_ref
import paged_ref as ref
from test_gpu_chunks import check_chunk
from test_gpu_fork import run_fork, shape, state
from test_gpu_paged import bf, dev, f8, filled_cache, i32

pytestmark = pytest.mark.gpu

PAGE, WINDOW = 128, 1 << 15


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def long_table(rng, nb, n_pages=6):
    return rng.integers(0, n_pages, (1, nb)).astype(np.int32)


@pytest.mark.parametrize("nb", [WINDOW + 1, WINDOW + 300, 2 * WINDOW + 77])
@pytest.mark.parametrize("Hq,Hkv,T", [(8, 1, 20), (2, 2, 150)])
def test_a_union_of_blocks_on_both_sides_of_a_window(api, nb, Hq, Hkv, T):
    """A prompt of millions of tokens in a few pages that its table names again and again."""
    rng = np.random.default_rng(nb)
    d, k, n_pages = 64, 9, 6
    table = long_table(rng, nb)
    pos = np.sort(rng.integers((nb - 1) * PAGE, nb * PAGE, T))
    qt, qv = bf(rng.standard_normal((T, Hq, d)))
    own = [n_pages * PAGE]                                       # every token of every page is written
    (k8, ks), (v8, vs) = (filled_cache(rng, n_pages, Hkv, d, np.arange(n_pages)[None], own) for _ in range(2))
    sel = np.full((T, Hkv, k), -1, np.int32)
    near = [b for b in (0, 31, 32, WINDOW - 1, WINDOW, WINDOW + 31, 2 * WINDOW - 1, 2 * WINDOW) if b < nb]
    for t in range(T):
        for h in range(Hkv):
            c = np.unique(np.concatenate([rng.choice(near, 3), rng.integers(0, nb, 4), [nb - 1]]))
            sel[t, h, :len(c)] = c
    sel[3] = -1                                                  # a row with blocks in one window only, and one without any
    sel[3, :, :2] = 5, WINDOW - 1
    sel[4] = -1
    sh = api.PagedShape(R=1, T=T, max_blocks=nb, n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=64, topk=k)
    args = (qt, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), None, i32(pos))
    r = (qv, k8, v8, ks, vs, table, np.zeros(T, int), pos, sel, float(np.float32(1) / np.sqrt(np.float32(d))))
    check_chunk(api, sh, args, [0, T], sel, r, T)


def test_scores_over_a_long_table(api):
    rng = np.random.default_rng(1)
    nb, T, n_pages = WINDOW + 300, 3, 6
    table, pos = long_table(rng, nb), np.array([nb * PAGE - 1, WINDOW * PAGE, 77])
    qt, qv = bf(rng.standard_normal((T, 2, 64)))
    kt, kv = bf(rng.standard_normal((n_pages, PAGE, 64)))
    sh = api.PagedShape(R=1, T=T, max_blocks=nb, n_pages=n_pages, Hq=2, Hkv=2, d=64, d_idx=64, topk=4)
    got = api.paged_chunk_scores(sh, qt, kt, i32(table), i32([0, T]), i32(pos)).double().cpu().numpy()
    want, mag = ref.block_scores(qv, kv, table, np.zeros(T, int), pos, 0.125)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= mag[fine] * (64 * 2.0 ** -23) + np.abs(want[fine]) * 2.0 ** -22)


@pytest.mark.parametrize("R,nb,kind", [(700, 1300, "swap"), (700, 1300, "half"), (20000, 12, "all")])
def test_fork_of_many_entries(api, R, nb, kind):
    rng = np.random.default_rng(R + nb)
    s = state(rng, R, nb, R // 6, spare=R + 5)
    src = {"swap": rng.permutation(R), "half": rng.integers(0, R, R), "all": rng.integers(-1, R, R)}[kind]
    fl = np.array([s[0][x] // 2 if x >= 0 else 0 for x in src]) if kind == "half" else None
    ws, got = run_fork(api, src, fl, s)
    api.check_device_status(ws)
    want = chunk_ref.fork(src, s[0], s[2], s[3], s[4], s[5], fl, s[1])
    for name, g, w in zip(("lens", "held", "table", "ring", "free", "shares", "moves"), got, want):
        if g is not None:
            assert np.array_equal(g, w), name


@pytest.mark.parametrize("R,nb,spare", [(900, 2000, 500000), (30000, 20, 2500000)])
def test_compaction_of_millions_of_pages(api, R, nb, spare):
    rng = np.random.default_rng(R)
    lens, held, table, ring, free, shares = state(rng, R, nb, R // 3, spare=spare)
    n_pages = len(ring)
    sh = shape(api, table, n_pages)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_COMPACT)
    ws[4096:].fill_(0xFF)
    p = api.paged_compact(sh, i32(lens), i32(table), i32(shares), workspace=ws)
    api.check_device_status(ws)
    for name, g, w in zip(p._fields, p, chunk_ref.compact(lens, table, n_pages, shares)):
        assert np.array_equal(g.cpu().numpy(), w), name
