"""Chunk calls whose q_starts go back: a request that begins in rows of an earlier one is left out, the others are as ever."""
import numpy as np
import pytest

import chunk_ref
import paged_ref as ref
from test_gpu_chunks import run_chunk
from test_gpu_paged import bf, dev, f8, filled_cache, i32, lay_out, pick

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def owners(starts, T):
    """Each row's request (-1: none), of those that fit and begin behind every earlier one that does."""
    req, end = np.full(T, -1), 0
    for r, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        if not 0 <= a <= b <= T:
            continue
        if a >= end:
            req[a:b] = r
        end = max(end, b)
    return req


def long_starts(R, back_at, by):
    steps = np.array([1 + i % 3 for i in range(R)])
    s = np.concatenate([[0], np.cumsum(steps)])
    s[back_at:] -= by
    return list(s)


CASES = {"short": [0, 10, 5, 8], "twice": [3, 20, 12, 30, 25, 40], "past the end": [0, 9, 60, 9, 21], "all of one": [0, 40, 2, 30, 40],
         "another CTA's width": long_starts(1500, 1200, 7), "at its border": long_starts(1300, 1024, 5), "early": long_starts(2100, 40, 30)}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("sparse", [True, False])
def test_starts_that_go_back(api, case, sparse):
    import torch
    starts = CASES[case]
    R, T = len(starts) - 1, max(40, starts[-1])
    Hq, Hkv, d, k = 4, 2, 64, 2
    rng = np.random.default_rng(R)
    lens = [int(x) for x in rng.integers(1, 300, R)]
    table, n_pages = lay_out(lens, rng, max_blocks=3)
    req = owners(starts, T)
    assert (req >= 0).any() and len(set(starts)) > len(set(req))
    pos = np.array([rng.integers(0, lens[r]) if r >= 0 else 2 for r in req])
    qt, qv = bf(rng.standard_normal((T, Hq, d)))
    (k8, ks), (v8, vs) = (filled_cache(rng, n_pages, Hkv, d, table, lens) for _ in range(2))
    sel = pick(rng, pos, Hkv, k) if sparse else None
    sh = api.PagedShape(R=R, T=T, max_blocks=3, n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=64, topk=k)
    args = (qt, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), None, i32(pos))
    ws, o, lse = run_chunk(api, sh, args, starts, sel, T, status=False)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    ow, lw, do, dl = chunk_ref.attn(qv, k8, v8, ks, vs, table, req, pos, sel, float(np.float32(1) / np.sqrt(np.float32(d))))
    o, lse, on = o.double().cpu().numpy(), lse.double().cpu().numpy(), req >= 0
    assert np.all(o[~on] == 3.0) and np.all(lse[~on] == 3.0)
    assert np.all(np.abs(lse - lw)[on] <= dl[on]) and np.all(np.abs(o - ow)[on] <= do[on])
    if sparse:
        return
    qi, qiv = bf(rng.standard_normal((T, Hkv, 64)))
    ki, kiv = bf(rng.standard_normal((n_pages, PAGE, 64)))
    ws, out = api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_SCORES), torch.full((T, Hkv, 3), 5.0, device="cuda")
    api.paged_chunk_scores(sh, qi, ki, i32(table), i32(starts), i32(pos), block_scores=out, workspace=ws)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    want, mag = ref.block_scores(qiv, kiv, table, req, pos, 0.125)
    got = out.double().cpu().numpy()
    assert np.all(got[~on] == 5.0) and np.array_equal(np.isneginf(got[on]), np.isneginf(want[on]))
    fine = on[:, None, None] & np.isfinite(want)
    assert np.all(np.abs(got[fine] - want[fine]) <= mag[fine] * (64 * 2.0 ** -23) + np.abs(want[fine]) * 2.0 ** -22 + 1e-30)
