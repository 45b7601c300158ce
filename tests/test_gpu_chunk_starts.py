"""Chunk calls whose q_starts do not fit: rows that belong to no request are left as they were."""
import numpy as np
import pytest

from test_gpu_chunks import run_chunk
from test_gpu_paged import attn_case, bf, i32, lay_out

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def scores(api, lens, starts, T, Hkv=2):
    import torch
    rng = np.random.default_rng(5)
    table, n_pages = lay_out(lens, rng, max_blocks=6)
    qt, _ = bf(rng.standard_normal((T, Hkv, 64)))
    kt, _ = bf(rng.standard_normal((n_pages, PAGE, 64)))
    pos = np.arange(T) + 150
    sh = api.PagedShape(R=len(lens), T=T, max_blocks=6, n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=64, d_idx=64, topk=4)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_SCORES)
    out = torch.full((T, Hkv, 6), 5.0, device="cuda")
    api.paged_chunk_scores(sh, qt, kt, i32(table), i32(starts), i32(pos), block_scores=out, workspace=ws)
    return ws, out


@pytest.mark.parametrize("T,Hkv", [(3, 2), (40, 8), (2, 300)])
def test_scores_of_requests_that_are_left_out(api, T, Hkv):
    for starts in ([T, 0], [0, T + 1], [-1, 2], [0, -3]):
        ws, out = scores(api, [300], starts, T, Hkv)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert (out == 5.0).all(), starts


def test_scores_of_the_requests_beside_one_that_is_left_out(api):
    T = 30
    _, good = scores(api, [300, 300, 300], [4, 14, 20, 28], T)
    assert (good[:4] == 5.0).all() and (good[28:] == 5.0).all() and not (good[4:28] == 5.0).any()
    ws, out = scores(api, [300, 300, 300], [4, 14, 20, T + 9], T)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert (out[4:20] == good[4:20]).all() and (out[:4] == 5.0).all() and (out[20:] == 5.0).all()
