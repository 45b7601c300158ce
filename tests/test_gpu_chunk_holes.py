"""Chunk calls over many short requests, some of whose tables name no page at all."""
import numpy as np
import pytest

from test_gpu_chunks import run_chunk, starts_of
from test_gpu_paged import attn_case, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


@pytest.mark.parametrize("sparse", [True, False])
@pytest.mark.parametrize("bad", [[5], [70, 71, 72, 73], [0, 1, 198, 199], list(range(20, 60)) + [90], list(range(200))])
def test_requests_without_any_page(api, sparse, bad):
    """Each is eight items (a tile and a group) without a page, one after another in a CTA's stretch; all the others' rows are
    what they are with whole tables."""
    import torch
    lens = [40 + 37 * (i % 9) for i in range(200)]
    q = [1 + i % 6 for i in range(200)]
    sh, args, sel, r = attn_case(api, lens=lens, q=q, Hq=16, Hkv=8, d=64, k=2, sparse=sparse)
    n = sum(q)
    _, o0, l0 = run_chunk(api, sh, args, starts_of(q), sel, n)
    table = r[5].copy()
    table[bad] = -1
    ws, o, l = run_chunk(api, sh, args[:5] + (i32(table),) + args[6:], starts_of(q), sel, n, status=False)
    with pytest.raises(api.MsaError) as e:
        api.check_device_status(ws)
    assert "TIMEOUT" not in str(e.value).upper()
    hit = torch.tensor(np.isin(r[6], bad), device="cuda")
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(l[~hit], l0[~hit])
    assert not o[hit].any() and torch.isneginf(l[hit]).all()


def test_long_requests_between_requests_without_any_page(api):
    """Pages, ends and empty items in turn, tiles cut."""
    import torch
    lens, q = [2000, 300, 300, 1500, 200, 1, 900, 128], [50, 9, 1, 3, 200, 1, 300, 40]
    sh, args, sel, r = attn_case(api, lens=lens, q=q, Hq=8, Hkv=8, d=128, k=2, sparse=False)
    n = sum(q)
    _, o0, l0 = run_chunk(api, sh, args, starts_of(q), None, n)
    for bad in ([1, 2], [4, 5], [0], [7], [1, 2, 3, 4, 5, 6, 7]):
        table = r[5].copy()
        table[bad] = 2 ** 30
        ws, o, l = run_chunk(api, sh, args[:5] + (i32(table),) + args[6:], starts_of(q), None, n, status=False)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        hit = torch.tensor(np.isin(r[6], bad), device="cuda")
        assert torch.equal(o[~hit], o0[~hit]) and torch.equal(l[~hit], l0[~hit]), bad
        assert not o[hit].any() and torch.isneginf(l[hit]).all()
