"""Rotary positions of as many tokens as an int holds."""
import numpy as np
import pytest

import chunk_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 3])
def test_tokens_up_to_the_largest_int(api, T):
    """68 GB in place, one head of 16 features; the last tokens, and some across 2^32 elements, against their definition."""
    import torch
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 68 GB of device memory")
    some = np.array([0, 1, 2 ** 28 - 1, 2 ** 28, T - 5, T - 4, T - 3, T - 2, T - 1])
    rng = np.random.default_rng(1)
    x = torch.empty(T, 1, 16, dtype=torch.bfloat16, device="cuda")
    at = torch.from_numpy(some).cuda()
    v = torch.from_numpy(rng.standard_normal((len(some), 1, 16)).astype(np.float32)).bfloat16()
    x[at] = v.cuda()
    sh, f = api.RotaryShape(T=T, Hq=1, Hkv=1, d=16), api.rotary_freqs(16)
    api.rotary_fwd(sh, x, None, f, q_out=x)
    got = x[at].double().cpu().numpy()
    xv = v.double().numpy()
    for i, p in enumerate(some):
        turns = np.array([((int(p) * int(w)) % 2 ** 64) * 2.0 ** -64 * 2 * np.pi for w in f.cpu()])
        want = ref.rotary(xv[i:i + 1], np.array([1.0]), turns, 16, False, 1.0, False)[0]
        # cosine and sine off by 2^-22 each, products and sums in fp32, once to bf16
        assert np.all(np.abs(got[i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(xv[i]).max()), p
