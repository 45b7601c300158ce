"""What rotary calls leave in the outputs of tokens without a position."""
import numpy as np
import pytest

from test_gpu_paged import bf, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T", [7, 6000])
@pytest.mark.parametrize("back", [False, True])
def test_fresh_outputs_of_tokens_without_a_position_are_zeros(api, inter, T, back):
    import torch
    rng = np.random.default_rng(T)
    sh, f = api.RotaryShape(T=T, Hq=8, Hkv=2, d=64, d_rot=32, interleaved=inter), api.rotary_freqs(32)
    (q, _), (k, _) = (bf(rng.standard_normal((T, h, 64))) for h in (8, 2))
    pos = rng.integers(-1, 50, T)
    pos[[0, 2, T - 1]] = -1, 9, -(2 ** 31)
    p, live = i32(pos), torch.tensor(pos >= 0, device="cuda")
    run = api.rotary_bwd if back else api.rotary_fwd
    for h in (8, 2):                                     # the memory that the outputs are going to have held something
        x = torch.full((T, h, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        del x
    qo, ko = run(sh, q, k, f, positions=p)
    assert not qo[~live].view(torch.int16).any() and not ko[~live].view(torch.int16).any()
    names = ("dq", "dk") if back else ("q_out", "k_out")
    q3, k3 = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    for given, mine, other, fresh in ((0, q3, 1, ko), (1, k3, 0, qo)):          # one given, one not
        out = run(sh, q, k, f, positions=p, **{names[given]: mine})
        assert out[given] is mine and (mine[~live] == 3.0).all() and torch.equal(mine[live], (qo, ko)[given][live])
        assert torch.equal(out[other], fresh)
    y = q.clone()
    run(sh, y, None, f, positions=p, **{names[0]: y})     # in place: left as it was
    assert torch.equal(y[~live], q[~live]) and torch.equal(y[live], qo[live])
