"""Rotary positions against their 64-bit definition: both pairings, part of the
head, given and implied positions up to 2^31 - 1, strides, in place, backward."""
import numpy as np
import pytest

import chunk_ref as ref
from test_gpu_paged import bf, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def radians(freqs):
    return np.array([float(int(f)) for f in freqs.cpu()]) * 2.0 ** -64 * 2 * np.pi


def angles_of(pos, freqs):
    """p f to fp64 whatever p: whole turns taken off in integers."""
    f = [int(x) for x in freqs.cpu()]
    return np.array([[((int(p) * x) % 2 ** 64) * 2.0 ** -64 * 2 * np.pi for x in f] for p in pos])


def want_of(x, pos, freqs, sh, back):
    """As ref.rotary, at angles that are exact."""
    ang = angles_of(pos, freqs)
    out = np.empty_like(x)
    for t in range(len(pos)):
        out[t] = ref.rotary(x[t:t + 1], np.array([1.0 if pos[t] >= 0 else -1.0]), ang[t], sh.d_rot or sh.d, sh.interleaved, sh.scale or 1.0, back)[0]
    return out


def check(got, x, want, sh, keep=None):
    """Cosine and sine fp32 of an angle cut to 2^-32 turns and rounded to fp32: off by 2^-22 each (2 pi 2^-25 of the rounding,
    sincospi's own 2^-23), two fp32 products and a sum 3 * 2^-24, once to bf16 2^-8 of the result."""
    mag = np.abs(x) + np.abs(x).max(2, keepdims=True)
    g = sh.scale or 1.0
    bound = 2.0 ** -8 * np.abs(want) + 2 * g * mag * 2.0 ** -21 + 1e-38
    ok = np.abs(got - want) <= bound
    rows = ~np.isnan(want[:, 0, 0])
    assert ok[rows].all(), np.max(np.abs(got - want)[rows])
    if keep is not None:
        assert np.array_equal(got[~rows], keep[~rows])


@pytest.mark.parametrize("T,Hq,Hkv,d,rot,offset,period", [(1, 1, 1, 16, 16, 0, 0), (3, 8, 2, 64, 64, 5, 0), (257, 64, 8, 128, 128, 0, 100), (33, 5, 3, 128, 32, 1000000, 7),
                                                          (9, 3, 1, 256, 240, 0, 0), (5000, 8, 2, 64, 48, 0, 1667), (17, 2, 2, 96, 96, 0, 0), (12, 130, 1, 80, 16, 2 ** 31 - 13, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_rotary(api, T, Hq, Hkv, d, rot, offset, period, inter, back):
    rng = np.random.default_rng(T + d + rot)
    sh = api.RotaryShape(T=T, Hq=Hq, Hkv=Hkv, d=d, d_rot=rot, interleaved=inter, offset=offset, period=period, scale=1.25 if T % 2 else 0.0)
    f = api.rotary_freqs(rot, 1e4 if d < 100 else 1e6)
    (q, qv), (k, kv) = (bf(rng.standard_normal((T, h, d)) * 3) for h in (Hq, Hkv))
    run = api.rotary_bwd if back else api.rotary_fwd
    qo, ko = run(sh, q, k, f)
    pos = offset + np.arange(T) % (period or T)
    some = np.arange(T) if T < 400 else rng.choice(T, 300, replace=False)
    for got, x, v in ((qo, q, qv), (ko, k, kv)):
        got = got.double().cpu().numpy()
        check(got[some], v[some], want_of(v[some], pos[some], f, sh, back), sh)
        assert np.array_equal(got[..., rot:], v[..., rot:])
    q1, none = run(sh, q, None, f)                                   # one of the two
    none2, k1 = run(sh, None, k, f)
    assert none is None and none2 is None and (q1 == qo).all() and (k1 == ko).all()


@pytest.mark.parametrize("inter", [False, True])
def test_given_positions_strides_and_in_place(api, inter):
    import torch
    rng = np.random.default_rng(7)
    T, Hq, Hkv, d, rot = 70, 8, 2, 64, 32
    pos = rng.integers(0, 1 << 20, T)
    pos[[0, 5, 69]] = 0, 2 ** 31 - 1, -1
    pos[20:30] = -1
    x, xv = bf(rng.standard_normal((T, Hq + 2 * Hkv, d)))
    sh = api.RotaryShape(T=T, Hq=Hq, Hkv=Hkv, d=d, d_rot=rot, interleaved=inter)
    f = api.rotary_freqs(rot, 5e5, factor=8.0, original_len=8192)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    qo, ko = (torch.full((T, h, d), 3.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
    assert api.rotary_fwd(sh, q, k, f, positions=i32(pos), q_out=qo, k_out=ko) == (qo, ko)
    for got, v in ((qo, xv[:, :Hq]), (ko, xv[:, Hq:Hq + Hkv])):
        check(got.double().cpu().numpy(), v, want_of(v, pos, f, sh, False), sh, np.full_like(v, 3.0))
    y = x.clone()                                                   # in place, in slices of one projection's output
    api.rotary_fwd(sh, y[:, :Hq], y[:, Hq:Hq + Hkv], f, positions=i32(pos), q_out=y[:, :Hq], k_out=y[:, Hq:Hq + Hkv])
    live = i32(pos) >= 0
    assert torch.equal(y[live][:, :Hq], qo[live]) and torch.equal(y[live][:, Hq:Hq + Hkv], ko[live])
    assert torch.equal(y[~live], x[~live]) and torch.equal(y[:, Hq + Hkv:], x[:, Hq + Hkv:])
    b = x.view(2, 35, Hq + 2 * Hkv, d)[:, :, :Hq]                   # leading dimensions as a training batch has them
    assert torch.equal(api.rotary_fwd(sh, b, None, f, positions=i32(np.abs(pos)))[0].view(T, Hq, d),
                       api.rotary_fwd(sh, q.contiguous(), None, f, positions=i32(np.abs(pos)))[0])


def test_backward_is_the_gradient(api):
    """Against differences of the forward pass' definition, and as the transposed map: <dy, R x> = <R^T dy, x>."""
    rng = np.random.default_rng(3)
    for inter in (False, True):
        T, H, d, rot = 13, 3, 32, 16
        sh = api.RotaryShape(T=T, Hq=H, Hkv=1, d=d, d_rot=rot, interleaved=inter, scale=1.5)
        f = api.rotary_freqs(rot)
        (x, xv), (dy, dyv) = (bf(rng.standard_normal((T, H, d))) for _ in range(2))
        dx = api.rotary_bwd(sh, dy, None, f)[0].double().cpu().numpy()
        loss = lambda v: float((ref.rotary(v, np.arange(T, dtype=float), radians(f), rot, inter, 1.5, False) * dyv).sum())
        for _ in range(20):
            at = tuple(rng.integers(n) for n in xv.shape)
            up, dn = xv.copy(), xv.copy()
            up[at] += 0.5
            dn[at] -= 0.5
            assert abs(loss(up) - loss(dn) - dx[at]) <= 2.0 ** -8 * abs(dx[at]) + 1e-5      # linear: the difference is the gradient
        y = api.rotary_fwd(sh, x, None, f)[0].double().cpu().numpy()
        slack = 2.0 ** -8 * (np.abs(y * dyv).sum() + np.abs(dx * xv).sum())
        assert abs((y * dyv).sum() - (dx * xv).sum()) <= slack


def test_special_values_stay_in_their_pairs(api):
    import torch
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 1, 3], x[1, 0, 40] = float("nan"), float("inf")
    sh = api.RotaryShape(T=2, Hq=2, Hkv=1, d=64, d_rot=32)
    y = api.rotary_fwd(sh, x, None, api.rotary_freqs(32), positions=i32([5, 9]))[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 1, 3] = bad[0, 1, 19] = bad[1, 0, 40] = True
    assert torch.equal(~torch.isfinite(y), bad)


def test_on_a_stream_and_in_a_graph(api):
    import torch
    rng = np.random.default_rng(5)
    q, _ = bf(rng.standard_normal((40, 8, 128)))
    k, _ = bf(rng.standard_normal((40, 2, 128)))
    sh, f = api.RotaryShape(T=40, Hq=8, Hkv=2, d=128), api.rotary_freqs(128)
    want = api.rotary_fwd(sh, q, k, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = api.rotary_fwd(sh, q, k, f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.rotary_fwd(sh, q, k, f)
        back = api.rotary_bwd(sh, *out, f)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0] * 2) and torch.equal(back[0], api.rotary_bwd(sh, want[0] * 2, None, f)[0])


def test_tensors_without_memory_of_their_own_are_refused(api):
    """Expanded tensors have one token's memory for all, or one head's: neither as inputs nor as outputs."""
    import torch
    sh = api.RotaryShape(T=6, Hq=4, Hkv=2, d=64)
    f = api.rotary_freqs(64)
    z = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    q = z(6, 4, 64)
    for bad in (z(1, 4, 64).expand(6, 4, 64), z(6, 1, 64).expand(6, 4, 64), z(1, 3, 4, 64).expand(2, 3, 4, 64), z(2, 1, 4, 64).expand(2, 3, 4, 64)):
        with pytest.raises(ValueError, match="q: need"):
            api.rotary_fwd(sh, bad, None, f)
        with pytest.raises(ValueError, match="q_out: need"):
            api.rotary_fwd(sh, q, None, f, q_out=bad)
    assert not q.any()
