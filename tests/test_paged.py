"""Host side of the paged-cache calls, without a GPU: refusals before any
launch, workspace sizes, and the numpy reference's own pins."""
import ctypes

import numpy as np
import pytest

import paged_ref as ref


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api, build
    build.build()
    return api


GOOD = dict(R=4, T=8, max_blocks=16, n_pages=64, Hq=8, Hkv=2, d=64, d_idx=64, topk=4)
P = ctypes.c_void_p
OPS = ("msa_paged_plan", "msa_paged_append", "msa_paged_block_scores", "msa_paged_block_topk", "msa_paged_attn")
N_PTR = {"msa_paged_plan": 13, "msa_paged_append": 10, "msa_paged_block_scores": 7, "msa_paged_block_topk": 3, "msa_paged_attn": 11}


def call(api, fn, sh, ptrs=None, ws=P(1 << 20), n=1 << 40):
    ptrs = [P(1 << 21)] * N_PTR[fn] if ptrs is None else ptrs
    ref_ = sh if sh is None else ctypes.byref(sh.c())
    return getattr(api.lib(), fn)(ref_, *ptrs, ws, n, None), api.lib().msa_last_error().decode()


@pytest.mark.parametrize("fn", OPS)
@pytest.mark.parametrize("change,code", [
    (dict(R=0), 1), (dict(T=0), 1), (dict(max_blocks=-1), 1), (dict(n_pages=0), 1), (dict(topk=0), 1), (dict(Hq=9), 1),
    (dict(scale=float("nan")), 1), (dict(scale_idx=float("inf")), 1), (dict(scale=-1.0), 1), (dict(Hq=6), 2),
    (dict(d=96), 2), (dict(d_idx=32), 2), (dict(topk=33), 2), (dict(Hq=32, Hkv=2), 2), (dict(max_blocks=(1 << 23) + 1), 2),
    (dict(n_pages=(1 << 23) + 1), 2), (dict(T=1 << 22), 2), (dict(R=(1 << 24) + 1), 2),
    (dict(n_pages=1 << 23, Hq=512, Hkv=512), 2)])
def test_bad_shapes_are_refused_by_every_call(api, fn, change, code):
    rc, msg = call(api, fn, api.PagedShape(**{**GOOD, **change}))
    assert rc == code and msg


@pytest.mark.parametrize("fn", OPS)
def test_bad_workspaces_are_refused(api, fn):
    sh = api.PagedShape(**GOOD)
    assert call(api, fn, None)[0] == 1
    assert call(api, fn, sh, ws=None) == (1, "workspace is NULL")
    rc, msg = call(api, fn, sh, ws=P((1 << 20) + 128))
    assert rc == 1 and "256-byte" in msg
    rc, msg = call(api, fn, sh, n=255)
    assert rc == 3 and "workspace too small" in msg


@pytest.mark.parametrize("fn,optional,wide", [
    ("msa_paged_plan", {2}, set()), ("msa_paged_block_scores", set(), {0, 1}), ("msa_paged_block_topk", set(), set()),
    ("msa_paged_attn", {8}, {0, 1, 2, 9})])
def test_null_and_misaligned_pointers_are_refused(api, fn, optional, wide):
    sh = api.PagedShape(**GOOD)
    for i in range(N_PTR[fn]):
        ptrs = [P(1 << 21)] * N_PTR[fn]
        if i not in optional:
            rc, msg = call(api, fn, sh, ptrs[:i] + [None] + ptrs[i + 1:])
            assert rc == 1 and "is NULL" in msg, i
        rc, msg = call(api, fn, sh, ptrs[:i] + [P((1 << 21) + (8 if i in wide else 2))] + ptrs[i + 1:])
        assert rc == 1 and "aligned" in msg, i


def test_append_wants_whole_groups(api):
    sh, g = api.PagedShape(**GOOD), P(1 << 21)
    # k_new, v_new, k_idx_new, slots, segs, k8, v8, k_scale, v_scale, k_idx
    assert call(api, "msa_paged_append", sh, [None, None, None, g, g, None, None, None, None, None])[1].startswith("nothing")
    for i in (0, 1, 5, 6, 7, 8):
        ptrs = [g] * 10
        ptrs[i] = None
        rc, msg = call(api, "msa_paged_append", sh, ptrs)
        assert rc == 1 and "is NULL" in msg, i
    for i in (2, 9):
        ptrs = [g] * 10
        ptrs[i] = None
        rc, msg = call(api, "msa_paged_append", sh, ptrs)
        assert rc == 1 and "k_idx" in msg, i
    for i in (3, 4):
        ptrs = [g] * 10
        ptrs[i] = None
        assert call(api, "msa_paged_append", sh, ptrs)[0] == 1


def test_workspace_sizes(api):
    sh = api.PagedShape(**GOOD)
    assert api.paged_workspace_size(sh, api.OP_PAGED_APPEND) == 256
    assert api.paged_workspace_size(sh, api.OP_PAGED_PLAN) == 4096 + 256   # behind the attention's counts: 16 bytes and 16 a request
    # attention: two states of a group's heads for each stretch, two to an SM, whatever the batch; none where rows are not cut
    for kw in (GOOD, {**GOOD, "T": 384}, {**GOOD, "T": 1, "R": 1, "max_blocks": 8192}, {**GOOD, "max_blocks": 4, "topk": 5}):
        s = api.PagedShape(**kw)
        n = api.paged_workspace_size(s, api.OP_PAGED_ATTN) - 256
        assert 0 < n <= 2 * 256 * (2 * 8 * (s.d + 2) * 4) + 4096
    for kw in ({"T": 385}, {"max_blocks": 4, "topk": 4}):
        assert api.paged_workspace_size(api.PagedShape(**{**GOOD, **kw}), api.OP_PAGED_ATTN) == 256
    with pytest.raises(api.MsaError):
        api.paged_workspace_size(sh, 15)
    with pytest.raises(api.MsaError):
        api.paged_workspace_size(sh, 21)


def test_binding_refuses_host_tensors_shapes_and_types(api):
    import torch
    sh = api.PagedShape(**GOOD)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.paged_plan(sh, i32(4), i32(4), i32(4, 16), i32(64), i32(2))
    with pytest.raises(ValueError, match="block_scores"):
        api.paged_block_topk(sh, torch.zeros(8, 2, 15), i32(8))
    with pytest.raises(ValueError, match="q_idx"):
        api.paged_block_scores(sh, torch.zeros(8, 2, 64), torch.zeros(64, 128, 64), i32(4, 16), i32(5), i32(8), i32(8))
    with pytest.raises(ValueError, match="slots"):
        api.paged_append(sh, None, None, torch.zeros(8, 64, dtype=torch.bfloat16), i32(7), i32(9), None, None, None, None, torch.zeros(64, 128, 64))
    with pytest.raises(ValueError, match="q:"):
        api.paged_attn(sh, torch.zeros(8, 8, 64), None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="k8 is None"):
        api.paged_attn(sh, torch.zeros(8, 8, 64, dtype=torch.bfloat16), None, None, None, None, None, None, None)


def test_shapes_are_copied_without_their_handles(api):
    import copy
    import pickle
    sh = api.PagedShape(**GOOD)
    assert set(sh._calls) == set(range(16, 21))
    for other in (copy.deepcopy(sh), pickle.loads(pickle.dumps(sh))):
        assert other == sh and "_calls" not in vars(other) and other._calls.keys() == sh._calls.keys()


def test_binding_names_what_it_refuses(api):
    import torch
    sh = api.PagedShape(**GOOD)
    call, h = api.binding().call, sh._calls[api.OP_PAGED_BLOCK_TOPK]
    ws, s, p = torch.zeros(256, dtype=torch.uint8), torch.zeros(8, 2, 16), torch.zeros(8, dtype=torch.int32)
    for args, what in (((s, None, None), "row_pos is None"), ((s.double(), p, None), "block_scores: need a contiguous Float"),
                       ((s.transpose(0, 1).contiguous().transpose(0, 1), p, None), "contiguous=0"), ((3, p, None), "block_scores: need a tensor"),
                       ((s, p[:7], None), r"row_pos.*\[8\].*\[7\]"), ((s, p, None), "need CUDA tensors, got cpu")):
        with pytest.raises(ValueError, match=what):
            call(h, ws, *args)
    with pytest.raises(TypeError, match="3 tensors expected"):
        call(h, ws, s, p)


# ------------------------------------------------------------------ the reference's pins
def test_e4m3_reference_against_torch():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    d = ref.e4m3_decode(codes)
    assert np.array_equal(np.isnan(t), np.isnan(d)) and np.array_equal(t[~np.isnan(t)], d[~np.isnan(d)])
    fine = codes[~np.isnan(d)]
    assert np.array_equal(ref.e4m3_encode(d[~np.isnan(d)]) & 0x7F, fine & 0x7F)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(0, 0.01, 20000), 2.0 ** rng.uniform(-12, 8.8, 20000)]).astype(np.float32)
    mids = ((ref._POS[1:] + ref._POS[:-1]) / 2).astype(np.float32)         # ties
    x = np.concatenate([x, mids, -mids, [0.0, -0.0, 448.0, np.nan]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_encode(x.astype(np.float64)) & 0x7F, want & 0x7F)


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (450.0, 2.0), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7), (0.0, 2.0 ** -112),
                                       (2.0 ** -130, 2.0 ** -112), (2.0 ** 127, 2.0 ** 119), (float(np.float32(3.38e38)), 2.0 ** 120)])
def test_scale_is_the_least_power_of_two(amax, want):
    assert ref.scale_of(np.array([amax, -amax / 2, np.nan, np.inf])) == want


def test_plan_reference_conserves_pages():
    """Over many steps with requests ending and starting, no page is ever held
    twice and held + free pages stay the whole pool."""
    rng = np.random.default_rng(3)
    R, nb, n_pages, T = 6, 5, 40, 400
    table, ring = np.full((R, nb), -1, np.int32), rng.permutation(n_pages).astype(np.int32)
    lens, free = np.zeros(R, np.int32), np.array([7, n_pages], np.int32)
    for step in range(60):
        ended = (rng.random(R) < 0.2).astype(np.int32)
        room = nb * 128 - np.where(ended, 0, lens)
        new = np.minimum(rng.integers(0, 60, R), room).astype(np.int32)
        table, ring, lens, free, starts, req, pos, slots, segs = ref.plan(new, lens, table, ring, free, ended, T)
        held = [p for r in range(R) for p in table[r, :(lens[r] + 127) // 128]]
        left = [ring[(free[0] + i) % n_pages] for i in range(free[1])]
        assert sorted(held + left) == list(range(n_pages))
        n = starts[-1]
        assert len(set(slots[:n])) == n and np.all(slots[n:] == -1)


def test_the_plan_with_held_pages_is_refused_like_the_plan(api):
    sh, g = api.PagedShape(**GOOD), P(1 << 21)
    fn = lambda ptrs, ws=P(1 << 20), n=1 << 40: (api.lib().msa_paged_plan_held(ctypes.byref(sh.c()), *ptrs, ws, n, None),
                                                 api.lib().msa_last_error().decode())
    for i in range(14):                                    # 2: ended, 3: held, both may be NULL
        if i not in (2, 3):
            rc, msg = fn([g] * i + [None] + [g] * (13 - i))
            assert rc == 1 and "is NULL" in msg, i
        rc, msg = fn([g] * i + [P((1 << 21) + 2)] + [g] * (13 - i))
        assert rc == 1 and "aligned" in msg, i
    assert fn([g] * 14, ws=None) == (1, "workspace is NULL") and fn([g] * 14, n=4096)[0] == 3
    import torch
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(ValueError, match="held"):
        api.paged_plan(sh, i32(4), i32(4), i32(4, 16), i32(64), i32(2), held=i32(3))


def test_a_workspace_is_sized_by_its_own_device(api, monkeypatch):
    """The attention's scratch goes by the SMs of the device that the workspace is for, not of the current one (devices are faked)."""
    import torch
    current = [0]

    class On:
        def __init__(self, dev):
            self.to = current[0] if torch.device(dev).index is None else torch.device(dev).index

        def __enter__(self):
            self.before, current[0] = current[0], self.to

        def __exit__(self, *_):
            current[0] = self.before

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: real(n, dtype=dtype))
    monkeypatch.setattr(api, "paged_workspace_size", lambda shape, op: 8192 + 256 * current[0])
    sh = api.PagedShape(**GOOD)
    for dev, n in (("cuda:3", 3), (torch.device("cuda", 2), 2), (1, 1), ("cuda", 0), (None, 0)):
        ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN, dev)
        assert ws.numel() == 8192 + 256 * n and not ws[:4096].any() and current == [0]
