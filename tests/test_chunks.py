"""Host side of the forking, compaction, copy, chunk and rotary calls, without
a GPU: refusals before any launch, workspace sizes, frequencies."""
import ctypes
import math

import numpy as np
import pytest

import chunk_ref as ref


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api, build
    build.build()
    return api


GOOD = dict(R=4, T=8, max_blocks=16, n_pages=64, Hq=8, Hkv=2, d=64, d_idx=64, topk=4)
P = ctypes.c_void_p
# pointers of each call, those that may be NULL, those of 16-byte alignment
CALLS = {"msa_paged_fork": (9, {1, 3}, set()), "msa_paged_compact": (9, {1}, set()), "msa_paged_copy": (6, {5}, {1, 2, 5}),
         "msa_paged_chunk_scores": (6, set(), {0, 1}), "msa_paged_chunk_attn": (11, {8}, {0, 1, 2, 9})}


def call(api, fn, sh, ptrs=None, ws=P(1 << 20), n=1 << 40, moves=4):
    ptrs = [P(1 << 21)] * CALLS[fn][0] if ptrs is None else list(ptrs)
    if fn == "msa_paged_copy":
        ptrs[1:1] = [moves]
    return getattr(api.lib(), fn)(sh if sh is None else ctypes.byref(sh.c()), *ptrs, ws, n, None), api.lib().msa_last_error().decode()


@pytest.mark.parametrize("fn", CALLS)
@pytest.mark.parametrize("change,code", [(dict(R=0), 1), (dict(T=0), 1), (dict(n_pages=0), 1), (dict(Hq=9), 1), (dict(scale=-1.0), 1), (dict(Hq=6), 2),
                                         (dict(d=96), 2), (dict(topk=33), 2), (dict(max_blocks=(1 << 23) + 1), 2), (dict(T=1 << 22), 2)])
def test_bad_shapes_are_refused_by_every_call(api, fn, change, code):
    rc, msg = call(api, fn, api.PagedShape(**{**GOOD, **change}))
    assert rc == code and msg


@pytest.mark.parametrize("fn", CALLS)
def test_bad_workspaces_and_pointers_are_refused(api, fn):
    sh = api.PagedShape(**GOOD)
    assert call(api, fn, None)[0] == 1
    assert call(api, fn, sh, ws=None) == (1, "workspace is NULL")
    assert call(api, fn, sh, ws=P((1 << 20) + 128))[0] == 1
    assert call(api, fn, sh, n=255)[0] == 3
    count, optional, wide = CALLS[fn]
    for i in range(count):
        ptrs = [P(1 << 21)] * count
        if i not in optional:
            rc, msg = call(api, fn, sh, ptrs[:i] + [None] + ptrs[i + 1:])
            assert rc == 1 and "NULL" in msg, i
        rc, msg = call(api, fn, sh, ptrs[:i] + [P((1 << 21) + (8 if i in wide else 2))] + ptrs[i + 1:])
        assert rc == 1 and "aligned" in msg, i


def test_copy_and_compact_want_whole_groups(api):
    sh, g = api.PagedShape(**GOOD), P(1 << 21)
    assert call(api, "msa_paged_copy", sh, [g] + [None] * 5)[1].startswith("nothing")
    for moves in (0, -1, (1 << 24) + 1):
        assert call(api, "msa_paged_copy", sh, moves=moves)[0] == 1
    for i in (3, 7):
        ptrs = [g] * 9
        ptrs[i] = None
        rc, msg = call(api, "msa_paged_compact", sh, ptrs)
        assert rc == 1 and "shares" in msg


def test_workspaces_grow_with_the_shape(api):
    small, big = api.PagedShape(**GOOD), api.PagedShape(**{**GOOD, "R": 40, "T": 500, "n_pages": 5000})
    for op in (api.OP_PAGED_FORK, api.OP_PAGED_COMPACT, api.OP_PAGED_CHUNK_SCORES, api.OP_PAGED_CHUNK_ATTN):
        a, b = api.paged_workspace_size(small, op), api.paged_workspace_size(big, op)
        assert 4096 <= a <= b and a % 256 == b % 256 == 0
    # a key by page, three numbers by request, one by piece of a row, a copy of the table
    assert api.paged_workspace_size(big, api.OP_PAGED_FORK) >= 4096 + 5000 * 8 + 40 * 12 + 40 * 4 + 40 * 16 * 4
    with pytest.raises(api.MsaError):
        api.paged_workspace_size(small, 37)


ROT = dict(T=8, Hq=4, Hkv=2, d=64, d_rot=32)


def turn(api, fn="msa_rotary_fwd", sh=None, ptrs=None, **strides):
    c = (sh or api.RotaryShape(**ROT)).c()
    for n, v in strides.items():
        setattr(c, n, v)
    rc = getattr(api.lib(), fn)(ctypes.byref(c), *([P(1 << 21)] * 2 + [None] + [P(1 << 21)] + [P(1 << 22)] * 2 if ptrs is None else ptrs), None)
    return rc, api.lib().msa_last_error().decode()


@pytest.mark.parametrize("fn", ["msa_rotary_fwd", "msa_rotary_bwd"])
@pytest.mark.parametrize("change,code", [
    (dict(T=0), 1), (dict(Hq=0), 1), (dict(d_rot=80), 1), (dict(period=-1), 1), (dict(offset=-1), 1), (dict(scale=float("inf")), 1),
    (dict(scale=-1.0), 1), (dict(offset=2 ** 31 - 8), 0), (dict(offset=2 ** 31 - 7), 1), (dict(d=72), 2), (dict(d=272), 2), (dict(d_rot=8), 2), (dict(Hq=40000), 2)])
def test_rotary_refuses_bad_shapes(api, fn, change, code):
    if code:
        rc, msg = turn(api, fn, api.RotaryShape(**{**ROT, **change}))
        assert rc == code and msg
    else:                                       # passes the shape's checks: stopped by the next one
        assert turn(api, fn, api.RotaryShape(**{**ROT, **change}), [P(1 << 21)] * 2 + [None, None] + [P(1 << 22)] * 2)[1] == "freqs is NULL"


def test_rotary_refuses_bad_pointers_and_strides(api):
    g, h = P(1 << 21), P(1 << 22)
    good = [g, g, None, g, h, h]
    assert turn(api, ptrs=[None, None, None, g, None, None])[1].startswith("nothing")
    for i, p, what in ((0, None, "q is NULL"), (1, None, "k is NULL"), (3, None, "freqs is NULL"), (4, None, "q_out is NULL"), (5, None, "k_out is NULL"),
                       (0, P((1 << 21) + 8), "q is not 16"), (5, P((1 << 22) + 8), "k_out is not 16"), (3, P((1 << 21) + 4), "freqs is not 8"),
                       (2, P((1 << 21) + 2), "positions is not 4")):
        rc, msg = turn(api, ptrs=good[:i] + [p] + good[i + 1:])
        assert rc == 1 and what in msg
    for kw in (dict(q_stride=255), dict(q_stride=260), dict(k_out_stride=64), dict(q_out_stride=-8), dict(k_stride=1 << 33)):
        assert turn(api, **kw)[0] == 1
    assert "another stride" in turn(api, ptrs=[g, None, None, g, g, None], q_stride=512)[1]
    assert api.lib().msa_rotary_fwd(None, *good, None) == 1


def test_rotary_frequencies(api):
    got = [int(x) for x in api.rotary_freqs(64, 1e4, device="cpu")]
    for i, x in enumerate(got):                 # fp64 arithmetic, a few parts in 2^53, to the nearest whole number
        want = 1e4 ** (-i / 32) / (2 * math.pi) * 2.0 ** 64
        assert abs(x - want) <= want * 2.0 ** -50 + 0.5
    halved = api.rotary_freqs(64, 1e4, factor=2.0, device="cpu")
    assert all(abs(int(a) * 2 - b) <= 2 + b * 2.0 ** -50 for a, b in zip(halved, got))
    parts = [int(x) for x in api.rotary_freqs(64, 1e4, factor=8.0, original_len=4096, device="cpu")]
    for i, x in enumerate(parts):
        turns = 4096 * 1e4 ** (-i / 32) / (2 * math.pi)
        keep = min(1, max(0, (turns - 1) / 3))
        assert abs(x - got[i] * (keep + (1 - keep) / 8)) <= got[i] * 2.0 ** -48 + 1
    assert parts[0] == got[0] and abs(parts[-1] * 8 - got[-1]) <= 8 + got[-1] * 2.0 ** -50
    assert api.rotary_scale(1.0) == 1.0 and abs(api.rotary_scale(8.0) - (1 + 0.1 * math.log(8))) < 1e-15
    for bad in (dict(d_rot=7), dict(d_rot=0), dict(d_rot=64, base=1.0), dict(d_rot=64, factor=0.5), dict(d_rot=64, original_len=-1), dict(d_rot=64, low=4.0, high=4.0)):
        with pytest.raises(ValueError):
            api.rotary_freqs(**bad, device="cpu")


def test_python_calls_refuse_host_tensors(api):
    import torch
    sh = api.PagedShape(**GOOD)
    z = lambda *n: torch.zeros(n, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for run in (lambda: api.paged_fork(sh, z(4), z(4), z(4, 16), z(64), z(2), z(64), workspace=ws), lambda: api.paged_compact(sh, z(4), z(4, 16), workspace=ws),
                lambda: api.paged_copy(sh, z(3, 3), None, None, None, None, torch.zeros(64, 128, 64, dtype=torch.bfloat16), workspace=ws)):
        with pytest.raises(ValueError, match="CUDA"):
            run()
    with pytest.raises(ValueError, match="shares"):
        api.paged_fork(sh, z(4), z(4), z(4, 16), z(64), z(2), z(63), workspace=ws)
    r = api.RotaryShape(**ROT)
    with pytest.raises(ValueError, match="CUDA"):
        api.rotary_fwd(r, torch.zeros(8, 4, 64, dtype=torch.bfloat16), None, torch.zeros(16, dtype=torch.int64))


def test_reference_pins():
    # two requests change places: nothing is given back, each takes a page of its own for its last tokens
    lens, held, table, ring, free, shares, moves = ref.fork(np.array([1, 0]), np.array([300, 129]), np.array([[0, 1, 2], [3, 4, 9]]), np.array([5, 6, 7, 8, 0, 0, 0, 0, 0, 0]),
                                                            np.array([0, 4]), np.zeros(10, int))
    assert table.tolist() == [[3, 5, 2], [0, 1, 6]] and lens.tolist() == [129, 300] and moves.tolist() == [[4, 5, 1], [2, 6, 44]]
    assert free.tolist() == [2, 4] and ring[4:6].tolist() == [2, 4] and not shares.any()
    # three go on from one; one ends
    out = ref.fork(np.array([0, 0, 0, -1]), np.array([256, 128, 1, 200]), np.array([[0, 1], [2, 9], [3, 9], [4, 5]]), np.arange(10), np.array([6, 4]), np.zeros(10, int))
    assert out[2].tolist() == [[0, 1], [0, 1], [0, 1], [4, 5]] and out[5].tolist() == [2, 2] + [0] * 8 and out[4].tolist() == [6, 8]
    t, ring, free, _, moves = ref.compact(np.array([200, 1]), np.array([[7, 0], [5, -1]]), 8)
    assert t.tolist() == [[2, 0], [1, -1]]
    assert moves[:2].tolist() == [[5, 1, 128], [7, 2, 128]] and free.tolist() == [0, 5] and ring[:5].tolist() == [3, 4, 5, 6, 7]
