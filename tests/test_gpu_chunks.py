"""Chunks of new tokens over the paged cache: scores and attention against
their 64-bit definitions, and whole serving steps with shared prompts."""
import numpy as np
import pytest

import chunk_ref
import paged_ref as ref
from test_gpu_paged import CASES, attn_case, bf, dev, f8, i32, lay_out, rows_of

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def starts_of(q):
    return np.concatenate([[0], np.cumsum(q)]).astype(np.int32)


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("Hkv,di,lens,q,pad", [
    (1, 64, [1], [1], 0), (2, 64, [127, 128, 129, 300], [1, 40, 129, 7], 3), (8, 128, [1000, 40, 700], [70, 40, 1], 0), (4, 64, [2500], [900], 5),
    (3, 128, [513, 260], [100, 200], 0), (300, 64, [200, 130], [2, 3], 1), (5, 64, [40, 1, 0, 200], [40, 1, 0, 3], 2),
    (8, 128, [150 + 61 * i for i in range(30)], [1 + 5 * i for i in range(30)], 9)])
@pytest.mark.parametrize("order", ["up", "shuffled"])
def test_chunk_scores(api, Hkv, di, lens, q, pad, order):
    import torch
    rng = np.random.default_rng(Hkv + di + sum(lens))
    table, n_pages = lay_out(lens, rng, max_blocks=max(1, max(lens) // PAGE + 2))
    starts, req, pos = rows_of(lens, q, pad)
    T, n = len(req), sum(q)
    if order == "shuffled":
        for r in range(len(q)):
            rng.shuffle(pos[starts[r]:starts[r + 1]])
        if n > 3:
            pos[2] = -1                                   # a row that is left as it was
    qt, qv = bf(rng.standard_normal((T, Hkv, di)))
    own = np.zeros((n_pages, PAGE), bool)
    for r, m in enumerate(lens):
        for j in range(m):
            own[table[r, j // PAGE], j % PAGE] = True
    kf = rng.standard_normal((n_pages, PAGE, di))
    kf[~own] = np.nan
    kt, kv = bf(kf)
    sh = api.PagedShape(R=len(lens), T=T, max_blocks=table.shape[1], n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=64, d_idx=di, topk=4)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_SCORES)
    ws[4096:].fill_(0xFF)
    out = torch.full((T, Hkv, table.shape[1]), 5.0, device="cuda")
    api.paged_chunk_scores(sh, qt, kt, i32(table), i32(starts), i32(pos), block_scores=out, workspace=ws)
    api.check_device_status(ws)
    assert not ws[:4096].any()
    live = np.where(pos >= 0, req, -1)
    want, mag = ref.block_scores(qv, kv, table, live, pos, float(np.float32(1) / np.sqrt(np.float32(di))))
    got = out.double().cpu().numpy()
    left = live < 0
    assert np.all(got[left] == 5.0)
    got, want, mag = got[~left], want[~left], mag[~left]
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    # sums of di exact products, each step off by 2^-23 of the sum of magnitudes; the scale's product
    assert np.all(np.abs(got - want)[fine] <= (mag * (di * 2.0 ** -23) + np.abs(want) * 2.0 ** -22 + 1e-30)[fine])


def test_chunk_scores_pass_over_a_page_out_of_range(api):
    import torch
    rng = np.random.default_rng(2)
    lens, q = [700], [90]
    table, n_pages = lay_out(lens, rng)
    starts, req, pos = rows_of(lens, q, 0)
    qt, _ = bf(rng.standard_normal((90, 2, 64)))
    kt, _ = bf(rng.standard_normal((n_pages, PAGE, 64)))
    sh = api.PagedShape(R=1, T=90, max_blocks=6, n_pages=n_pages, Hq=2, Hkv=2, d=64, d_idx=64, topk=4)
    good = api.paged_chunk_scores(sh, qt, kt, i32(table), i32(starts), i32(pos))
    for page in (-1, n_pages, 2 ** 31 - 1):
        table[0, 3] = page
        ws = api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_SCORES)
        got = api.paged_chunk_scores(sh, qt, kt, i32(table), i32(starts), i32(pos), workspace=ws)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        want = good.clone()
        want[:, :, 3] = -float("inf")
        assert torch.equal(got, want)


# ------------------------------------------------------------------ attention
CHUNKS = [
    dict(lens=[300], q=[300], Hq=8, Hkv=1, d=128, k=3), dict(lens=[700, 1500, 40], q=[129, 64, 40], Hq=8, Hkv=2, d=64, k=4, pad=3),
    dict(lens=[2000, 1, 900], q=[33, 1, 500], Hq=16, Hkv=8, d=128, k=8, max_blocks=30), dict(lens=[1300, 260], q=[260, 250], Hq=2, Hkv=2, d=64, k=4),
    dict(lens=[5000], q=[17], Hq=16, Hkv=2, d=128, k=16), dict(lens=[0, 130, 0, 128, 129], q=[0, 5, 0, 128, 1], Hq=4, Hkv=1, d=128, k=2),
    dict(lens=[9000], q=[40], Hq=8, Hkv=1, d=64, k=32), dict(lens=[128 * 5], q=[128 * 5], Hq=8, Hkv=8, d=128, k=1)]


def run_chunk(api, sh, args, starts, sel, n, status=True):
    """args as attn_case gives them."""
    import torch
    ws = api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_ATTN)
    ws[4096:].fill_(0xFF)
    o = torch.full((sh.T, sh.Hq, sh.d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sh.T, sh.Hq), 3.0, device="cuda")
    api.paged_chunk_attn(sh, *args[:6], i32(starts), args[7], sel_idx=None if sel is None else i32(sel), o=o, lse=lse, workspace=ws)
    if status:
        api.check_device_status(ws)
        assert not ws[:4096].any()
    return ws, o, lse


def check_chunk(api, sh, args, starts, sel, r, n):
    ws, o, lse = run_chunk(api, sh, args, starts, sel, n)
    ow, lw, do, dl = chunk_ref.attn(*r)
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    left = (r[6] < 0) | (r[7] < 0)
    assert np.all(og[left] == 3.0) and np.all(lg[left] == 3.0)
    og, lg, ow, lw, do, dl = (x[~left] for x in (og, lg, ow, lw, do, dl))
    none = np.isneginf(lw)
    assert np.array_equal(none, np.isneginf(lg)) and np.all(og[none] == 0)
    assert np.all(np.abs(lg - lw)[~none] <= dl[~none]), np.max((np.abs(lg - lw) / dl)[~none])
    assert np.all(np.abs(og - ow) <= do + 1e-30), np.max((np.abs(og - ow) / (do + 1e-30)))


@pytest.mark.parametrize("case", range(len(CHUNKS) + len(CASES)))
@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_attention(api, case, sparse):
    c = (CHUNKS + CASES)[case]
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    check_chunk(api, sh, args, starts_of(c["q"]), sel, r, sum(c["q"]))


@pytest.mark.parametrize("kw", [dict(gain=30.0), dict(gain=1e-3), dict(scale=0.7), dict(qgain=1e-6), dict(qgain=100.0), dict(gain=2.0 ** 60, qgain=2.0 ** -62)])
def test_chunk_attention_of_other_magnitudes(api, kw):
    c = dict(lens=[700, 260], q=[100, 20], Hq=8, Hkv=2, d=128, k=3)
    sh, args, sel, r = attn_case(api, sparse=True, **c, **kw)
    check_chunk(api, sh, args, starts_of(c["q"]), sel, r, 120)


@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_positions_in_any_order(api, sparse):
    from test_gpu_paged import pick
    c = dict(lens=[900, 400], q=[300, 50], Hq=8, Hkv=2, d=64, k=4)
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    rng = np.random.default_rng(8)
    pos = r[7].copy()
    rng.shuffle(pos[:300])
    pos[300:] = 200                                   # equal ones
    pos[[7, 310]] = -1                                # rows that are left as they were
    if sparse:
        sel = pick(rng, pos, 2, 4)
    args = args[:7] + (i32(pos),)
    check_chunk(api, sh, args, starts_of(c["q"]), sel, r[:7] + (pos, sel) + r[9:], 350)


def test_chunk_rows_without_blocks_and_gaps_in_the_selection(api):
    c = dict(lens=[1500, 700], q=[40, 30], Hq=8, Hkv=2, d=64, k=8)
    sh, args, sel, r = attn_case(api, sparse=True, **c)
    sel[0, 0] = -1
    sel[1, 1] = [-1, 3, -1, -1, 5, 7, -1, 8]
    sel[40:, 1] = -1                                  # a whole tile without any block
    check_chunk(api, sh, args, starts_of(c["q"]), sel, r[:8] + (sel,) + r[9:], 70)


def test_chunk_attention_leaves_out_bad_entries(api):
    import torch
    c = dict(lens=[1500], q=[3], Hq=4, Hkv=1, d=64, k=4)
    sh, args, sel, r = attn_case(api, sparse=True, **c)
    base = np.array([[[2, 7, 9, 11]], [[0, 1, 2, 11]], [[3, 4, 5, 11]]], np.int32)

    def run(row, table=None):
        s = base.copy()
        s[1, 0] = row
        a = args if table is None else args[:5] + (table,) + args[6:]
        return run_chunk(api, sh, a, [0, 3], s, 3, status=False)

    for bad, same in (([2, 2, 5, 11], [2, -1, 5, 11]), ([5, 2, 7, 11], [5, -1, 7, 11]), ([2, 7, 11, 12], [2, 7, 11, -1]),
                      ([2, 7, 11, 2 ** 31 - 1], [2, 7, 11, -1]), ([2, -5, 7, 11], [2, -1, 7, 11])):
        ws, o, l = run(bad)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        ws, o2, l2 = run(same)
        api.check_device_status(ws)
        assert torch.equal(o, o2) and torch.equal(l, l2), bad
    for page in (-1, sh.n_pages, 2 ** 31 - 1):
        table = args[5].clone()
        table[0, 7] = page
        ws, o, l = run([2, 7, 8, 11], table)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        b0 = base.copy()
        b0[0, 0, 1] = -1
        b0[1, 0] = [2, -1, 8, 11]
        _, o2, l2 = run_chunk(api, sh, args, [0, 3], b0, 3)
        assert torch.equal(o, o2) and torch.equal(l, l2)
    _, o2, l2 = run_chunk(api, sh, args, [0, 3], base, 3)
    pos = args[7].clone()
    pos[1] = 12 * PAGE
    ws, o, l = run_chunk(api, sh, args[:7] + (pos,), [0, 3], base, 3, status=False)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    # the row's blocks are in no union now, and the others' pages add up in another order: each is within its bound of the definition
    ow, lw, do, dl = chunk_ref.attn(*r[:8], base, r[9])
    assert (o[1] == 3.0).all() and all((np.abs(o[t].double().cpu().numpy() - ow[t]) <= do[t]).all() and (np.abs(l[t].double().cpu().numpy() - lw[t]) <= dl[t]).all() for t in (0, 2))
    for starts in ([3, 0], [0, 4], [-1, 2], [0, -3]):
        ws, o, l = run_chunk(api, sh, args, starts, base, 3, status=False)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert (o == 3.0).all() and (l == 3.0).all()


@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_nan_reaches_only_its_rows(api, sparse):
    """A NaN query head spoils itself; a NaN key code the rows of its group that see the token; a NaN value code one feature of them."""
    import torch
    c = dict(lens=[400, 300], q=[200, 10], Hq=8, Hkv=2, d=64, k=2)
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    pos, table = r[7], r[5]
    sees = lambda t, j, g: pos[t] >= j and (sel is None or j // PAGE in sel[t, g])
    _, o0, l0 = run_chunk(api, sh, args, [0, 200, 210], sel, 210)
    q = args[0].clone()
    q[5, 3, 7] = float("nan")
    _, o, l = run_chunk(api, sh, (q,) + args[1:], [0, 200, 210], sel, 210)
    hit = torch.zeros(210, 8, dtype=torch.bool, device="cuda")
    hit[5, 3] = True
    assert torch.equal(torch.isnan(l), hit) and torch.equal(o[~hit], o0[~hit]) and torch.isnan(o[hit]).all()
    for j in (10, 330, 399):                                       # a token of the first request, group 1
        want = torch.tensor([[r[6][t] == 0 and h >= 4 and sees(t, j, 1) for h in range(8)] for t in range(210)], device="cuda")
        for which in (1, 2):
            a = list(args)
            codes = a[which].clone()
            codes.view(torch.uint8)[table[0, j // PAGE], 1, j % PAGE, 9] = 0xFF
            a[which] = codes
            _, o, l = run_chunk(api, sh, tuple(a), [0, 200, 210], sel, 210)
            assert torch.equal(o[~want], o0[~want]) and torch.equal(l[~want], l0[~want]), (j, which)
            if which == 1:
                assert torch.isnan(l[want]).all() and torch.isnan(o[want]).all()
            else:
                assert torch.equal(l, l0) and torch.isnan(o[want][:, 9]).all() and not torch.isnan(o[want][:, :9]).any() and not torch.isnan(o[want][:, 10:]).any()


def test_chunk_small_probabilities_keep_their_bits(api):
    """Thousands of tokens under a sink whose values are zero: what they weigh together is the answer, at any distance."""
    import torch
    n, d, T = 4000, 64, 20
    rng = np.random.default_rng(0)
    table, n_pages = lay_out([n], rng)
    for far in (10.0, 30.0, 60.0):
        q = np.zeros((T, 8, d))
        q[..., 0] = far * np.sqrt(d) / 4
        k, v = np.zeros((n_pages, 1, PAGE, d)), np.zeros((n_pages, 1, PAGE, d))
        v[:] = rng.integers(1, 9, v.shape)
        k[table[0, 0], 0, 0, 0] = 4.0                                # the sink: a logit of `far`, the others' are 0
        v[table[0, 0], 0, 0] = 0
        ones = np.ones((n_pages, 1), np.float32)
        qt, qv = bf(q)
        pos = np.arange(n - T, n)
        r = (qv, ref.e4m3_encode(k), ref.e4m3_encode(v), ones, ones, table, np.zeros(T, int), pos, None, float(np.float32(1) / np.sqrt(np.float32(d))))
        sh = api.PagedShape(R=1, T=T, max_blocks=table.shape[1], n_pages=n_pages, Hq=8, Hkv=1, d=d, d_idx=64, topk=1)
        check_chunk(api, sh, (qt, f8(r[1]), f8(r[2]), dev(ones), dev(ones), i32(table), None, i32(pos)), [0, T], None, r, T)


def test_chunk_attention_agrees_with_itself_and_the_row_calls(api):
    import torch
    c = dict(lens=[3000, 1700, 20], q=[200, 130, 20], Hq=16, Hkv=4, d=128, k=8)
    sh, args, sel, r = attn_case(api, sparse=True, **c)
    for s in (sel, None):
        _, o, l = run_chunk(api, sh, args, starts_of(c["q"]), s, 350)
        for _ in range(3):
            _, o2, l2 = run_chunk(api, sh, args, starts_of(c["q"]), s, 350)
            assert torch.equal(o, o2) and torch.equal(l, l2)
        o3, l3 = api.paged_attn(sh, *args, sel_idx=None if s is None else i32(s))
        assert (l - l3).abs().max() < 1e-4 and ((o - o3).float().norm() / o3.float().norm()) < 2.0 ** -7


def test_chunk_offsets_past_32_bits(api):
    """Pages at the end of a pool of more than 2^32 bytes."""
    import torch
    n_pages, Hq, Hkv, d = 36000, 8, 8, 128
    rng = np.random.default_rng(1)
    k8, v8 = (torch.zeros(n_pages, Hkv, PAGE, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(n_pages, Hkv, device="cuda") for _ in range(2))
    ki = torch.zeros(n_pages, PAGE, 128, dtype=torch.bfloat16, device="cuda")
    pages = [n_pages - 1, 0, n_pages - 7]
    small = rng.integers(0, 0x60, (2, 3, Hkv, PAGE, d), dtype=np.uint8)
    kidx, kidxv = bf(rng.standard_normal((3, PAGE, 128)))
    for i, page in enumerate(pages):
        k8[page], v8[page], ki[page] = dev(small[0, i]), dev(small[1, i]), kidx[i]
    q, qv = bf(rng.standard_normal((60, Hq, d)) * 0.05)
    pos = np.arange(300, 360)
    sh = api.PagedShape(R=1, T=60, max_blocks=3, n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=128, topk=2)
    args = (q, k8.view(torch.float8_e4m3fn), v8.view(torch.float8_e4m3fn), ks, vs, i32([pages]), None, i32(pos))
    one = np.ones((3, Hkv), np.float32)
    r = (qv, small[0], small[1], one, one, np.array([[0, 1, 2]]), np.zeros(60, int), pos, None, float(np.float32(1) / np.sqrt(np.float32(d))))
    check_chunk(api, sh, args, [0, 60], None, r, 60)
    got = api.paged_chunk_scores(sh, q, ki, i32([pages]), i32([0, 60]), i32(pos)).double().cpu().numpy()
    want, mag = ref.block_scores(qv, kidxv, np.array([[0, 1, 2]]), np.zeros(60, int), pos, float(np.float32(1) / np.sqrt(np.float32(d))))
    assert np.all(np.abs(got - want) <= mag * 2.0 ** -16 + np.abs(want) * 2.0 ** -22)
    api.paged_copy(sh, i32([[n_pages - 1, n_pages - 2, 77]]), *args[1:5], ki)
    assert torch.equal(k8[n_pages - 2, :, :77], k8[n_pages - 1, :, :77]) and not k8[n_pages - 2, :, 77:].any()
    assert torch.equal(ki[n_pages - 2, :77], ki[n_pages - 1, :77])


# ------------------------------------------------------------------ a run of them
@pytest.mark.parametrize("graph", [False, True])
def test_prompts_shared_and_served_in_chunks(api, graph):
    """A prompt in two chunks, requests that go on from it, their own chunk, some ends and a compaction: what the rows attend
    to is what each request's own tokens say, whatever the pages."""
    import torch
    rng = np.random.default_rng(11)
    Hq, Hkv, d, di, k, R, nb = 8, 2, 64, 64, 3, 4, 8
    n_pages, T = 24, 512
    sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=di, topk=k)
    rsh, ish = api.RotaryShape(T=T, Hq=Hq, Hkv=Hkv, d=d), api.RotaryShape(T=T, Hq=Hkv, Hkv=1, d=di, d_rot=32)
    f, fi = api.rotary_freqs(d), api.rotary_freqs(32)
    k8, v8 = (torch.full((n_pages, Hkv, PAGE, d), 0xFF, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((n_pages, Hkv), float("nan"), device="cuda") for _ in range(2))
    ki = torch.full((n_pages, PAGE, di), float("nan"), dtype=torch.bfloat16, device="cuda")
    lens, table = i32(np.zeros(R)), i32(np.full((R, nb), -1))
    ring, free, shares = i32(rng.permutation(n_pages)), i32([0, n_pages]), i32(np.zeros(n_pages))
    ws = torch.zeros(max(api.paged_workspace_size(sh, op) for op in (*range(16, 21), *range(32, 37))), dtype=torch.uint8, device="cuda")
    new, src = i32(np.zeros(R)), i32(np.arange(R))
    x = {n: torch.zeros(T, h, w, dtype=torch.bfloat16, device="cuda") for n, h, w in (("q", Hq, d), ("k", Hkv, d), ("v", Hkv, d), ("qi", Hkv, di), ("ki", 1, di))}
    box = {}

    def step():
        moves = api.paged_fork(sh, src, lens, table, ring, free, shares, workspace=ws)
        api.paged_copy(sh, moves, k8, v8, ks, vs, ki, workspace=ws)
        p = api.paged_plan(sh, new, lens, table, ring, free, workspace=ws)
        lens.copy_(p.lens)
        free.copy_(p.free_state)
        q, kk = api.rotary_fwd(rsh, x["q"], x["k"], f, positions=p.row_pos)
        qi, kki = api.rotary_fwd(ish, x["qi"], x["ki"], fi, positions=p.row_pos)
        api.paged_append(sh, kk, x["v"], kki[:, 0], p.slots, p.segs, k8, v8, ks, vs, ki, workspace=ws)
        s = api.paged_chunk_scores(sh, qi, ki, table, p.q_starts, p.row_pos, workspace=ws)
        sel = api.paged_block_topk(sh, s, p.row_pos, workspace=ws)
        o, lse = api.paged_chunk_attn(sh, q, k8, v8, ks, vs, table, p.q_starts, p.row_pos, sel_idx=sel, workspace=ws)
        dense = api.paged_chunk_attn(sh, q, k8, v8, ks, vs, table, p.q_starts, p.row_pos, workspace=ws)
        box.update(o=o, lse=lse, dense=dense, sel=sel, p=p, q=q, kk=kk, s=s)

    if graph:
        step()                                       # an idle step: handles and kernels are there
        api.check_device_status(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    text = [[] for _ in range(R)]                    # per request the values of its tokens (k turned, v) as they were given
    for it, (n_new, n_src) in enumerate([([300, 0, 0, 0], [0, 1, 2, 3]), ([150, 0, 0, 7], [0, 1, 2, 3]), ([5, 200, 1, 0], [0, 0, 0, 3]),
                                         ([1, 1, 130, 1], [1, 1, 0, 3]), ([0, 3, 0, 300], [0, 1, -1, 1])]):
        new.copy_(i32(n_new))
        src.copy_(i32(n_src))
        for n in x:
            x[n].copy_(bf(rng.standard_normal(x[n].shape))[0])
        g.replay() if graph else step()
        api.check_device_status(ws)
        was = [list(t) for t in text]
        text = [was[s] if s >= 0 else [] for s in n_src]
        text = [list(t) for t in text]
        kk, vv, t0 = box["kk"].double().cpu().numpy(), x["v"].double().cpu().numpy(), 0
        pos = box["p"].row_pos.cpu().numpy()
        for r in range(R):
            for i in range(n_new[r]):
                assert pos[t0 + i] == len(text[r])
                text[r].append((kk[t0 + i], vv[t0 + i]))
            t0 += n_new[r]
        assert np.array_equal(lens.cpu().numpy(), [len(t) for t in text])
        sel, q = box["sel"].cpu().numpy(), box["q"].double().cpu().numpy()
        req, n = box["p"].row_req.cpu().numpy(), sum(n_new)
        for t in rng.choice(n, min(n, 25), replace=False):
            K, V = (np.stack([row[i] for row in text[req[t]]])[:pos[t] + 1] for i in (0, 1))
            for (o, _), blocks in (((box["o"], 0), sel[t]), (box["dense"], None)):
                for h in range(Hq):
                    seen = np.ones(len(K), bool) if blocks is None else np.isin(np.arange(len(K)) // PAGE, blocks[h // 4])
                    s = K[seen, h // 4] @ q[t, h] / np.sqrt(d)
                    e = np.exp(s - s.max())
                    want = e / e.sum() @ V[seen, h // 4]
                    got = o[t, h].double().cpu().numpy()
                    # e4m3 keeps 4 bits of keys and values: a twentieth of the values' size, by far
                    assert np.abs(got - want).max() < 0.25 and np.linalg.norm(got - want) < 0.05 * np.sqrt(d)
        if it == 3 and not graph:
            c = api.paged_compact(sh, lens, table, shares, workspace=ws)
            api.paged_copy(sh, c.moves, k8, v8, ks, vs, ki, workspace=ws)
            for a, b in ((table, c.block_table), (ring, c.free_pages), (free, c.free_state), (shares, c.shares)):
                a.copy_(b)
            api.check_device_status(ws)
    used = int(n_pages - free[1].item())
    tb, ln = table.cpu().numpy(), lens.cpu().numpy()
    held = {int(tb[r, b]) for r in range(R) for b in range(-(-ln[r] // PAGE))}
    assert len(held) == used                         # no page is lost


@pytest.mark.parametrize("G,Hkv", [(8, 2), (4, 1), (1, 3)])
@pytest.mark.parametrize("stretch", [1, 3, 9])
def test_chunk_blocks_that_one_half_of_a_tile_selects(api, G, Hkv, stretch):
    """Runs of blocks that only the first, or only the last, rows of a tile have."""
    rng = np.random.default_rng(G + stretch)
    tokens = 256 // G
    lens, q = [7000, 300], [2 * tokens + tokens // 2 + 3, 5]
    sh, args, _, r = attn_case(api, lens=lens, q=q, Hq=G * Hkv, Hkv=Hkv, d=64, k=24, sparse=True)
    pos, sel = r[7], np.full((sh.T, Hkv, 24), -1, np.int32)
    for t, p in enumerate(pos):
        late = (t % tokens) >= tokens // 2
        for g in range(Hkv):
            c = [b for b in range(p // PAGE) if (b // stretch % 2 == 1) == late]
            c = sorted(rng.choice(c, min(len(c), 20 if t % 5 else 3), replace=False)) if c else []
            c += [p // PAGE] if t % 3 else []
            sel[t, g, :len(c)] = c[:24]
    # a row's list holds no more entries than it has blocks
    for t, p in enumerate(pos):
        sel[t, :, min(24, p // PAGE + 1):] = -1
    check_chunk(api, sh, args, starts_of(q), sel, r[:8] + (sel,) + r[9:], sh.T)


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_extreme_queries_stay_in_their_rows(api, value, sparse):
    import torch
    c = dict(lens=[700, 300], q=[150, 10], Hq=8, Hkv=2, d=64, k=3)
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    _, o0, l0 = run_chunk(api, sh, args, [0, 150, 160], sel, 160)
    q = args[0].clone()
    q[40, 6, 11], q[155, 1, :] = value, value
    _, o, l = run_chunk(api, sh, (q,) + args[1:], [0, 150, 160], sel, 160)
    hit = torch.zeros(160, 8, dtype=torch.bool, device="cuda")
    hit[40, 6] = hit[155, 1] = True
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(l[~hit], l0[~hit])
    if np.isinf(value):
        assert not torch.isfinite(l[hit]).any()


def test_chunk_calls_on_two_streams_at_once(api):
    import torch
    jobs = []
    for c, sparse in ((dict(lens=[3000, 1700], q=[300, 130], Hq=16, Hkv=4, d=128, k=8), True), (dict(lens=[2000], q=[500], Hq=8, Hkv=2, d=64, k=4), False)):
        sh, args, sel, r = attn_case(api, sparse=sparse, **c)
        jobs.append((sh, args[:6] + (i32(starts_of(c["q"])), args[7]), None if sel is None else i32(sel)))
    alone = [api.paged_chunk_attn(sh, *a, sel_idx=s) for sh, a, s in jobs]
    spaces = [api.new_paged_workspace(sh, api.OP_PAGED_CHUNK_ATTN) for sh, _, _ in jobs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[api.paged_chunk_attn(sh, *a, sel_idx=s, workspace=ws, stream=st) for (sh, a, s), ws, st in zip(jobs, spaces, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    for both in got:
        for (o, l), (o0, l0) in zip(both, alone):
            assert torch.equal(o, o0) and torch.equal(l, l0)
    for ws in spaces:
        api.check_device_status(ws)


def test_one_workspace_for_all_calls_and_shapes(api):
    """A workspace of the largest need serves smaller shapes and the other calls in between."""
    import torch
    big = attn_case(api, sparse=True, lens=[3000, 1700, 20], q=[200, 130, 20], Hq=16, Hkv=4, d=128, k=8)
    small = attn_case(api, sparse=False, lens=[130, 1], q=[5, 1], Hq=8, Hkv=2, d=64, k=4)
    calls = [(big[0], big[1], i32(big[2]), [200, 130, 20]), (small[0], small[1], None, [5, 1])]
    ws = api.new_paged_workspace(big[0], api.OP_PAGED_CHUNK_ATTN)
    need = max(api.new_paged_workspace(c[0], op).numel() for c in calls for op in (api.OP_PAGED_CHUNK_ATTN, api.OP_PAGED_CHUNK_SCORES))
    assert ws.numel() >= need
    run = lambda c, w: api.paged_chunk_attn(c[0], *c[1][:6], i32(starts_of(c[3])), c[1][7], sel_idx=c[2], workspace=w)
    first = [run(c, None) for c in calls]
    kx, _ = bf(np.random.default_rng(0).standard_normal((small[0].n_pages, PAGE, 64)))
    qx, _ = bf(np.random.default_rng(1).standard_normal((small[0].T, 2, 64)))
    for _ in range(3):
        for c, f in zip(calls, first):
            o, l = run(c, ws)
            n = sum(c[3])
            assert torch.equal(o[:n], f[0][:n]) and torch.equal(l[:n], f[1][:n])
            api.paged_chunk_scores(small[0], qx, kx, small[1][5], i32(starts_of([5, 1])), small[1][7], workspace=ws)
    api.check_device_status(ws)
    assert not ws[:4096].any()


@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_calls_with_a_page_twice_and_single_tokens(api, sparse):
    """Requests whose tables name one page at several blocks, most of them without rows, the others with one."""
    q = [0] * 400 + [1] * 70 + [0] * 30 + [2]
    c = dict(lens=[0] * 400 + [200 + 11 * i for i in range(70)] + [0] * 30 + [900], q=q, Hq=8, Hkv=2, d=64, k=4)
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    table = r[5].copy()
    table[410:420, 1] = table[410:420, 0]
    table[-1, 1:] = table[-1, 0]
    check_chunk(api, sh, args[:5] + (i32(table),) + args[6:], starts_of(q), sel, r[:5] + (table,) + r[6:], sum(q))
