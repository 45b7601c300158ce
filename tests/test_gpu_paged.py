"""The paged-cache operators against their 64-bit definitions (paged_ref): the
step's plan, the quantising append, block scores, block selection and
attention over the 8-bit cache, one by one and as a serving loop runs them."""
import numpy as np
import pytest

import paged_ref as ref
from msa_testutil import to_torch

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def bf(a):
    """float array -> (bf16 tensor, the values it holds in 64 bits)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


def f8(codes):
    import torch
    return torch.from_numpy(codes.copy()).cuda().view(torch.float8_e4m3fn)


def status_ok(api, ws):
    api.check_device_status(ws)


def lay_out(lens, rng, max_blocks=None, spare=3):
    """A block table for the lengths over randomly ordered pages; unused entries hold garbage."""
    need = [(n + PAGE - 1) // PAGE for n in lens]
    nb = max_blocks or max(1, max(need))
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages)
    table = rng.integers(-2 ** 31, 2 ** 31 - 1, (len(lens), nb)).astype(np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at:at + m]
        at += m
    return table, n_pages


def rows_of(lens, q, pad):
    starts = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    req = np.concatenate([np.repeat(np.arange(len(q)), q), np.full(pad, -1)]).astype(np.int32)
    pos = np.concatenate([[lens[r] - q[r] + i for r in range(len(q)) for i in range(q[r])], np.full(pad, -1)]).astype(np.int32)
    return starts, req, pos


# ------------------------------------------------------------------ plan
def run_plan(api, sh, new, lens, table, ring, free, ended, inplace=False):
    import torch
    t = [i32(x) for x in (new, lens, table, ring, free)]
    e = None if ended is None else i32(ended)
    out = None
    if inplace:
        z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
        out = api.PagedPlan(t[1], t[4], z(sh.R + 1), z(sh.T), z(sh.T), z(sh.T), z(sh.n_segs + 1))
    ws = api.new_paged_workspace(sh, api.OP_PAGED_PLAN)
    ws[256:].fill_(0xFF)
    p = api.paged_plan(sh, *t, ended=e, workspace=ws, out=out)
    n = lambda x: x.cpu().numpy()
    return ws, (n(t[2]), n(t[3]), n(p.lens), n(p.free_state), n(p.q_starts), n(p.row_req), n(p.row_pos), n(p.slots), n(p.segs))


@pytest.mark.parametrize("R,T,nb,top,ends", [(1, 1, 1, 1, False), (1, 1000, 9, 1000, False), (7, 64, 3, 9, True), (64, 64, 20, 1, True),
                                             (33, 5000, 40, 150, True), (2500, 2600, 2, 1, True), (1100, 9000, 4, 8, True)])
@pytest.mark.parametrize("inplace", [False, True])
def test_plan(api, R, T, nb, top, ends, inplace):
    rng = np.random.default_rng(R * 31 + T)
    new = rng.integers(0, top + 1, R)
    new[rng.random(R) < 0.1] = 0
    new = np.minimum(new, nb * PAGE)
    while new.sum() > T:
        new[rng.integers(R)] = 0
    lens = np.minimum(rng.integers(0, nb * PAGE + 1, R), nb * PAGE - new)
    lens[rng.random(R) < 0.2] = 0
    ended = (rng.random(R) < 0.2).astype(np.int32) if ends else None    # some slots end and start anew in the same step
    held = (lens + PAGE - 1) // PAGE
    n_pages = int(held.sum() + ((new + PAGE - 1) // PAGE + 1).sum() + 5)
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((R, nb), -7, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    head, count = int(rng.integers(n_pages)), n_pages - at
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(count)) % n_pages] = ids[at:]
    sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=8, Hkv=2, d=64, d_idx=64, topk=4)
    ws, got = run_plan(api, sh, new, lens, table, ring, [head, count], ended, inplace)
    status_ok(api, ws)
    want = ref.plan(new, lens, table, ring, [head, count], ended, T)
    for name, g, w in zip(("table", "ring", "lens", "free", "q_starts", "row_req", "row_pos", "slots", "segs"), got, want):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("T", [40, 4500])
@pytest.mark.parametrize("change", ["rows", "pages", "long", "negative", "negative length", "ring head", "ring count"])
def test_plan_that_does_not_fit_changes_nothing(api, T, change):
    new, lens, ended = np.array([3, 5, 0, 2]), np.array([126, 0, 300, 128]), np.array([0, 0, 1, 0])
    table, ring, free = np.arange(12).reshape(4, 3).astype(np.int32), np.arange(100, 120).astype(np.int32), [4, 6]
    if change == "rows":
        T, new[1] = 8, 4
    if change == "pages":
        free = [4, 2]          # takes three
    if change == "long":
        new[3] = 257
    if change == "negative":
        new[0] = -1
    if change == "negative length":
        lens[0] = -1
    if change == "ring head":
        free = [20, 6]
    if change == "ring count":
        free = [4, 18]         # three pages come back: 21 of 20
    sh = api.PagedShape(R=4, T=T, max_blocks=3, n_pages=20, Hq=8, Hkv=2, d=64, d_idx=64, topk=4)
    ws, got = run_plan(api, sh, new, lens, table, ring, free, ended)
    with pytest.raises(api.MsaError, match="MSA_ERR_DEVICE"):
        api.check_device_status(ws)
    assert np.array_equal(got[0], table) and np.array_equal(got[1], ring) and np.array_equal(got[2], lens) and np.array_equal(got[3], free)
    assert np.all(got[4] == 0) and np.all(got[5] == -1) and np.all(got[6] == -1) and np.all(got[7] == -1) and np.all(got[8] == 0)
    status_ok(api, ws)         # the word was cleared


def test_plan_gives_no_slot_on_a_page_out_of_range(api):
    """A ring entry that is no page: its rows get no slot, the others do, and the append leaves them out."""
    import torch
    sh = api.PagedShape(R=2, T=4, max_blocks=2, n_pages=4, Hq=2, Hkv=1, d=64, d_idx=64, topk=2)
    ws, got = run_plan(api, sh, [2, 2], [0, 0], np.full((2, 2), -1, np.int32), np.array([9, 3, 0, 1], np.int32), [0, 4], None)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert got[7].tolist() == [-1, -1, 3 * PAGE, 3 * PAGE + 1]
    ki = torch.zeros(4, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    new, val = bf(np.random.default_rng(0).standard_normal((4, 64)))
    ws = api.new_paged_workspace(sh, api.OP_PAGED_APPEND)
    api.paged_append(sh, None, None, new, i32(got[7]), i32(got[8]), None, None, None, None, ki, workspace=ws)
    status_ok(api, ws)
    want = np.zeros((4, PAGE, 64))
    want[3, :2] = val[2:]
    assert np.array_equal(ki.double().cpu().numpy(), want)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("Hkv,d,di,old,new", [
    (2, 64, 64, [0], [1]), (8, 128, 128, [0, 127, 128, 5, 100], [1, 1, 1, 1, 1]), (1, 128, 64, [3, 0, 120, 64], [300, 128, 9, 63]),
    (3, 64, 128, [0, 255], [1000, 2])])
@pytest.mark.parametrize("kind", ["normal", "wide", "special"])
def test_append(api, Hkv, d, di, old, new, kind):
    rng = np.random.default_rng(len(old) * 100 + Hkv + len(kind))
    old, new = np.array(old), np.array(new)
    lens = old + new
    table, n_pages = lay_out(lens, rng)
    starts, req, pos = rows_of(lens, new, 3)
    T = len(req)
    slots = np.where(req >= 0, table[req, np.maximum(pos, 0) // PAGE].astype(np.int64) * PAGE + pos % PAGE, -1).astype(np.int32)
    sh = api.PagedShape(R=len(old), T=T, max_blocks=table.shape[1], n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=d, d_idx=di, topk=2)
    first = [t for t in range(starts[-1]) if t in starts or pos[t] % PAGE == 0]
    segs = np.array(first + [starts[-1]] * (sh.n_segs + 1 - len(first)), np.int32)

    def rows(*shape):
        x = rng.standard_normal(shape)
        if kind == "wide":                              # scales that grow, and values that end among the subnormals
            x = x * 2.0 ** rng.integers(-18, 14, shape)
        if kind == "special":
            x = np.where(rng.random(shape) < 0.02, rng.choice([0.0, np.inf, -np.inf, np.nan, 3.3e38, -1e-40], shape), x)
            x[rng.integers(shape[0])] = 0.0
        return bf(x)

    codes = {n: rng.integers(0, 256, (n_pages, Hkv, PAGE, d)).astype(np.uint8) for n in "kv"}
    scales = {n: (2.0 ** rng.integers(-12, 3, (n_pages, Hkv))).astype(np.float32) for n in "kv"}
    t8 = {n: f8(codes[n]) for n in "kv"}
    ts = {n: dev(scales[n]) for n in "kv"}
    (kn, kv), (vn, vv) = rows(T, Hkv, d), rows(T, Hkv, d)
    kin, _ = bf(rng.standard_normal((T, di)))
    ki, _ = bf(rng.standard_normal((n_pages, PAGE, di)))
    want_ki = ki.clone()
    ws = api.new_paged_workspace(sh, api.OP_PAGED_APPEND)
    import torch
    for _ in range(2):                                  # again: the same rows to the same slots change nothing
        api.paged_append(sh, kn, vn, kin, i32(slots), i32(segs), t8["k"], t8["v"], ts["k"], ts["v"], ki, workspace=ws)
        status_ok(api, ws)
        if _ == 0:
            for n, x in (("k", kv), ("v", vv)):
                ref.append(x, slots, segs, codes[n], scales[n])
            for t in range(starts[-1]):
                want_ki[slots[t] // PAGE, slots[t] % PAGE] = kin[t]
        for n in "kv":
            assert np.array_equal(ts[n].cpu().numpy(), scales[n]), n
            got = t8[n].view(torch.uint8).cpu().numpy()
            same = (got == codes[n]) | ((got & 0x7F == 0x7F) & (codes[n] & 0x7F == 0x7F))   # any NaN for a NaN
            assert same.all(), (n, np.argwhere(~same)[:5])
        assert torch.equal(ki.view(torch.int16), want_ki.view(torch.int16))


def test_append_leaves_out_bad_segments(api):
    """A slot past the pool and a segment that runs off its page: recorded, nothing written."""
    import torch
    sh = api.PagedShape(R=2, T=300, max_blocks=4, n_pages=3, Hq=2, Hkv=1, d=64, d_idx=64, topk=2)
    new, _ = bf(np.ones((300, 64)))
    for slots0, segs in ((3 * PAGE, [0, 1]), (2 * PAGE + 100, [0, 100]), (0, [0, 129]), (0, [-4, 2]), (0, [0, 301])):
        ki = torch.zeros(3, PAGE, 64, dtype=torch.bfloat16, device="cuda")
        ws = api.new_paged_workspace(sh, api.OP_PAGED_APPEND)
        slots = np.full(300, slots0, np.int32)
        sg = np.array(segs + [segs[-1]] * (sh.n_segs - 1), np.int32)
        api.paged_append(sh, None, None, new, i32(slots), i32(sg), None, None, None, None, ki, workspace=ws)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert not ki.any()


# ------------------------------------------------------------------ block scores and selection
@pytest.mark.parametrize("Hkv,di,lens,q,pad", [
    (2, 64, [1], [1], 0), (8, 128, [128, 129, 127, 1000, 1, 256], [1] * 6, 2), (4, 128, [500, 700, 40], [3, 17, 40], 5),
    (1, 64, [4000, 130], [100, 130], 0), (40, 128, [300, 260], [2, 1], 1), (5, 64, [777], [11], 0), (8, 64, [5000], [1], 0),
    (2, 64, [900, 700, 1], [300, 300, 1], 2)])
def test_block_scores(api, Hkv, di, lens, q, pad):
    import torch
    rng = np.random.default_rng(sum(lens) + Hkv)
    table, n_pages = lay_out(lens, rng, max_blocks=max((n + 127) // 128 for n in lens) + 3)
    starts, req, pos = rows_of(lens, q, pad)
    T, nb = len(req), table.shape[1]
    qt, qv = bf(rng.standard_normal((T, Hkv, di)))
    kx = rng.standard_normal((n_pages, PAGE, di))
    kt, kv = bf(kx)
    kt2 = kt.clone()
    seen = np.zeros((n_pages, PAGE), bool)
    for r, n in enumerate(lens):
        for j in range(n):
            seen[table[r, j // PAGE], j % PAGE] = True
    kt2[torch.from_numpy(~seen).cuda()] = float("nan")        # what no row may see
    sh = api.PagedShape(R=len(lens), T=T, max_blocks=nb, n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=64, d_idx=di, topk=4)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_SCORES)
    out = torch.full((T, Hkv, nb), 7.5, device="cuda")
    api.paged_block_scores(sh, qt, kt2, i32(table), i32(starts), i32(req), i32(pos), block_scores=out, workspace=ws)
    status_ok(api, ws)
    got = out.cpu().numpy()
    want, mag = ref.block_scores(qv, kv, table, req, pos, di ** -0.5)
    n = starts[-1]
    assert np.all(got[n:] == 7.5)
    fine = np.isfinite(want[:n])
    assert np.array_equal(fine, np.isfinite(got[:n])) and np.all(got[:n][~fine] == -np.inf)
    # d products in fp32, each step off by 2^-23 of the magnitudes at most; the scale's rounding and its product
    bound = di * 2.0 ** -23 * mag[:n] + 2.0 ** -23 * np.abs(want[:n])
    assert np.all(np.abs(got[:n] - want[:n])[fine] <= bound[fine])


def test_block_scores_pass_over_a_page_out_of_range(api):
    import torch
    rng = np.random.default_rng(2)
    table, n_pages = lay_out([600], rng)
    starts, req, pos = rows_of([600], [1], 0)
    sh = api.PagedShape(R=1, T=1, max_blocks=5, n_pages=n_pages, Hq=2, Hkv=2, d=64, d_idx=64, topk=4)
    (q, _), (k, _) = bf(rng.standard_normal((1, 2, 64))), bf(rng.standard_normal((n_pages, PAGE, 64)))
    want = api.paged_block_scores(sh, q, k, i32(table), i32(starts), i32(req), i32(pos)).cpu().numpy()
    for bad in (-1, n_pages, 2 ** 31 - 1):
        tb = table.copy()
        tb[0, 2] = bad
        ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_SCORES)
        got = api.paged_block_scores(sh, q, k, i32(tb), i32(starts), i32(req), i32(pos), workspace=ws).cpu().numpy()
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert np.all(got[:, :, 2] == -np.inf) and np.array_equal(np.delete(got, 2, 2), np.delete(want, 2, 2))
    # a row of a request that is none, and one past its table
    for rq, ps in ((1, 5), (0, 640)):
        ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_SCORES)
        api.paged_block_scores(sh, q, k, i32(table), i32(starts), i32([rq]), i32([ps]), workspace=ws)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)


@pytest.mark.parametrize("T,Hkv,nb,k", [(1, 1, 1, 1), (3, 2, 40, 16), (64, 8, 256, 16), (2, 2, 8192, 16), (5, 3, 1000, 32), (7, 2, 70, 1),
                                        (9, 1, 333, 2), (3000, 8, 33, 4), (1300, 8, 300, 17), (2, 2, 65, 32)])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_block_topk(api, T, Hkv, nb, k, kind):
    import torch
    rng = np.random.default_rng(T + nb + k)
    s = rng.standard_normal((T, Hkv, nb)).astype(np.float32)
    if kind == "ties":
        s = np.round(s * 2) / 2 * np.where(rng.random(s.shape) < 0.5, 1, -1)       # zeros of both signs too
    if kind == "special":
        s = np.where(rng.random(s.shape) < 0.5, rng.choice([np.nan, -np.inf, np.inf, 0.0, -0.0, 1e-45, -3.4e38], s.shape), s)
    s = s.astype(np.float32)
    pos = rng.integers(0, nb * PAGE, T).astype(np.int32)
    pos[0] = nb * PAGE - 1
    if T > 2:
        pos[-1] = -1
    sh = api.PagedShape(R=T, T=T, max_blocks=nb, n_pages=1, Hq=Hkv, Hkv=Hkv, d=64, d_idx=64, topk=k)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_TOPK)
    out = torch.full((T, Hkv, k), -5, dtype=torch.int32, device="cuda")
    api.paged_block_topk(sh, dev(s), i32(pos), sel_idx=out, workspace=ws)
    status_ok(api, ws)
    want = ref.topk(s, pos, k)
    want[pos < 0] = -5
    assert np.array_equal(out.cpu().numpy(), want)


def test_block_topk_leaves_out_rows_past_the_table(api):
    import torch
    sh = api.PagedShape(R=1, T=2, max_blocks=3, n_pages=1, Hq=1, Hkv=1, d=64, d_idx=64, topk=2)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_TOPK)
    out = torch.full((2, 1, 2), -5, dtype=torch.int32, device="cuda")
    api.paged_block_topk(sh, torch.zeros(2, 1, 3, device="cuda"), i32([3 * PAGE, 130]), sel_idx=out, workspace=ws)
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert out.flatten().tolist() == [-5, -5, 0, 1]


# ------------------------------------------------------------------ attention
def filled_cache(rng, n_pages, Hkv, d, table, lens, gain=1.0):
    """Codes and scales of a cache; every byte that no request owns is a NaN code, every such scale NaN."""
    x = rng.standard_normal((n_pages, Hkv, PAGE, d)) * gain
    s = (2.0 ** np.ceil(np.log2(np.abs(x).max((2, 3)) / 448)) * 2.0 ** rng.integers(0, 3, (n_pages, Hkv))).astype(np.float32)
    codes = ref.e4m3_encode(x / s[:, :, None, None])
    own = np.zeros((n_pages, PAGE), bool)
    for r, n in enumerate(lens):
        for j in range(n):
            own[table[r, j // PAGE], j % PAGE] = True
    codes[np.broadcast_to(~own[:, None, :, None], codes.shape)] = rng.choice([0x7F, 0xFF])
    s[~own.any(1)] = np.nan
    return codes, s


def pick(rng, pos, Hkv, k):
    sel = np.full((len(pos), Hkv, k), -1, np.int32)
    for t, p in enumerate(pos):
        c0 = p // PAGE
        for h in range(Hkv if p >= 0 else 0):
            m = min(k, c0 + 1)
            sel[t, h, :m] = np.sort(np.append(rng.choice(c0, m - 1, replace=False), c0)) if c0 else [0]
    return sel


def attn_case(api, lens, q, Hq, Hkv, d, k, sparse, pad=0, gain=1.0, scale=0.0, qgain=1.0, seed=0, max_blocks=None):
    rng = np.random.default_rng(sum(lens) + Hq + d + seed)
    table, n_pages = lay_out(lens, rng, max_blocks)
    starts, req, pos = rows_of(lens, q, pad)
    T = len(req)
    qt, qv = bf(rng.standard_normal((T, Hq, d)) * qgain)
    k8, ks = filled_cache(rng, n_pages, Hkv, d, table, lens, gain)
    v8, vs = filled_cache(rng, n_pages, Hkv, d, table, lens)
    sel = pick(rng, pos, Hkv, k) if sparse else None
    sh = api.PagedShape(R=len(lens), T=T, max_blocks=table.shape[1], n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=64, topk=k, scale=scale)
    args = (qt, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), i32(req), i32(pos))
    sc = float(np.float32(scale)) if scale else float(np.float32(1) / np.sqrt(np.float32(d)))
    return sh, args, sel, (qv, k8, v8, ks, vs, table, req, pos, sel, sc)


def check_attn(api, sh, args, sel, r, n):
    import torch
    ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
    ws[4096:].fill_(0xFF)
    o = torch.full((sh.T, sh.Hq, sh.d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sh.T, sh.Hq), 3.0, device="cuda")
    api.paged_attn(sh, *args, sel_idx=None if sel is None else i32(sel), o=o, lse=lse, workspace=ws)
    status_ok(api, ws)
    assert not ws[:4096].any()                                      # as the next call needs them
    ow, lw, do, dl = ref.attn(*r)
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(og[n:] == 3.0) and np.all(lg[n:] == 3.0)          # rows behind the last request
    none = np.isneginf(lw[:n])
    assert np.array_equal(none, np.isneginf(lg[:n])) and np.all(og[:n][none] == 0)
    fine = ~none
    assert np.all(np.abs(lg[:n] - lw[:n])[fine] <= dl[:n][fine]), np.max((np.abs(lg[:n] - lw[:n]) / dl[:n])[fine])
    assert np.all(np.abs(og[:n] - ow[:n]) <= do[:n] + 1e-30)
    return o, lse


CASES = [
    dict(lens=[1], q=[1], Hq=2, Hkv=2, d=64, k=4), dict(lens=[127, 128, 129, 31, 33, 2], q=[1] * 6, Hq=8, Hkv=1, d=128, k=4, pad=2),
    dict(lens=[1000, 5, 640, 2049], q=[1, 1, 1, 1], Hq=16, Hkv=4, d=128, k=8), dict(lens=[900, 300], q=[5, 130], Hq=8, Hkv=2, d=64, k=4, pad=3),
    dict(lens=[6000], q=[1], Hq=8, Hkv=8, d=128, k=16), dict(lens=[5000, 4097], q=[2, 1], Hq=8, Hkv=4, d=64, k=32),
    dict(lens=[300], q=[1], Hq=8, Hkv=1, d=64, k=1, max_blocks=50),
    dict(lens=[2100 + 37 * i for i in range(40)], q=[1] * 40, Hq=16, Hkv=8, d=64, k=16, max_blocks=40),       # rows of several CTAs, CTAs of several rows
    dict(lens=[400, 130, 5, 1300], q=[1, 2, 1, 1], Hq=16, Hkv=2, d=128, k=16),                            # fewer blocks than slots
    dict(lens=[38500], q=[1], Hq=8, Hkv=1, d=128, k=32),                                                 # a row in many pieces
    dict(lens=[21000, 40000], q=[1, 1], Hq=4, Hkv=1, d=64, k=32),
    dict(lens=[2 + 97 * i % 900 for i in range(120)], q=[1 + (i % 7 == 0) for i in range(120)], Hq=16, Hkv=4, d=64, k=8, pad=5),   # many short rows
    dict(lens=[400, 330], q=[300, 310], Hq=2, Hkv=1, d=64, k=2, pad=7),                                   # more rows than are cut
    dict(lens=[3000, 100, 7], q=[1, 1, 1], Hq=64, Hkv=8, d=128, k=16, max_blocks=200)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("sparse", [True, False])
def test_attention(api, case, sparse):
    c = CASES[case]
    sh, args, sel, r = attn_case(api, sparse=sparse, **c)
    check_attn(api, sh, args, sel, r, sum(c["q"]))


@pytest.mark.parametrize("kw", [dict(gain=30.0), dict(gain=1e-3), dict(scale=0.7), dict(qgain=1e-6), dict(qgain=100.0), dict(gain=2.0 ** 60, qgain=2.0 ** -62)])
def test_attention_of_other_magnitudes(api, kw):
    sh, args, sel, r = attn_case(api, lens=[700, 260], q=[1, 2], Hq=8, Hkv=2, d=128, k=3, sparse=True, **kw)
    check_attn(api, sh, args, sel, r, 3)


def test_attention_rows_without_blocks_and_gaps_in_the_selection(api):
    sh, args, sel, r = attn_case(api, lens=[1500, 700], q=[3, 2], Hq=8, Hkv=2, d=64, k=8, sparse=True)
    sel[0, 0] = -1                                   # no block at all
    sel[1, 1] = [-1, 3, -1, -1, 5, 7, -1, 8]         # gaps, and not the row's own block
    sel[4, :] = -1
    r = r[:8] + (sel,) + r[9:]
    check_attn(api, sh, args, sel, r, 5)


def test_attention_leaves_out_bad_entries(api):
    """Selections that do not ascend, lie past the row's block, or name no page: left out and recorded."""
    import torch
    sh, args, sel, r = attn_case(api, lens=[1500], q=[1], Hq=4, Hkv=1, d=64, k=4, sparse=True)
    run = lambda s, a=args, **kw: api.paged_attn(sh, *a, sel_idx=i32(np.array(s).reshape(1, 1, 4)), **kw)
    for bad, same in (([2, 2, 5, 11], [2, -1, 5, 11]), ([5, 2, 7, 11], [5, -1, 7, 11]), ([2, 7, 11, 12], [2, 7, 11, -1]),
                      ([2, 7, 11, 2 ** 31 - 1], [2, 7, 11, -1])):
        ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
        got, want = run(bad, workspace=ws), run(same)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    short, a2, _, _ = attn_case(api, lens=[200], q=[1], Hq=4, Hkv=1, d=64, k=4, sparse=True)      # two blocks: two slots
    ws = api.new_paged_workspace(short, api.OP_PAGED_ATTN)
    got, want = (api.paged_attn(short, *a2, sel_idx=i32(np.array(s).reshape(1, 1, 4)), workspace=w) for s, w in (([-1, 0, 1, -1], ws), ([-1, 0, -1, -1], None)))
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for page in (-1, sh.n_pages, 2 ** 31 - 1):
        table = args[5].clone()
        table[0, 7] = page
        ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
        got, want = run([2, 7, 8, 11], args[:5] + (table,) + args[6:], workspace=ws), run([2, -1, 8, 11])
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for req, pos in ((1, 5), (0, 12 * PAGE)):
        ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
        o = torch.full((1, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        api.paged_attn(sh, *args[:6], i32([req]), i32([pos]), o=o, workspace=ws)
        with pytest.raises(api.MsaError):
            api.check_device_status(ws)
        assert (o == 3.0).all()


def test_attention_nan_reaches_only_its_rows(api):
    """A NaN query head spoils itself; a NaN code in a visible token its group's rows that see it; one behind the row's
    position nothing (filled_cache puts them everywhere there)."""
    import torch
    sh, args, sel, r = attn_case(api, lens=[400, 300], q=[2, 1], Hq=8, Hkv=2, d=64, k=4, sparse=False)
    o0, l0 = api.paged_attn(sh, *args)
    qt = args[0].clone()
    qt[0, 3, 5] = float("inf")
    o, l = api.paged_attn(sh, qt, *args[1:])
    hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
    hit[0, 3] = True
    assert torch.equal(torch.isnan(l), hit) and torch.equal(torch.isnan(o).any(2), hit)
    assert torch.equal(o[~hit], o0[~hit])
    for which in (1, 2):
        a = list(args)
        a[which] = a[which].clone()
        page = int(a[5][0, 399 // PAGE])
        a[which].view(torch.uint8)[page, 1, 399 % PAGE] = 0x7F          # token 399: only the second row of request 0 sees it
        o, l = api.paged_attn(sh, *a)
        hit = torch.zeros(3, 8, dtype=torch.bool, device="cuda")
        hit[1, 4:] = True
        assert torch.equal(torch.isnan(o).all(2), hit) and torch.equal(o[~hit], o0[~hit]) and torch.equal(torch.isnan(l), hit if which == 1 else hit & False)


def test_attention_is_the_same_on_every_run_and_stream(api):
    import torch
    sh, args, sel, r = attn_case(api, lens=[5000, 2000, 90], q=[1, 3, 1], Hq=16, Hkv=2, d=128, k=16, sparse=True)
    s = i32(sel)
    want = api.paged_attn(sh, *args, sel_idx=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = api.paged_attn(sh, *args, sel_idx=s, stream=side)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ together
class Server:
    """The calls of a serving loop, beside a plain record of every request's tokens."""

    def __init__(self, api, R, nb, n_pages, Hq, Hkv, d, di, k, T, seed):
        import torch
        self.api, self.rng = api, np.random.default_rng(seed)
        self.sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=di, topk=k)
        self.table = torch.full((R, nb), -1, dtype=torch.int32, device="cuda")
        self.ring = i32(self.rng.permutation(n_pages))
        self.free, self.lens = i32([3, n_pages]), i32([0] * R)
        z = lambda *n, dtype: torch.zeros(n, dtype=torch.uint8, device="cuda").view(dtype) if dtype is torch.float8_e4m3fn else torch.zeros(n, dtype=dtype, device="cuda")
        self.k8, self.v8 = (z(n_pages, Hkv, PAGE, d, dtype=torch.float8_e4m3fn) for _ in "kv")
        self.ks, self.vs = (z(n_pages, Hkv, dtype=torch.float32) for _ in "kv")
        self.ki = z(n_pages, PAGE, di, dtype=torch.bfloat16)
        self.toks = [np.zeros((0, di)) for _ in range(R)]
        self.ws = {op: api.new_paged_workspace(self.sh, op) for op in range(16, 21)}

    def step(self, new, ended, x):
        """One step; x: the rows' k, v, k_idx, q, q_idx."""
        a, s, w = self.api, self.sh, self.ws
        plan = a.paged_plan(s, new, self.lens, self.table, self.ring, self.free, ended=ended, workspace=w[16])
        self.lens, self.free = plan.lens, plan.free_state
        a.paged_append(s, x["k"], x["v"], x["ki"], plan.slots, plan.segs, self.k8, self.v8, self.ks, self.vs, self.ki, workspace=w[17])
        bs = a.paged_block_scores(s, x["qi"], self.ki, self.table, plan.q_starts, plan.row_req, plan.row_pos, workspace=w[18])
        sel = a.paged_block_topk(s, bs, plan.row_pos, workspace=w[19])
        o, lse = a.paged_attn(s, x["q"], self.k8, self.v8, self.ks, self.vs, self.table, plan.row_req, plan.row_pos, sel_idx=sel, workspace=w[20])
        return plan, bs, sel, o, lse

    def rows(self):
        s, r = self.sh, self.rng
        return {n: bf(r.standard_normal(shp)) for n, shp in (("k", (s.T, s.Hkv, s.d)), ("v", (s.T, s.Hkv, s.d)), ("ki", (s.T, s.d_idx)),
                                                           ("q", (s.T, s.Hq, s.d)), ("qi", (s.T, s.Hkv, s.d_idx)))}


def test_serving_loop(api):
    """Prompts, decoding, slots that end and start anew, all through the five
    calls; every step is checked: lengths, scores against the tokens as they
    were given, the selection against the scores, attention against the cache."""
    import torch
    sv = Server(api, R=4, nb=9, n_pages=40, Hq=8, Hkv=2, d=64, di=64, k=3, T=600, seed=5)
    steps = [([300, 0, 128, 1], None), ([1, 200, 1, 1], None), ([1, 1, 1, 0], None), ([130, 1, 0, 1], [0, 0, 1, 0]), ([1, 1, 250, 1], [0, 1, 0, 0]), ([2, 3, 2, 400], None)]
    lens = np.zeros(4, int)
    for new, ended in steps:
        x = sv.rows()
        plan, bs, sel, o, lse = sv.step(i32(new), None if ended is None else i32(ended), {n: v[0] for n, v in x.items()})
        for ws in sv.ws.values():
            status_ok(api, ws)
        req, pos, st = (t.cpu().numpy() for t in (plan.row_req, plan.row_pos, plan.q_starts))
        for r in range(4):
            if ended and ended[r]:
                sv.toks[r] = sv.toks[r][:0]
            sv.toks[r] = np.concatenate([sv.toks[r], x["ki"][1][st[r]:st[r + 1]]])
        assert plan.lens.tolist() == [len(t) for t in sv.toks]
        n, table = st[-1], sv.table.cpu().numpy()
        got = bs.cpu().numpy()
        for t in range(0, n, 7):
            c0 = pos[t] // PAGE
            s = x["qi"][1][t] @ sv.toks[req[t]][:pos[t] + 1].T / 8
            want = np.stack([s[:, c * PAGE:(c + 1) * PAGE].max(1) for c in range(c0 + 1)], 1)
            assert np.allclose(got[t, :, :c0 + 1], want, rtol=0, atol=64 * 2.0 ** -23 * 64) and np.all(got[t, :, c0 + 1:] == -np.inf)
        sel_n = sel.cpu().numpy()
        assert np.array_equal(sel_n[:n], ref.topk(got, pos, 3)[:n])
        ow, lw, do, dl = ref.attn(x["q"][1], *(c.view(torch.uint8).cpu().numpy() for c in (sv.k8, sv.v8)), sv.ks.cpu().numpy(), sv.vs.cpu().numpy(),
                                  table, req, pos, sel_n, 0.125)
        assert np.all(np.abs(o.double().cpu().numpy()[:n] - ow[:n]) <= do[:n])
        assert np.all(np.abs(lse.double().cpu().numpy()[:n] - lw[:n]) <= dl[:n])


def test_decode_agrees_with_the_contiguous_calls(api):
    """A uniform batch: the paged scores and selection against msa_index_select
    on the same keys laid out contiguously, and attention with every block
    selected against the form without a selection."""
    import torch
    rng = np.random.default_rng(8)
    R, Hq, Hkv, d, k, n = 3, 16, 4, 128, 16, 30 * PAGE + 77
    table, n_pages = lay_out([n] * R, rng)
    starts, req, pos = rows_of([n] * R, [1] * R, 0)
    ki, _ = bf(rng.standard_normal((n_pages, PAGE, d)))
    qi, _ = bf(rng.standard_normal((R, Hkv, d)))
    flat = ki[i32(table).long()].reshape(R, -1, d).contiguous()
    old = api.Shape(B=R, Nq=1, Nk=n, Hq=Hq, Hkv=Hkv, d=d, d_idx=d, topk=k, q_offset=n - 1, kv_rows=flat.shape[1])
    sel0, bs0 = api.index_select(old, qi[:, None].contiguous(), flat, return_scores=True)
    sh = api.PagedShape(R=R, T=R, max_blocks=table.shape[1], n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=d, topk=k)
    bs = api.paged_block_scores(sh, qi, ki, i32(table), i32(starts), i32(req), i32(pos))
    assert torch.allclose(bs, bs0[:, 0], rtol=0, atol=1e-4)
    assert torch.equal(api.paged_block_topk(sh, bs0[:, 0].contiguous(), i32(pos)), sel0[:, :, 0])
    k8, ks = filled_cache(rng, n_pages, Hkv, d, table, [n] * R)
    v8, vs = filled_cache(rng, n_pages, Hkv, d, table, [n] * R)
    q, _ = bf(rng.standard_normal((R, Hq, d)))
    args = (q, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), i32(req), i32(pos))
    full = api.PagedShape(R=R, T=R, max_blocks=table.shape[1], n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=d, topk=31)
    every = i32(np.broadcast_to(np.arange(31), (R, Hkv, 31)))
    a, b = api.paged_attn(full, *args, sel_idx=every), api.paged_attn(full, *args)
    assert torch.allclose(a[1], b[1], rtol=0, atol=2.0 ** -16 * 16) and torch.allclose(a[0].float(), b[0].float(), rtol=2.0 ** -7, atol=2.0 ** -9)


def test_decode_loop_in_a_captured_graph(api):
    """The five calls captured once and replayed, lengths and ring updated in
    place, against the same steps run eagerly on another state."""
    import torch
    mk = lambda: Server(api, R=3, nb=6, n_pages=18, Hq=8, Hkv=2, d=128, di=128, k=2, T=3, seed=9)
    eager, graph = mk(), mk()
    one = i32([1, 1, 1])
    stat = {n: v[0].clone() for n, v in graph.rows().items()}
    eager.rows()

    def body():
        a, s, w = api, graph.sh, graph.ws
        z = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
        out = api.PagedPlan(graph.lens, graph.free, z(4), z(3), z(3), z(3), z(s.n_segs + 1))
        p = a.paged_plan(s, one, graph.lens, graph.table, graph.ring, graph.free, workspace=w[16], out=out)
        a.paged_append(s, stat["k"], stat["v"], stat["ki"], p.slots, p.segs, graph.k8, graph.v8, graph.ks, graph.vs, graph.ki, workspace=w[17])
        bs = a.paged_block_scores(s, stat["qi"], graph.ki, graph.table, p.q_starts, p.row_req, p.row_pos, workspace=w[18])
        sel = a.paged_block_topk(s, bs, p.row_pos, workspace=w[19])
        return a.paged_attn(s, stat["q"], graph.k8, graph.v8, graph.ks, graph.vs, graph.table, p.row_req, p.row_pos, sel_idx=sel, workspace=w[20])

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = body()
    for step in range(300):                            # over two page borders
        x = {n: v[0] for n, v in eager.rows().items()}
        for n in stat:
            stat[n].copy_(x[n])
        g.replay()
        if step in (0, 1, 126, 127, 128, 255, 256, 299):
            torch.cuda.synchronize()
        ow, lw = eager.step(one, None, x)[3:]
        assert torch.equal(o, ow) and torch.equal(lse, lw), step
    assert graph.lens.tolist() == [300] * 3 and torch.equal(graph.free, eager.free)
    for ws in graph.ws.values():
        status_ok(api, ws)


def test_cache_offsets_past_32_bits(api):
    """Pages whose K and V lie more than 4 GB into their pools."""
    import torch
    Hkv, d, n_pages = 8, 128, 36000                    # 36,000 pages x 131,072 bytes: 4.7 GB each
    sh = api.PagedShape(R=2, T=2, max_blocks=2, n_pages=n_pages, Hq=16, Hkv=Hkv, d=d, d_idx=128, topk=2)
    small = api.PagedShape(R=2, T=2, max_blocks=2, n_pages=4, Hq=16, Hkv=Hkv, d=d, d_idx=128, topk=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *n: torch.randn(*n, device="cuda", generator=g).bfloat16()
    pages = [n_pages - 1, 33000, n_pages - 2, 5]
    res = []
    x = {n: rnd(2, *m) for n, m in (("k", (Hkv, d)), ("v", (Hkv, d)), ("ki", (128,)), ("q", (16, d)), ("qi", (Hkv, 128)))}
    code = torch.randint(0, 0x7E, (2, 4, Hkv, PAGE, d), dtype=torch.uint8, device="cuda", generator=g)
    ki0 = rnd(4, PAGE, 128)
    for s, ids in ((sh, pages), (small, [0, 1, 2, 3])):
        k8, v8 = (torch.zeros(s.n_pages, Hkv, PAGE, d, dtype=torch.uint8, device="cuda") for _ in "kv")
        ki = torch.zeros(s.n_pages, PAGE, 128, dtype=torch.bfloat16, device="cuda")
        at = torch.tensor(ids, device="cuda")
        k8[at], v8[at], ki[at] = code[0], code[1], ki0
        ks, vs = (torch.full((s.n_pages, Hkv), 2.0 ** -8, device="cuda") for _ in "kv")
        table = i32(np.array(ids).reshape(2, 2))
        slots = i32([ids[1] * PAGE + 71, ids[3] * PAGE + 3])
        f = torch.float8_e4m3fn
        api.paged_append(s, x["k"], x["v"], x["ki"], slots, i32([0, 1, 2]), k8.view(f), v8.view(f), ks, vs, ki)
        rr, rp = i32([0, 1]), i32([PAGE + 71, PAGE + 3])
        bs = api.paged_block_scores(s, x["qi"], ki, table, i32([0, 1, 2]), rr, rp)
        o, lse = api.paged_attn(s, x["q"], k8.view(f), v8.view(f), ks, vs, table, rr, rp)
        res.append((k8[at], v8[at], ki[at], ks[at], bs, o, lse))
    for a, b in zip(*res):
        assert torch.equal(a.view(torch.uint8) if a.dtype is torch.float8_e4m3fn else a, b)


def test_steps_without_rows(api):
    """Every request idle, or no row that belongs to one: nothing is written and nothing recorded."""
    import torch
    sv = Server(api, R=3, nb=4, n_pages=8, Hq=8, Hkv=2, d=64, di=64, k=2, T=5, seed=1)
    x = sv.rows()
    for new in ([0, 0, 0], [2, 0, 3], [0, 0, 0]):
        before = [t.clone() for t in (sv.table, sv.ring, sv.ks, sv.ki)]
        plan, bs, sel, o, lse = sv.step(i32(new), None, {n: v[0] for n, v in x.items()})
        for ws in sv.ws.values():
            status_ok(api, ws)
        if sum(new) == 0:
            assert not plan.q_starts.any() and (plan.row_req == -1).all()
            assert all(torch.equal(a, b) for a, b in zip(before, (sv.table, sv.ring, sv.ks, sv.ki)))
    assert sv.lens.tolist() == [2, 0, 3] and sv.free.tolist()[1] == 6


def test_two_streams_at_once(api):
    """Two callers on two streams, each with its own workspace and outputs, over the same cache."""
    import torch
    cases = [attn_case(api, lens=[3000 + 50 * i for i in range(20)], q=[1] * 20, Hq=16, Hkv=2, d=128, k=16, sparse=True, seed=s) for s in (0, 1)]
    want = [api.paged_attn(sh, *args, sel_idx=i32(sel)) for sh, args, sel, r in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [api.new_paged_workspace(c[0], api.OP_PAGED_ATTN) for c in cases]
    sels = [i32(c[2]) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [api.paged_attn(c[0], *c[1], sel_idx=s, workspace=w, stream=st) for c, s, w, st in zip(cases, sels, spaces, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_one_workspace_for_every_call(api):
    """The five calls in turn on one workspace, rows cut between CTAs: as on workspaces of their own."""
    import torch
    sizes = dict(R=3, nb=20, n_pages=60, Hq=16, Hkv=2, d=128, di=64, k=16, T=64, seed=3)
    own, one = Server(api, **sizes), Server(api, **sizes)
    most = max(w.numel() for w in one.ws.values())
    space = torch.zeros(most, dtype=torch.uint8, device="cuda")
    one.ws = {op: space for op in one.ws}
    x = own.rows()
    for new in [[30, 0, 34], [1, 60, 1]] * 12:
        a, b = (s.step(i32(new), None, {n: v[0] for n, v in x.items()}) for s in (own, one))
        status_ok(api, space)
        n = sum(new)
        assert torch.equal(a[3][:n], b[3][:n]) and torch.equal(a[4][:n], b[4][:n]) and torch.equal(a[2][:n], b[2][:n])


def test_workspace_shared_by_graphs_replayed_in_turn(api):
    """Two graphs over one workspace, one after the other on a stream, as the workspace rule allows."""
    import torch
    (sh, args, sel, _), (sh2, args2, _, _) = (attn_case(api, lens=[2500, 900, 4000], q=[1, 1, 1], Hq=16, Hkv=2, d=128, k=16, sparse=sp, seed=7) for sp in (True, False))
    sel = i32(sel)
    want, want2 = api.paged_attn(sh, *args, sel_idx=sel), api.paged_attn(sh2, *args2)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
    graphs, outs = [], []
    for call in (lambda: api.paged_attn(sh, *args, sel_idx=sel, workspace=ws), lambda: api.paged_attn(sh2, *args2, workspace=ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for i in range(30):
        graphs[i % 2].replay()
        graphs[(i + i // 3) % 2].replay()
    torch.cuda.synchronize()
    for got, w in zip(outs, (want, want2)):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    status_ok(api, ws)


def test_outputs_on_a_given_stream_are_not_reused_early(api):
    """Outputs and workspaces that a call allocates belong to the stream it runs on: calls on a side stream, their results
    dropped and memory asked for again on the current stream meanwhile."""
    import torch
    sh, args, sel, _ = attn_case(api, lens=[5000] * 16, q=[1] * 16, Hq=16, Hkv=2, d=128, k=16, sparse=True)
    sel = i32(sel)
    want = api.paged_attn(sh, *args, sel_idx=sel)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        o, lse = api.paged_attn(sh, *args, sel_idx=sel, stream=side)       # its own workspace, freed on return
        junk = [torch.full((1 << 18,), 7, dtype=torch.int32, device="cuda") for _ in range(8)]
        side.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        del o, lse, junk


@pytest.mark.parametrize("Hkv,di,lens,q", [(8, 128, [500, 700, 40, 2000], [3, 17, 40, 16]), (1, 64, [4000, 130], [100, 130]), (40, 128, [300, 1260], [2, 5]),
                                           (2, 64, [900, 700], [300, 300]), (8, 128, [5000], [4])])
@pytest.mark.parametrize("order", ["down", "shuffled", "equal"])
def test_positions_of_a_request_in_any_order(api, Hkv, di, lens, q, order):
    """Rows whose positions do not ascend (branches of a draft, say): each row's scores and attention are its own."""
    import torch
    rng = np.random.default_rng(sum(lens) + Hkv)
    table, n_pages = lay_out(lens, rng, max_blocks=max((n + 127) // 128 for n in lens) + 2)
    starts, req, pos = rows_of(lens, q, 2)
    for r in range(len(q)):
        at = slice(starts[r], starts[r + 1])
        pos[at] = {"down": pos[at][::-1], "shuffled": rng.integers(0, lens[r], q[r]), "equal": np.where(rng.random(q[r]) < 0.5, lens[r] // 2, lens[r] - 1)}[order]
    T, nb, n = len(req), table.shape[1], starts[-1]
    qt, qv = bf(rng.standard_normal((T, Hkv, di)))
    kt, kv = bf(rng.standard_normal((n_pages, PAGE, di)))
    sh = api.PagedShape(R=len(lens), T=T, max_blocks=nb, n_pages=n_pages, Hq=Hkv, Hkv=Hkv, d=64, d_idx=di, topk=3)
    ws = api.new_paged_workspace(sh, api.OP_PAGED_BLOCK_SCORES)
    got = api.paged_block_scores(sh, qt, kt, i32(table), i32(starts), i32(req), i32(pos), workspace=ws)
    status_ok(api, ws)
    sel = api.paged_block_topk(sh, got, i32(pos)).cpu().numpy()
    got = got.cpu().numpy()
    want, mag = ref.block_scores(qv, kv, table, req, pos, di ** -0.5)
    fine = np.isfinite(want[:n])
    assert np.array_equal(fine, np.isfinite(got[:n])) and np.all(got[:n][~fine] == -np.inf)
    assert np.all(np.abs(got[:n][fine] - want[:n][fine]) <= di * 2.0 ** -23 * mag[:n][fine] + 2.0 ** -23 * np.abs(want[:n][fine]))
    assert np.array_equal(sel[:n], ref.topk(got, pos, 3)[:n])
    k8, ks = filled_cache(rng, n_pages, Hkv, 64, table, lens)
    v8, vs = filled_cache(rng, n_pages, Hkv, 64, table, lens)
    q8, qv = bf(rng.standard_normal((T, Hkv, 64)))
    args = (q8, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), i32(req), i32(pos))
    check_attn(api, sh, args, sel, (qv, k8, v8, ks, vs, table, req, pos, sel, 0.125), n)


def test_attention_beside_kernels_that_take_all_of_tensor_memory(api):
    """Chained attention calls on one stream, the contiguous selection (512 columns a CTA) on another, at sizes that share
    an SM: both come out as alone."""
    import torch
    sh, args, sel, _ = attn_case(api, lens=[3000 + 50 * i for i in range(20)], q=[1] * 20, Hq=16, Hkv=2, d=64, k=16, sparse=True)
    sel, ws = i32(sel), api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
    full = api.Shape(B=1, Nq=2048, Nk=2048, Hq=8, Hkv=2, d=64, d_idx=64, topk=4)
    g = torch.Generator(device="cuda").manual_seed(4)
    qi, ki = (torch.randn(1, 2048, *m, 64, device="cuda", generator=g).bfloat16() for m in ((2,), ()))
    want, want2 = api.paged_attn(sh, *args, sel_idx=sel, workspace=ws), api.index_select(full, qi, ki)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [api.paged_attn(sh, *args, sel_idx=sel, workspace=ws, stream=streams[0]) for _ in range(6)]
        with torch.cuda.stream(streams[1]):
            got2 = [api.index_select(full, qi, ki) for _ in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(a[0], want[0]) and torch.equal(a[1], want[1]) for a in got)
        assert all(torch.equal(a, want2) for a in got2)
    status_ok(api, ws)
