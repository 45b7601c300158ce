"""Chunk attention over pages whose V scales are far apart: zero, tiny and
large values, under logits that rise behind a row's first page."""
import numpy as np
import pytest

import chunk_ref
import paged_ref as ref
from test_gpu_chunks import check_chunk, starts_of
from test_gpu_paged import bf, dev, f8, i32, lay_out, pick, rows_of

pytestmark = pytest.mark.gpu

PAGE = 128


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def rising_case(api, gains, lens, q, Hq, Hkv, d, k, sparse, up):
    """Values of gains[b % len] in block b (0: zeros, whose scale an append makes 2^-112); one key of each block but the first
    lies along the queries, further in later blocks, up to `up` in the last: a logit of 3.5 up sqrt(d)."""
    rng = np.random.default_rng(sum(lens) + d + len(gains))
    table, n_pages = lay_out(lens, rng)
    starts, req, pos = rows_of(lens, q, 0)
    qt, qv = bf(rng.uniform(0.9, 1.1, (len(req), Hq, d)) * up)
    k8, v8 = (np.full((n_pages, Hkv, PAGE, d), 0x7F, np.uint8) for _ in range(2))      # tokens that nobody wrote are NaN
    ks, vs = np.full((n_pages, Hkv), 2.0 ** -7, np.float32), np.ones((n_pages, Hkv), np.float32)
    for r, m in enumerate(lens):
        nb = -(-m // PAGE)
        for b in range(nb):
            n, page = min(PAGE, m - b * PAGE), table[r, b]
            x = np.clip(rng.standard_normal((Hkv, n, d)) * 0.5, -3.5, 3.5)
            if b:
                x[:, min(n - 1, 5)] = 3.5 * (b + 1) / nb
            k8[page, :, :n] = ref.e4m3_encode(x * 2.0 ** 7)
            v = rng.standard_normal((Hkv, n, d)) * gains[b % len(gains)]
            for h in range(Hkv):
                vs[page, h] = s = ref.scale_of(v[h])
                v8[page, h, :n] = ref.e4m3_encode(v[h] / s)
    sel = pick(rng, pos, Hkv, k) if sparse else None
    sh = api.PagedShape(R=len(lens), T=len(req), max_blocks=table.shape[1], n_pages=n_pages, Hq=Hq, Hkv=Hkv, d=d, d_idx=64, topk=k)
    args = (qt, f8(k8), f8(v8), dev(ks), dev(vs), i32(table), i32(req), i32(pos))
    return sh, args, sel, (qv, k8, v8, ks, vs, table, req, pos, sel, float(np.float32(1) / np.sqrt(np.float32(d))))


GAINS = {"zero": [0.0], "tiny": [2.0 ** -60], "least": [2.0 ** -100], "zero first": [0.0, 1.0, 1.0], "zero between": [1.0, 0.0, 0.0],
         "tiny first": [2.0 ** -60, 1.0], "tiny between": [1.0, 2.0 ** -60], "zero, large": [0.0, 2.0 ** 60, 1.0],
         "large first": [2.0 ** 60, 1.0, 2.0 ** -60], "large between": [1.0, 2.0 ** 100, 0.0], "largest": [2.0 ** 120], "beyond": [2.0 ** 125.5]}


@pytest.mark.parametrize("kind", GAINS)
@pytest.mark.parametrize("shape", ["whole", "cut", "halves in turn"])
@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_values_of_any_size_under_rising_logits(api, kind, shape, sparse):
    """A logit up to 55 above the first page's (d = 128), 39 (d = 64).  A weight that falls out of fp32 is 2^-28 of the row's
    largest at most, less than the sum's own rounding of 2^-23 a token; a P that falls out of bf16 2^-52 of the largest."""
    c = {"whole": dict(lens=[600 + i for i in range(90)], q=[40] * 90, Hq=8, Hkv=1, d=128, k=3, up=1.4),
         "cut": dict(lens=[3000, 1500], q=[70, 33], Hq=8, Hkv=2, d=64, k=9, up=1.4),
         "halves in turn": dict(lens=[900, 1300, 130, 700], q=[5, 9, 1, 3], Hq=4, Hkv=2, d=128, k=4, up=1.0)}[shape]
    sh, args, sel, r = rising_case(api, GAINS[kind], sparse=sparse, **c)
    check_chunk(api, sh, args, starts_of(c["q"]), sel, r, sum(c["q"]))


@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_sums_over_zero_values_stay_finite(api, sparse):
    """Two pages of a head whose values are zero, a key along the queries in the second one: the logsumexp is what its logit says."""
    sh, args, sel, r = rising_case(api, [0.0], lens=[256, 250], q=[20, 100], Hq=8, Hkv=1, d=128, k=2, sparse=sparse, up=1.0)
    o, lse = api.paged_chunk_attn(sh, *args[:6], i32([0, 20, 120]), args[7], sel_idx=None if sel is None else i32(sel))
    want = chunk_ref.attn(*r)
    assert not o.any() and np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= want[3]) and lse.max() > 39.0


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("c", [dict(lens=[2100], q=[300], Hq=8, Hkv=1, d=128, k=6), dict(lens=[900, 130, 1500], q=[5, 130, 70], Hq=4, Hkv=2, d=64, k=4),
                               dict(lens=[300 + i for i in range(60)], q=[9] * 60, Hq=8, Hkv=2, d=64, k=2), dict(lens=[30000], q=[20], Hq=8, Hkv=1, d=64, k=32)])
@pytest.mark.parametrize("sparse", [True, False])
def test_chunk_no_token_is_missing(api, flat, c, sparse):
    """Each token's value is a single feature's, so that a feature is the weight of a few tokens and its bound theirs: one of a
    thousand that went missing, or was taken twice, shows (flat: equal weights, from queries of zero)."""
    from test_gpu_paged import attn_case
    sh, args, sel, r = attn_case(api, sparse=sparse, qgain=0.0 if flat else 1.0, **c)
    v8 = np.zeros_like(r[2])
    j = np.arange(PAGE)
    for page in range(sh.n_pages):
        v8[page, :, j, (j * 5 + page * 3) % sh.d] = 0x38            # 1
    v8[r[2] % 128 == 0x7F] = 0x7F                                   # tokens that nobody wrote
    vs = np.where(np.isnan(r[4]), r[4], np.float32(0.25))
    check_chunk(api, sh, args[:2] + (f8(v8), args[3], dev(vs)) + args[5:], starts_of(c["q"]), sel, r[:2] + (v8, r[3], vs) + r[5:], sum(c["q"]))
