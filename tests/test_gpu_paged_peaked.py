"""Attention over the 8-bit cache where one token outweighs thousands of others that together still count: an attention
sink above a long tail, the sink's value small or not, pages of very different V scales, rows cut between CTAs and whole.

The bound follows the kernel's arithmetic, token by token, without a term that grows with their number.  With p the
softmax's weights and V the cache's values:
  scores  fp32 sums of d products, each step off by at most 2^-23 of the magnitudes, and the query's two-term split, off
          by 2^-23 of the row's largest scaled feature:  ds <= d 2^-23 sum|q k| scale + 2^-22 max|q| sum|k| scale
  exp     p relative 2 ds (its own and the sum's) + 2^-20 (exp2, and the factors of the running maximum)
  split   p relative 2^-8, half a step of 8 significant bits, down to 2^-42 of the largest weight p vs; below,
          2^-50 of that weight on a code of at most 448.  (The reference is at most the largest weight; x = 32 p vs /
          reference is held in two e4m3 terms hi + lo / 32 at one of three scales 2^15 apart: 8 bits down to 2^-7 at the
          first, to 2^-37 at the last, whose least step is 2^-9 / 32 / 2^30 = 2^-44, half of it 2^-50 of the reference.)
  sums    fp32, 32 tokens at a time: each of the n / 32 steps off by at most 2^-23 of the sum
  o       rounded once to bf16, 2^-8 relative."""
import numpy as np
import pytest

import paged_ref as ref
from test_gpu_paged import PAGE, bf, dev, f8, i32, lay_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


def expected(q, K, V, sv, scale):
    """o, lse and the bounds of their errors: q [Hq, d] over K, V [n, d], all heads of one group; sv [n] the V scales."""
    s = K @ q.T * scale                                          # [n, Hq]
    ds = (np.abs(K) @ np.abs(q).T * (K.shape[1] * 2.0 ** -23) + np.abs(K).sum(1)[:, None] * np.abs(q).max(1) * 2.0 ** -22) * scale
    m = s.max(0)
    e = np.exp(s - m)
    z = e.sum(0)
    p = e / z
    o, mag = p.T @ V, p.T @ np.abs(V)
    dz = (p * ds).sum(0)                                         # the sum's relative error
    steps = len(K) / 32 * 2.0 ** -23
    rel = dz[:, None] + 2.0 ** -20 + 2.0 ** -8 + 2 * steps
    do = (p * ds).T @ np.abs(V) + rel * mag + (2.0 ** -50 * 448 * len(K) * (p * sv[:, None]).max(0))[:, None] + 2.0 ** -8 * np.abs(o)
    lse = m + np.log(z)
    return o, lse, do, dz + steps + 2.0 ** -21 * (1 + np.abs(lse) + np.abs(m))


def peaked(n, d, G, rest, value, seed=0, least=9, most=16):
    """One request of n tokens, token 0 above the rest by 9 to 16 nats (another gap for each head).
    rest: the other tokens' logits all equal, or N(0, 1).  value: of the cache, every value one ("ones"), the sink's zero
    and the others' 0.5 + N(0, 1) / 2 ("sink"), the same with the scale of the sink's page and of one in the tail 2^12
    times the others', their other values at feature 0 alone ("scales"), or N(0, 1) ("normal")."""
    rng = np.random.default_rng(n + d + G + seed)
    table, n_pages = lay_out([n], rng)
    gaps = least + (most - least) * np.arange(G) / max(1, G - 1)
    half = d // 2
    q = np.zeros((G, d))
    q[:, :half] = (gaps * np.sqrt(d) / half)[:, None]
    q[:, half:] = 1.0
    K = np.zeros((table.shape[1] * PAGE, d))
    if rest == "normal":
        K[:, half:] = rng.standard_normal((len(K), half)) * np.sqrt(d / half)
    K[0] = 0
    K[0, :half] = 1.0
    V = {"ones": lambda s: np.ones(s), "normal": rng.standard_normal}.get(value, lambda s: 0.5 + rng.standard_normal(s) / 2)((len(K), d))
    vs = np.full(table.shape[1], 2.0 ** -6)
    if value in ("sink", "scales"):
        V[0] = 0
    if value == "scales":
        for c in {0, table.shape[1] // 2}:
            V[c * PAGE:(c + 1) * PAGE, 1:] = 0
            vs[c] *= 2.0 ** 12
            V[c * PAGE + 1:(c + 1) * PAGE, 0] = 0.25 * vs[c]
    ks = np.full(table.shape[1], 2.0 ** -5)
    pages = table[0]
    out = []
    for x, sc in ((K, ks), (V, vs)):
        codes = np.full((n_pages, 1, PAGE, d), 0x7F, np.uint8)
        scales = np.full((n_pages, 1), np.nan, np.float32)
        c = ref.e4m3_encode(np.clip(x.reshape(-1, PAGE, d) / sc[:, None, None], -448, 448))
        c.reshape(-1, d)[n:] = 0x7F                             # behind the request: NaN
        codes[pages, 0], scales[pages, 0] = c, sc
        out += [codes, scales]
    return q, out, table, n_pages


def run(api, q, cache, table, n_pages, n, G, d, R=1, sel=None, k=16):
    k8, ks, v8, vs = cache
    sh = api.PagedShape(R=R, T=R, max_blocks=table.shape[1], n_pages=n_pages, Hq=G, Hkv=1, d=d, d_idx=64, topk=k)
    qt, qv = bf(np.broadcast_to(q, (R, G, d)))
    ws = api.new_paged_workspace(sh, api.OP_PAGED_ATTN)
    s = None if sel is None else i32(np.broadcast_to(sel, (R, 1, k)))
    o, lse = api.paged_attn(sh, qt, f8(k8), f8(v8), dev(ks), dev(vs), i32(np.repeat(table, R, 0)), i32(np.arange(R)),
                            i32([n - 1] * R), sel_idx=s, workspace=ws)
    api.check_device_status(ws)
    blocks = np.arange((n + PAGE - 1) // PAGE) if sel is None else sel[sel >= 0]
    seen = ((blocks[:, None] * PAGE + np.arange(PAGE)) < n).reshape(-1)
    pages = table[0, blocks]
    K = (ref.e4m3_decode(k8[pages, 0]) * ks[pages, 0].astype(np.float64)[:, None, None]).reshape(-1, d)[seen]
    V = (ref.e4m3_decode(v8[pages, 0]) * vs[pages, 0].astype(np.float64)[:, None, None]).reshape(-1, d)[seen]
    sv = np.repeat(vs[pages, 0].astype(np.float64), PAGE)[seen]
    ow, lw, do, dl = expected(qv[0], K, V, sv, float(np.float32(1) / np.sqrt(np.float32(d))))
    og, lg = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.abs(lg - lw) <= dl), np.max(np.abs(lg - lw) / dl)
    assert np.all(np.abs(og - ow) <= do), (np.max(np.abs(og - ow) / do), np.argwhere(np.abs(og - ow) > do)[:3])
    return og


@pytest.mark.parametrize("n,d,G", [(130, 64, 8), (2048, 128, 8), (2048, 64, 2), (32768, 128, 8), (131072, 64, 8), (131035, 128, 4), (20000, 64, 1)])
@pytest.mark.parametrize("rest", ["equal", "normal"])
@pytest.mark.parametrize("value", ["ones", "sink", "scales", "normal"])
def test_a_peaked_row(api, n, d, G, rest, value):
    """One row: cut into as many pieces as its length gives, the first with the sink."""
    q, cache, table, n_pages = peaked(n, d, G, rest, value)
    o = run(api, q, cache, table, n_pages, n, G, d)
    if value == "ones":
        assert np.all(np.abs(o - 1) <= 2.0 ** -7)


@pytest.mark.parametrize("R,n", [(64, 32768), (400, 2048), (400, 300)])
@pytest.mark.parametrize("rest", ["equal", "normal"])
@pytest.mark.parametrize("value", ["ones", "sink"])
def test_peaked_rows_cut_and_whole(api, R, n, rest, value):
    """Many requests over the same pages, in one or two pieces each (64) or whole (400 are not cut)."""
    q, cache, table, n_pages = peaked(n, 64, 8, rest, value)
    run(api, q, cache, table, n_pages, n, 8, 64, R=R)


@pytest.mark.parametrize("n,R", [(2048, 1), (2048, 64), (131072, 1), (131072, 400)])
@pytest.mark.parametrize("value", ["ones", "sink", "scales"])
def test_a_peaked_row_with_a_selection(api, n, R, value):
    """Sixteen blocks with the sink's among them, also where rows are not cut."""
    q, cache, table, n_pages = peaked(n, 128, 8, "normal", value)
    nb = table.shape[1]
    sel = np.unique(np.append(np.random.default_rng(n).choice(nb, 16, replace=False), [0, nb // 2, nb - 1]))
    sel = np.append(sel[sel != sel[3]] if len(sel) > 16 else sel, [-1] * 16)[:16].astype(np.int32)
    run(api, q, cache, table, n_pages, n, 8, 128, R=R, sel=sel)


def test_a_weight_that_grows_page_by_page(api):
    """Each page's weights outgrow all before it: what the levels below the first hold is rescaled with the rest."""
    d, G, n = 64, 8, 40 * PAGE
    q, cache, table, n_pages = peaked(n, d, G, "normal", "sink")
    k8, ks = cache[:2]
    for c in range(table.shape[1]):
        k8[table[0, c], 0, 17, :d // 2] = ref.e4m3_encode(np.full(d // 2, c * 0.03 / ks[table[0, c], 0]))
    run(api, q, cache, table, n_pages, n, G, d)
    run(api, q, cache, table, n_pages, n, G, d, R=400)


@pytest.mark.parametrize("n,d", [(200, 64), (9000, 128)])
@pytest.mark.parametrize("rest", ["equal", "normal"])
@pytest.mark.parametrize("value", ["sink", "scales"])
def test_tails_down_to_the_last_level(api, n, d, rest, value):
    """Sixteen to thirty-six nats below a sink without value: 8 bits down to 2^-42 (29 nats; 21 where the sink's page has 2^12
    times the scale), less behind that, nothing from 2^-50 on."""
    q, cache, table, n_pages = peaked(n, d, 8, rest, value, least=16, most=36)
    run(api, q, cache, table, n_pages, n, 8, d)
