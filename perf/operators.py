"""The operators of serving from a paged 8-bit KV cache: their cases, plain forms and 64-bit values.

Five operators make one decode (or chunked) step over a ragged batch of requests whose caches live in
128-token pages: the step's plan (page allocation, block tables, slot maps), the append that quantises the
new tokens' K and V rows to e4m3 with one power-of-two scale per (page, KV head), the index branch's block
scores, the block selection, and attention over the selected pages (or all of them).

A case is a dict of plain values.  "ctx" is the longest request's length after the step; the other
requests' lengths spread evenly from it down to an eighth (see _lens).  "q" is the most new tokens a
request brings: one in decoding, a few in speculative decoding, more in a prefill chunk.
"""
import math

import numpy as np
import torch

own = False

PAGE = 128

# Head layouts (Hq, Hkv, d, d_idx, topk) of the workload table and the parity tests.
HEADS = ((64, 8, 128, 128, 16), (32, 8, 128, 128, 16), (16, 4, 128, 64, 16), (8, 2, 64, 64, 4))


def _heads(i):
    return dict(zip(("Hq", "Hkv", "d", "d_idx", "k"), HEADS[i]))


def listed():
    big, mid, tiny = _heads(0), _heads(1), _heads(3)
    return [
        # one decode step of 64 requests, some of them idle: host-visible latency before the first kernel of a step
        {"name": "plan_decode_64", "op": "plan", "R": 64, "T": 64, "ctx": 32768, "ended": False},
        # chunked prefill of many requests at once, some slots freed in the same step
        {"name": "plan_chunks_256", "op": "plan", "R": 256, "T": 32768, "ctx": 131072, "ended": True},
        # one token per request into partly filled pages
        {"name": "append_decode_64", "op": "append", "R": 64, "q": 1, "ctx": 4096, **big},
        # prompts of up to 4,096 tokens written in one step, first and last pages partly filled
        {"name": "append_prefill_16", "op": "append", "R": 16, "q": 4096, "ctx": 5000, **mid},
        # a small model's scores over a short cache: latency
        {"name": "scores_small", "op": "scores", "R": 4, "q": 1, "ctx": 1000, **tiny},
        # the index scan of decoding at 1,048,576-token caches
        {"name": "scores_1m", "op": "scores", "R": 4, "q": 1, "ctx": 1048576, **big},
        # ranking 256 blocks per (request, group)
        {"name": "topk_decode_64", "op": "topk", "T": 64, "nb": 256, **big},
        # ranking a prefill chunk's rows over 1,024 blocks (131,072 tokens)
        {"name": "topk_chunk_1k", "op": "topk", "T": 1000, "nb": 1024, **big},
        # one request of a small model, every block of a short cache
        {"name": "attn_small", "op": "attn", "R": 1, "q": 1, "ctx": 1000, "sparse": False, **tiny},
        # ragged batch decoding over the selected blocks
        {"name": "attn_decode_64", "op": "attn", "R": 64, "q": 1, "ctx": 65536, "sparse": True, **big},
        # speculative decoding: up to five rows a request, each with its own selection
        {"name": "attn_spec_24", "op": "attn", "R": 24, "q": 5, "ctx": 20001, "sparse": True, **mid},
        # a layer that attends to everything, at 131,072-token caches
        {"name": "attn_dense_128k", "op": "attn", "R": 8, "q": 1, "ctx": 131072, "sparse": False, **big},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "append", "scores", "topk", "attn", "attn"))
    h = _heads(rng.randrange(len(HEADS)))
    if op == "plan":
        R = _between(rng, 1, 512)
        return {"op": op, "R": R, "T": R + _between(rng, 1, 32000) - 1, "ctx": _between(rng, 130, 131072), "ended": rng.random() < 0.5}
    if op == "append":
        R = _between(rng, 1, 256)
        q = _between(rng, 1, min(4096, 32768 // R))
        return {"op": op, "R": R, "q": q, "ctx": q + _between(rng, 1, 4096) - 1, **h}
    if op == "topk":
        T = _between(rng, 1, 1000)
        return {"op": op, "T": T, "nb": _between(rng, 1, min(8192, 1000000 // T)), **h}
    R = _between(rng, 1, 128)
    if op == "scores":
        q = _between(rng, 1, 16) if rng.random() < 0.5 else 1
        return {"op": op, "R": R, "q": q, "ctx": q + _between(rng, 1, min(524288, 1048576 // (R * q))) - 1, **h}
    sparse = rng.random() < 0.6
    q = _between(rng, 1, max(1, min(8, 160 // R))) if rng.random() < 0.5 else 1
    most = 131072 if sparse else min(131072, 524288 // (R * q))
    return {"op": op, "R": R, "q": q, "ctx": q + _between(rng, 1, min(most, 2097152 // R)) - 1, "sparse": sparse, **h}


# ---------------------------------------------------------------- lengths of a case (the same for every seed, up to their order)
def _lens(c):
    """(length after the step, new tokens) of each request."""
    i = np.arange(c["R"])
    q = c["q"] - (5 * i) % c["q"]
    n = (c["ctx"] * (1 - 0.875 * i / max(1, c["R"] - 1))).astype(np.int64) - (37 * i) % PAGE
    return np.maximum(n, q), q


def _plan_lens(c, rs):
    """(lengths before the step, new tokens, slots whose request ended) for a plan."""
    R, T = c["R"], c["T"]
    w = rs.exponential(size=R) ** 2
    new = np.floor((T - R) * w / w.sum()).astype(np.int64) + 1
    new = np.minimum(new, c["ctx"])
    new[rs.random(R) < 0.06] = 0
    old = rs.randint(0, c["ctx"] + 1, R)
    old = np.minimum(old, c["ctx"] - new)
    ended = (rs.random(R) < 0.1) & bool(c["ended"])
    new[ended] = 0
    return old, new, ended


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _pages(c, lens, rs):
    """A block table for the lengths, its pages in random order, and the number of pages of the pool."""
    need = (lens + PAGE - 1) // PAGE
    nb = int((c["ctx"] + PAGE - 1) // PAGE)
    n_pages = int(need.sum() + 5 + need.sum() // 16)
    ids = rs.permutation(n_pages)
    table = np.full((len(lens), nb), -1, dtype=np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at:at + m]
        at += m
    return table, n_pages


def _scale_of(amax):
    """The smallest power of two that brings amax to at most 448, the largest e4m3 value (2^-112 at the least)."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -112).clamp(min=-112)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _cache(g, n_pages, Hkv, d):
    """A filled 8-bit cache [n_pages, Hkv, 128, d] with its scales: normal rows, some features larger, as keys have them."""
    gain = torch.exp(0.3 * _randn(g, 1, Hkv, 1, d))
    codes = torch.empty(n_pages, Hkv, PAGE, d, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(n_pages, Hkv, device="cuda")
    step = max(1, (1 << 27) // (Hkv * PAGE * d))
    for a in range(0, n_pages, step):
        x = (_randn(g, min(step, n_pages - a), Hkv, PAGE, d) * gain).bfloat16().float()
        s = _scale_of(x.abs().amax((2, 3)))
        scales[a:a + step] = s
        codes[a:a + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
    return codes, scales


def _rows(lens, q):
    """q_starts, the request of each row and its position."""
    starts = np.concatenate([[0], np.cumsum(q)])
    req = np.repeat(np.arange(len(q)), q)
    pos = lens[req] - q[req] + np.arange(starts[-1]) - starts[req]
    return starts, req, pos


def prepare(case, seed):
    c, rs, g = case, np.random.RandomState(seed), _gen(seed)
    st = {"case": c}
    if c["op"] == "plan":
        old, new, ended = _plan_lens(c, np.random.RandomState(c["R"] * 7 + c["T"]))
        nb = (c["ctx"] + PAGE - 1) // PAGE
        held = (old + PAGE - 1) // PAGE
        n_pages = int(held.sum() + (new // PAGE + 1).sum() + 9)
        ids = rs.permutation(n_pages).astype(np.int32)
        table = np.full((c["R"], nb), -1, dtype=np.int32)
        at = 0
        for r, m in enumerate(held):
            table[r, :m] = ids[at:at + m]
            at += m
        free, head = n_pages - at, int(rs.randint(n_pages))
        ring = np.full(n_pages, -1, dtype=np.int32)
        ring[(head + np.arange(free)) % n_pages] = ids[at:]
        st.update(new_lens=_i32(new), lens=_i32(old), table=_i32(table), ring=_i32(ring), free=_i32([head, free]),
                  ended=_i32(ended) if c["ended"] else None, n_pages=n_pages)
        return st
    if c["op"] == "topk":
        T, nb = c["T"], c["nb"]
        pos = rs.randint(0, nb * PAGE, T)
        pos[0] = nb * PAGE - 1
        s = _randn(g, T, c["Hkv"], nb)
        s = torch.where(torch.rand(T, 1, 1, device="cuda", generator=g) < 0.25, (s * 8).round() / 8, s)  # rows with ties
        pos = _i32(pos)
        s.masked_fill_(torch.arange(nb, device="cuda") > (pos // PAGE)[:, None, None], -math.inf)
        st.update(scores=s, pos=pos)
        return st
    lens, q = _lens(c)
    order = rs.permutation(c["R"])
    lens, q = lens[order], q[order]
    starts, req, pos = _rows(lens, q)
    table, n_pages = _pages(c, lens, rs)
    st.update(table=_i32(table), starts=_i32(starts), req=_i32(req), pos=_i32(pos), n_pages=n_pages, T=len(req))
    Hq, Hkv, d, di = c["Hq"], c["Hkv"], c["d"], c["d_idx"]
    if c["op"] == "append":
        slots = table[req, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
        first = np.flatnonzero((pos % PAGE == 0) | (np.arange(len(req)) == starts[req]))
        S = min(len(req), 2 * c["R"] + len(req) // PAGE)
        segs = np.full(S + 1, len(req), dtype=np.int32)
        segs[:len(first)] = first
        st["n_segs"] = len(first)
        st["k8"], st["k_scale"] = _cache(g, n_pages, Hkv, d)
        st["v8"], st["v_scale"] = _cache(g, n_pages, Hkv, d)
        st["k_idx"] = _randn(g, n_pages, PAGE, di).bfloat16()
        T = len(req)
        st.update(slots=_i32(slots), segs=_i32(segs), k_new=(2 * _randn(g, T, Hkv, d)).bfloat16(),
                  v_new=_randn(g, T, Hkv, d).bfloat16(), k_idx_new=_randn(g, T, di).bfloat16())
    elif c["op"] == "scores":
        st["q_idx"] = _randn(g, len(req), Hkv, di).bfloat16()
        st["k_idx"] = torch.empty(n_pages, PAGE, di, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    else:
        st["q"] = _randn(g, len(req), Hq, d).bfloat16()
        st["k8"], st["k_scale"] = _cache(g, n_pages, Hkv, d)
        st["v8"], st["v_scale"] = _cache(g, n_pages, Hkv, d)
        st["sel"] = None
        if c["sparse"]:
            nb, k = table.shape[1], c["k"]
            c0 = (st["pos"] // PAGE)[:, None, None]
            s = torch.rand(len(req), Hkv, nb, device="cuda", generator=g)
            at = torch.arange(nb, device="cuda")
            s = torch.where(at < c0, s, torch.where(at == c0, 2.0, -1.0))
            v, i = s.topk(min(k, nb), dim=2)
            i = torch.where(v >= 0, i, nb).sort(dim=2).values
            sel = torch.full((len(req), Hkv, k), -1, dtype=torch.int32, device="cuda")
            sel[:, :, :i.shape[2]] = torch.where(i < nb, i, -1).int()
            st["sel"] = sel
    return st


# ---------------------------------------------------------------- the framework's calls
def _handles(st, op_name):
    """The shape and workspace that a serving loop keeps: made on a state's first pass."""
    if "own" not in st:
        from block_sparse_gqa_causal_gb300 import api
        c = st["case"]
        if c["op"] == "topk":
            T, R, nb, n_pages = c["T"], c["T"], c["nb"], 1
        elif c["op"] == "plan":
            T, R, nb, n_pages = c["T"], c["R"], st["table"].shape[1], st["n_pages"]
        else:
            T, R, nb, n_pages = st["T"], c["R"], st["table"].shape[1], st["n_pages"]
        h = c if "Hq" in c else _heads(0)
        sh = api.PagedShape(R=R, T=T, max_blocks=nb, n_pages=n_pages, Hq=h["Hq"], Hkv=h["Hkv"], d=h["d"], d_idx=h["d_idx"], topk=h["k"])
        st["own"] = (api, sh, api.new_paged_workspace(sh, getattr(api, op_name)))
    return st["own"]


def _run_own(st):
    op = st["case"]["op"]
    if op == "plan":
        api, sh, ws = _handles(st, "OP_PAGED_PLAN")
        p = api.paged_plan(sh, st["new_lens"], st["lens"], st["table"], st["ring"], st["free"], ended=st["ended"], workspace=ws)
        return {"table": st["table"], "ring": st["ring"], "lens": p.lens, "free": p.free_state, "starts": p.q_starts,
                "req": p.row_req, "pos": p.row_pos, "slots": p.slots, "segs": p.segs}
    if op == "append":
        api, sh, ws = _handles(st, "OP_PAGED_APPEND")
        api.paged_append(sh, st["k_new"], st["v_new"], st["k_idx_new"], st["slots"], st["segs"], st["k8"], st["v8"], st["k_scale"],
                         st["v_scale"], st["k_idx"], workspace=ws)
        return {"k8": st["k8"], "v8": st["v8"], "k_scale": st["k_scale"], "v_scale": st["v_scale"], "k_idx": st["k_idx"]}
    if op == "scores":
        api, sh, ws = _handles(st, "OP_PAGED_BLOCK_SCORES")
        return api.paged_block_scores(sh, st["q_idx"], st["k_idx"], st["table"], st["starts"], st["req"], st["pos"], workspace=ws)
    if op == "topk":
        api, sh, ws = _handles(st, "OP_PAGED_BLOCK_TOPK")
        return api.paged_block_topk(sh, st["scores"], st["pos"], workspace=ws)
    api, sh, ws = _handles(st, "OP_PAGED_ATTN")
    o, lse = api.paged_attn(sh, st["q"], st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["table"], st["req"], st["pos"],
                            sel_idx=st["sel"], workspace=ws)
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- the plain forms
def _plain_plan(st):
    new, table, ring = st["new_lens"].long(), st["table"], st["ring"]
    dev, R, T = new.device, st["case"]["R"], st["case"]["T"]
    nb, n_pages = table.shape[1], st["n_pages"]
    head, count = st["free"][0].long(), st["free"][1].long()
    lens = st["lens"].long()
    ended = torch.zeros(R, dtype=torch.bool, device=dev) if st["ended"] is None else st["ended"] != 0
    pages = lambda n: (n + PAGE - 1) // PAGE  # noqa: E731
    gone = torch.where(ended, pages(lens), 0)
    old = torch.where(ended, 0, lens)
    held, after = pages(old), pages(old + new)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)])
    take = after - held
    base = take.cumsum(0) - take
    back = gone.cumsum(0) - gone
    nseg = torch.where(new > 0, after - old // PAGE, 0)
    sbase = nseg.cumsum(0) - nseg
    # released pages go behind the free ones
    col = torch.arange(nb, device=dev)
    mask = col < gone[:, None]
    at = torch.where(mask, (head + count + back[:, None] + col) % n_pages, n_pages)
    wide = torch.cat([ring, ring.new_zeros(1)])
    wide.scatter_(0, at.reshape(-1), table.reshape(-1))
    ring_out = wide[:-1]
    # new pages come from the front
    mask = (col >= held[:, None]) & (col < after[:, None])
    table_out = torch.where(mask, ring[(head + base[:, None] + col - held[:, None]) % n_pages], table)
    t = torch.arange(T, device=dev)
    live = t < starts[-1]
    req = torch.searchsorted(starts[1:], t, right=True).clamp(max=R - 1)
    pos = old[req] + t - starts[req]
    blk = pos // PAGE
    slots = table_out[req, blk.clamp(max=nb - 1)].long() * PAGE + pos % PAGE
    opens = live & ((t == starts[req]) | (pos % PAGE == 0))
    S = min(T, 2 * R + T // PAGE)
    segs = torch.full((S + 2,), 0, dtype=torch.int64, device=dev) + starts[-1]
    segs.scatter_(0, torch.where(opens, sbase[req] + blk - old[req] // PAGE, S + 1), t)
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table_out, "ring": ring_out, "lens": i32(old + new),
            "free": i32(torch.stack([(head + take.sum()) % n_pages, count - take.sum() + gone.sum()])), "starts": i32(starts),
            "req": i32(torch.where(live, req, -1)), "pos": i32(torch.where(live, pos, -1)), "slots": i32(torch.where(live, slots, -1)),
            "segs": i32(segs[:S + 1])}


def _plain_append_one(new, codes, scales, seg_of, page, off0, slots):
    """The new rows [T, H, d] into the cache's pages: a page keeps one scale per head for all of its rows."""
    S, H = page.shape[0], codes.shape[1]
    x = new.float()
    amax = torch.zeros(S, H, device=x.device).scatter_reduce_(0, seg_of[:, None].expand(-1, H), x.abs().amax(2), "amax")
    need = _scale_of(amax)
    had = scales[page]
    s = torch.where(off0[:, None] > 0, torch.maximum(had, need), need)
    flat = codes.view(torch.uint8)
    before = flat[page].view(torch.float8_e4m3fn).float() * (had / s)[:, :, None, None]
    kept = torch.arange(PAGE, device=x.device)[None, None, :, None] < off0[:, None, None, None]
    flat[page] = torch.where(kept, before.to(torch.float8_e4m3fn).view(torch.uint8), flat[page])
    scales[page] = s
    flat[slots // PAGE, :, slots % PAGE] = (x / s[seg_of][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(st):
    segs, slots = st["segs"].long()[:st["n_segs"] + 1], st["slots"].long()
    page, off0 = slots[segs[:-1]] // PAGE, slots[segs[:-1]] % PAGE
    seg_of = torch.searchsorted(segs[1:], torch.arange(st["T"], device=segs.device), right=True)
    _plain_append_one(st["k_new"], st["k8"], st["k_scale"], seg_of, page, off0, slots)
    _plain_append_one(st["v_new"], st["v8"], st["v_scale"], seg_of, page, off0, slots)
    st["k_idx"].view(-1, st["k_idx"].shape[2])[slots] = st["k_idx_new"]
    return {"k8": st["k8"], "v8": st["v8"], "k_scale": st["k_scale"], "v_scale": st["v_scale"], "k_idx": st["k_idx"]}


def _padded(st, x):
    """x [T, ...] as [R, q, ...], and the place of each row in it."""
    R, q = st["case"]["R"], st["case"]["q"]
    i = torch.arange(q, device=x.device)
    at = (st["starts"][:-1, None].long() + i).clamp(max=st["T"] - 1)
    req = st["req"].long()
    return x[at], req, torch.arange(st["T"], device=x.device) - st["starts"].long()[req]


def _plain_scores(st):
    c, table = st["case"], st["table"].long().clamp(min=0)
    R, nb, di = c["R"], table.shape[1], c["d_idx"]
    k = st["k_idx"][table].float().reshape(R, nb * PAGE, di)
    qp, req, i = _padded(st, st["q_idx"].float())
    s = torch.matmul(qp.reshape(R, -1, di), k.transpose(1, 2)) / math.sqrt(di)
    s = s.reshape(R, c["q"], c["Hkv"], nb, PAGE)[req, i]
    at = torch.arange(nb * PAGE, device=s.device).reshape(nb, PAGE)
    return s.masked_fill_(at > st["pos"][:, None, None, None], -math.inf).amax(3)


def _plain_topk(st):
    c, s = st["case"], st["scores"]
    nb, k = s.shape[2], c["k"]
    c0 = (st["pos"] // PAGE)[:, None, None]
    at = torch.arange(nb, device=s.device)
    s = torch.where(at == c0, math.inf, torch.where(at < c0, s, -math.inf))
    i = torch.sort(s, dim=2, descending=True, stable=True).indices[:, :, :k]
    i = torch.where(i <= c0, i, nb).sort(dim=2).values
    i = torch.cat([i, i.new_full((s.shape[0], s.shape[1], k - i.shape[2]), nb)], dim=2)
    return torch.where(i < nb, i, -1).int()


def _plain_attn(st):
    c = st["case"]
    T, Hq, Hkv, d = st["T"], c["Hq"], c["Hkv"], c["d"]
    G, pos, req = Hq // Hkv, st["pos"].long(), st["req"].long()
    head = torch.arange(Hkv, device=pos.device)

    def pages(codes, scales, page, h):
        return codes.view(torch.uint8)[page, h].view(torch.float8_e4m3fn).float() * scales[page, h][..., None, None]

    if st["sel"] is not None:
        sel = st["sel"].long()
        page = st["table"].long()[req[:, None, None], sel.clamp(min=0)].clamp(min=0)
        h = head[None, :, None].expand_as(page)
        at = sel[..., None] * PAGE + torch.arange(PAGE, device=pos.device)
        out = ((sel < 0)[..., None] | (at > pos[:, None, None, None])).reshape(T, Hkv, 1, -1)
        k = pages(st["k8"], st["k_scale"], page, h).reshape(T, Hkv, -1, d)
        s = torch.matmul(st["q"].float().reshape(T, Hkv, G, d), k.transpose(2, 3)) / math.sqrt(d)
        del k
        s.masked_fill_(out, -math.inf)
        m = s.amax(3, keepdim=True)
        e = torch.exp(s - m)
        z = e.sum(3, keepdim=True)
        o = torch.matmul(e, pages(st["v8"], st["v_scale"], page, h).reshape(T, Hkv, -1, d)) / z
        return {"o": o.reshape(T, Hq, d).bfloat16(), "lse": (m + z.log()).reshape(T, Hq)}
    R, q, nb = c["R"], c["q"], st["table"].shape[1]
    page = st["table"].long().clamp(min=0)[:, None, :].expand(R, Hkv, nb)
    h = head[None, :, None].expand_as(page)
    qp, req, i = _padded(st, st["q"].float())
    pp, _, _ = _padded(st, pos)
    qp = qp.reshape(R, q, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, q * G, d)
    k = pages(st["k8"], st["k_scale"], page, h).reshape(R, Hkv, nb * PAGE, d)
    s = torch.matmul(qp, k.transpose(2, 3)) / math.sqrt(d)
    del k
    late = torch.arange(nb * PAGE, device=pos.device) > pp[:, :, None]
    s.view(R, Hkv, q, G, -1).masked_fill_(late[:, None, :, None], -math.inf)
    m = s.amax(3, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(3, keepdim=True)
    o = torch.matmul(e, pages(st["v8"], st["v_scale"], page, h).reshape(R, Hkv, nb * PAGE, d)) / z
    back = lambda x: x.reshape(R, Hkv, q, G, -1).permute(0, 2, 1, 3, 4)[req, i].reshape(T, Hq, -1)  # noqa: E731
    return {"o": back(o).bfloat16(), "lse": back(m + z.log())[..., 0].contiguous()}


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "append": _plain_append, "scores": _plain_scores, "topk": _plain_topk, "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "plan":
        old, new, ended = _plan_lens(c, np.random.RandomState(c["R"] * 7 + c["T"]))
        pages = lambda n: (n + PAGE - 1) // PAGE  # noqa: E731
        before = np.where(ended, 0, old)
        taken = int((pages(before + new) - pages(before)).sum())
        freed = int(np.where(ended, pages(old), 0).sum())
        S = min(c["T"], 2 * c["R"] + c["T"] // PAGE)
        return {"bytes": 4 * (4 * c["R"] + 2 * taken + 2 * freed + 3 * c["T"] + S + 6), "flops": 0}
    if c["op"] == "topk":
        rs_free = c["T"] * c["Hkv"]
        return {"bytes": 4 * (rs_free * (c["nb"] // 2 + c["k"]) + c["T"]), "flops": 0}
    lens, q = _lens(c)
    T = int(q.sum())
    if c["op"] == "append":
        tok = 2 * c["Hkv"] * c["d"]
        return {"bytes": T * (tok * 3 + c["d_idx"] * 4 + 4), "flops": 0}
    if c["op"] == "scores":
        n = int(lens.sum())
        last = (lens + PAGE - 1) // PAGE
        return {"bytes": n * c["d_idx"] * 2 + T * c["Hkv"] * (c["d_idx"] * 2 + 4 * int(last.max())),
                "flops": 2 * int((lens * q).sum()) * c["Hkv"] * c["d_idx"]}
    pos = _rows(lens, q)[2]
    if c["sparse"]:
        nblk = np.minimum(pos // PAGE + 1, c["k"])
        seen = (nblk - 1) * PAGE + pos % PAGE + 1
    else:
        seen = pos + 1
    kv = int(np.minimum(np.bincount(_rows(lens, q)[1], seen), lens).sum())  # a request's rows share what they read
    return {"bytes": kv * c["Hkv"] * c["d"] * 2 + T * c["Hq"] * (c["d"] * 4 + 4), "flops": 4 * int(seen.sum()) * c["Hq"] * c["d"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """The nearest e4m3 values, ties to even, of doubles within +-448."""
    y = x.abs()
    e = torch.floor(torch.log2(y.clamp(min=2.0 ** -20))).clamp(min=-6)
    e = torch.where(y >= _two_to(e + 1), e + 1, e)
    e = torch.where(y < _two_to(e), e - 1, e).clamp(min=-6)
    step = _two_to(e - 3)
    return torch.round(x / step) * step


def _exact_append(st):
    res = {}
    slots, segs = st["slots"].tolist(), st["segs"].tolist()
    spans = [(a, b) for a, b in zip(segs[:-1], segs[1:]) if b > a]
    if len(spans) > 1500:
        return None
    for name in ("k", "v"):
        codes, scales = st[name + "8"].double(), st[name + "_scale"].double()
        new = st[name + "_new"].double()
        for a, b in spans:
            page, off = divmod(slots[a], PAGE)
            x = new[a:b].transpose(0, 1)
            top = x.abs().amax((1, 2))
            e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -112)))
            e = torch.where(448 * _two_to(e - 1) >= top, e - 1, e).clamp(min=-112)
            e = torch.where(448 * _two_to(e) < top, e + 1, e)
            s = _two_to(e)
            if off:
                s = torch.maximum(s, scales[page])
                codes[page, :, :off] = _e4m3(codes[page, :, :off] * (scales[page] / s)[:, None, None])
            codes[page, :, off:off + b - a] = _e4m3(x / s[:, None, None])
            scales[page] = s
        res[name + "8"], res[name + "_scale"] = codes, scales
    flat = st["k_idx"].double()
    flat.view(-1, flat.shape[2])[st["slots"].long()] = st["k_idx_new"].double()
    res["k_idx"] = flat
    return res


def exact(case, seed):
    c = case
    if c["op"] in ("plan", "topk"):
        return None  # whole numbers
    st = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(st)
    lens, q = _lens(c)
    order = np.random.RandomState(seed).permutation(c["R"])
    lens, q = lens[order], q[order]
    table, t0 = st["table"].long(), 0
    nb = table.shape[1]
    if c["op"] == "scores":
        res = torch.full((st["T"], c["Hkv"], nb), -math.inf, dtype=torch.float64, device="cuda")
        for r in range(c["R"]):
            for i in range(int(q[r])):
                n = int(lens[r] - q[r] + i + 1)
                blocks = (n + PAGE - 1) // PAGE
                for a in range(0, blocks, 1024):
                    b = min(blocks, a + 1024)
                    k = st["k_idx"][table[r, a:b]].double().flatten(0, 1)
                    s = torch.einsum("gd,nd->gn", st["q_idx"][t0].double(), k) * c["d_idx"] ** -0.5
                    s[:, max(0, n - a * PAGE):] = -math.inf
                    res[t0, :, a:b] = s.reshape(c["Hkv"], b - a, PAGE).amax(2)
                t0 += 1
        return res
    G, d = c["Hq"] // c["Hkv"], c["d"]
    o = torch.zeros(st["T"], c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["T"], c["Hq"], dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        for i in range(int(q[r])):
            n = int(lens[r] - q[r] + i + 1)
            for g in range(c["Hkv"]):
                if st["sel"] is None:
                    blocks = torch.arange((n + PAGE - 1) // PAGE, device="cuda")
                else:
                    blocks = st["sel"][t0, g].long()
                    blocks = blocks[blocks >= 0]
                page = table[r, blocks]
                seen = (blocks[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten() < n
                k = (st["k8"].view(torch.uint8)[page, g].view(torch.float8_e4m3fn).double() * st["k_scale"][page, g].double()[:, None, None]).flatten(0, 1)[seen]
                v = (st["v8"].view(torch.uint8)[page, g].view(torch.float8_e4m3fn).double() * st["v_scale"][page, g].double()[:, None, None]).flatten(0, 1)[seen]
                h = slice(g * G, (g + 1) * G)
                x = torch.einsum("hd,nd->hn", st["q"][t0, h].double(), k) / math.sqrt(d)
                lse[t0, h] = torch.logsumexp(x, 1)
                o[t0, h] = torch.softmax(x, 1) @ v
            t0 += 1
    return {"o": o, "lse": lse}
