"""The operators of prompts served in chunks from the paged 8-bit KV cache, and the rotary positions that serving and
training put on queries and keys: their cases, plain forms and 64-bit values.

  rotary        queries and keys turned by their positions (forward, and backward for training)
  fork          requests that go on from another request's cache (beams, shared prompts): whole pages shared and counted,
                partly filled ones copied, pages that nobody holds any more given back
  compact       the pages in use moved to the pool's front
  chunk_scores  the index branch's block scores for chunks of new tokens, whose rows share what they read
  chunk_attn    attention of such chunks over selected blocks, or over everything

A case is a dict of plain values.  "ctx" is the longest request's length after the step; the other requests' lengths
spread evenly from it down to an eighth (see _lens).  "q" is the most new tokens a request brings.
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
        # one decode step of 64 requests in a long-context model: latency
        {"name": "rotary_decode_64", "op": "rotary", "bwd": False, "T": 64, "N": 0, "ctx": 1048576, "rot": 128, "inter": False,
         "fused": True, "base": 1e6, "factor": 8.0, **big},
        # a training step's queries and keys, slices of one projection's output
        {"name": "rotary_train_32k", "op": "rotary", "bwd": False, "T": 32768, "N": 32768, "ctx": 32768, "rot": 128, "inter": False,
         "fused": True, "base": 1e4, "factor": 1.0, **big},
        # the gradients of such a step: half of each head turned, neighbours paired, an odd length
        {"name": "rotary_train_bwd", "op": "rotary", "bwd": True, "T": 3 * 8001, "N": 8001, "ctx": 8001, "rot": 64, "inter": True,
         "fused": False, "base": 1e4, "factor": 1.0, **mid},
        # eight beams of a small model that change places after a step: latency
        {"name": "fork_beams_8", "op": "fork", "R": 8, "width": 8, "ctx": 1000, **tiny},
        # 256 requests started from four long prompts
        {"name": "fork_prompts_256", "op": "fork", "R": 256, "width": 64, "ctx": 32120, **big},
        # a small pool with a third of its pages in use
        {"name": "compact_small", "op": "compact", "R": 8, "ctx": 2000, "live": 0.33, **tiny},
        # a pool of which most requests have ended, to be cut to what is in use
        {"name": "compact_half", "op": "compact", "R": 24, "ctx": 20000, "live": 0.5, **big},
        # short chunks of a small model
        {"name": "scores_chunk_small", "op": "chunk_scores", "R": 3, "q": 100, "ctx": 1000, **tiny},
        # a 2,048-token chunk at the end of a 32,768-token prompt
        {"name": "scores_chunk_2k", "op": "chunk_scores", "R": 1, "q": 2048, "ctx": 32768, **big},
        # several short chunks of a small model, every block
        {"name": "attn_chunk_small", "op": "chunk_attn", "R": 12, "q": 19, "ctx": 3001, "sparse": False, **tiny},
        # two prompts' chunks over the blocks that their rows selected
        {"name": "attn_chunk_sparse", "op": "chunk_attn", "R": 2, "q": 1500, "ctx": 50001, "sparse": True, **mid},
        # a layer that attends to everything: a 2,048-token chunk at the end of a 32,768-token prompt
        {"name": "attn_chunk_dense", "op": "chunk_attn", "R": 1, "q": 2048, "ctx": 32768, "sparse": False, **big},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "rotary", "fork", "compact", "chunk_scores", "chunk_attn", "chunk_attn"))
    h = _heads(rng.randrange(len(HEADS)))
    if op == "rotary":
        rot = h["d"] if rng.random() < 0.6 else 16 * rng.randint(1, h["d"] // 16)
        train = rng.random() < 0.7
        T = _between(rng, 1, 32768) if train else _between(rng, 1, 512)
        N = _between(rng, 1, T) if train else 0
        ctx = N if train else _between(rng, 1, 1048576)
        return {"op": op, "bwd": train and rng.random() < 0.5, "T": T, "N": N, "ctx": ctx, "rot": rot, "inter": rng.random() < 0.5,
                "fused": rng.random() < 0.5, "base": rng.choice((1e4, 5e5, 1e6)), "factor": rng.choice((1.0, 4.0, 8.0)), **h}
    if op == "fork":
        width = _between(rng, 2, 64)
        return {"op": op, "R": width * _between(rng, 1, 240 // width), "width": width, "ctx": _between(rng, 1, 32000), **h}
    if op == "compact":
        R, live = _between(rng, 1, 64), rng.uniform(0.25, 0.95)
        return {"op": op, "R": R, "ctx": _between(rng, 1, int(280000 * min(1, 0.5 / (1 - live))) // R), "live": live, **h}
    R = _between(rng, 1, 16)
    q = _between(rng, 1, 2048 // R)
    most = 32768 * 2048 // (R * q)
    if op == "chunk_scores":
        return {"op": op, "R": R, "q": q, "ctx": q + _between(rng, 1, min(131072 // R, most) - q) - 1, **h}
    sparse = rng.random() < 0.5
    return {"op": op, "R": R, "q": q, "ctx": q + _between(rng, 1, min(131072 // R, most) - q) - 1, "sparse": sparse, **h}


# ---------------------------------------------------------------- lengths of a case (the same for every seed, up to their order)
def _lens(c):
    """(length after the step, new tokens) of each request."""
    i = np.arange(c["R"])
    q = c["q"] - (5 * i) % c["q"]
    n = (c["ctx"] * (1 - 0.875 * i / max(1, c["R"] - 1))).astype(np.int64) - (37 * i) % PAGE
    return np.maximum(n, q), q


def _fork_lens(c):
    """Requests come in families of `width`: (the family's length, its whole pages that all members share) of each request."""
    fam = np.arange(c["R"]) // c["width"]
    n = np.maximum(1, (c["ctx"] * (1 - 0.5 * fam / max(1, fam.max()))).astype(np.int64) - 37 * fam % PAGE)
    return n, np.maximum(0, n // PAGE - 2)


def _fork_src(c, rs):
    """Whom each request goes on from: of a family, its first member stays, one in sixteen ends, the others take a member's cache."""
    i = np.arange(c["R"])
    first = i // c["width"] * c["width"]
    ends = (rs.random(c["R"]) < 1 / 16) & (i > first)
    src = first + np.where(rs.random(c["R"]) < 0.5, 0, rs.randint(0, c["width"], c["R"]))
    src = np.where(ends[src], first, src)
    return np.where(i == first, i, np.where(ends, -1, src))


def _compact_lens(c):
    """Lengths of the requests that are left; the first four share their first half."""
    i = np.arange(c["R"])
    return np.maximum(1, (c["ctx"] * (1 - 0.75 * i / max(1, c["R"] - 1))).astype(np.int64) - (37 * i) % PAGE)


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g, dtype=torch.float32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _scale_of(amax):
    """The smallest power of two that brings amax to at most 448, the largest e4m3 value."""
    m, e = torch.frexp(amax)
    return ((e - 9 + (m > 0.875).int() + 127) << 23).to(torch.int32).view(torch.float32)


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


def _caches(st, g, c, n_pages):
    st["k8"], st["k_scale"] = _cache(g, n_pages, c["Hkv"], c["d"])
    st["v8"], st["v_scale"] = _cache(g, n_pages, c["Hkv"], c["d"])
    st["k_idx"] = torch.empty(n_pages, PAGE, c["d_idx"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _rows(lens, q):
    """q_starts, the request of each row and its position."""
    starts = np.concatenate([[0], np.cumsum(q)])
    req = np.repeat(np.arange(len(q)), q)
    pos = lens[req] - q[req] + np.arange(starts[-1]) - starts[req]
    return starts, req, pos


def _selection(g, st, c):
    """Blocks as a trained index branch selects them: some matter to a whole request, some to a stretch of its rows, some to one row."""
    T, H, nb, k = st["T"], c["Hkv"], st["table"].shape[1], c["k"]
    req, pos = st["req"].long(), st["pos"].long()
    spell = pos // 64
    spell = spell - spell.min()
    s = _randn(g, c["R"], H, nb)[req] + _randn(g, int(spell.max()) + 1, H, nb)[spell]
    s += 0.5 * _randn(g, T, H, nb)
    c0 = (pos // PAGE)[:, None, None]
    at = torch.arange(nb, device="cuda")
    s = torch.where(at < c0, s, torch.where(at == c0, math.inf, -math.inf))
    v, i = s.topk(min(k, nb), dim=2)
    i = torch.where(v > -math.inf, i, nb).sort(dim=2).values
    sel = torch.full((T, H, k), -1, dtype=torch.int32, device="cuda")
    sel[:, :, :i.shape[2]] = torch.where(i < nb, i, -1).int()
    return sel


def prepare(case, seed):
    c, rs, g = case, np.random.RandomState(seed), _gen(seed)
    st = {"case": c}
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "rotary":
        T = c["T"]
        x = _randn(g, T, Hq + 2 * Hkv, d).bfloat16()
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
        if not c["fused"]:
            q, k = q.contiguous(), k.contiguous()
        st.update(q=q, k=k, pos=None if c["N"] else _i32(rs.randint(0, c["ctx"], T)))
        return st
    if c["op"] == "fork":
        R = c["R"]
        lens, common = _fork_lens(c)
        held = _pages_of(lens)
        nb = int(held.max()) + 3
        fam = np.arange(R) // c["width"]
        heads = np.arange(0, R, c["width"])
        n_pages = int((held - common).sum() + common[heads].sum() + 2 * R + 7)
        ids = rs.permutation(n_pages)
        table = np.full((R, nb), -1, dtype=np.int32)
        shares = np.zeros(n_pages, dtype=np.int32)
        at = 0
        for f, r in enumerate(heads):
            m = int(common[r])
            members = np.flatnonzero(fam == f)
            table[members, :m] = ids[at:at + m]
            shares[ids[at:at + m]] = len(members) - 1
            at += m
            for i in members:
                table[i, m:held[i]] = ids[at:at + held[i] - m]
                at += int(held[i] - m)
        count, head = n_pages - at, int(rs.randint(n_pages))
        ring = np.full(n_pages, -1, dtype=np.int32)
        ring[(head + np.arange(count)) % n_pages] = ids[at:]
        src = _fork_src(c, np.random.RandomState(R * 7 + c["ctx"]))
        moved = np.flatnonzero((src >= 0) & (src != np.arange(R)) & (lens % PAGE != 0))
        st.update(src=_i32(src), lens=_i32(lens), table=_i32(table), ring=_i32(ring), free=_i32([head, count]), shares=_i32(shares),
                  moved=torch.from_numpy(moved).cuda(), n_pages=n_pages)
        _caches(st, g, c, n_pages)
        return st
    if c["op"] == "compact":
        lens = _compact_lens(c)
        held = _pages_of(lens)
        half = int(held[:4].min()) // 2
        with_first = np.arange(c["R"]) < 4
        used = int(held.sum() - half * max(0, min(4, c["R"]) - 1))
        n_pages = int(used / c["live"]) + 3
        ids = rs.permutation(n_pages)
        table = np.full((c["R"], int(held.max())), -1, dtype=np.int32)
        shares = np.zeros(n_pages, dtype=np.int32)
        table[with_first, :half] = ids[:half]
        shares[ids[:half]] = int(with_first.sum()) - 1
        at = half
        for r, m in enumerate(held):
            b = half if with_first[r] else 0
            table[r, b:m] = ids[at:at + m - b]
            at += int(m - b)
        st.update(lens=_i32(lens), table=_i32(table), shares=_i32(shares), n_pages=n_pages, n_moves=int((ids[:at] >= at).sum()))
        _caches(st, g, c, n_pages)
        return st
    lens, q = _lens(c)
    order = rs.permutation(c["R"])
    lens, q = lens[order], q[order]
    starts, req, pos = _rows(lens, q)
    need = _pages_of(lens)
    n_pages = int(need.sum() + 5 + need.sum() // 16)
    ids = rs.permutation(n_pages)
    table = np.full((c["R"], int(_pages_of(c["ctx"]))), -1, dtype=np.int32)
    at = 0
    for r, m in enumerate(need):
        table[r, :m] = ids[at:at + m]
        at += m
    st.update(table=_i32(table), starts=_i32(starts), req=_i32(req), pos=_i32(pos), n_pages=n_pages, T=len(req))
    if c["op"] == "chunk_scores":
        st["q_idx"] = _randn(g, st["T"], Hkv, c["d_idx"]).bfloat16()
        st["k_idx"] = torch.empty(n_pages, PAGE, c["d_idx"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    else:
        st["q"] = _randn(g, st["T"], Hq, d).bfloat16()
        st["k8"], st["k_scale"] = _cache(g, n_pages, Hkv, d)
        st["v8"], st["v_scale"] = _cache(g, n_pages, Hkv, d)
        st["sel"] = _selection(g, st, c) if c["sparse"] else None
    return st


# ---------------------------------------------------------------- the framework's calls
def _handles(st):
    """The shapes, tables and workspaces that a program keeps: made on a state's first pass."""
    if "own" not in st:
        from block_sparse_gqa_causal_gb300 import api
        c = st["case"]
        if c["op"] == "rotary":
            sh = api.RotaryShape(T=c["T"], Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"], d_rot=c["rot"], interleaved=c["inter"], period=c["N"],
                                 scale=api.rotary_scale(c["factor"]))
            st["own"] = (api, sh, api.rotary_freqs(c["rot"], c["base"], factor=c["factor"], original_len=8192))
        else:
            sh = api.PagedShape(R=c["R"], T=st.get("T", c["R"]), max_blocks=st["table"].shape[1], n_pages=st["n_pages"], Hq=c["Hq"],
                                Hkv=c["Hkv"], d=c["d"], d_idx=c["d_idx"], topk=c["k"])
            op = {"fork": api.OP_PAGED_FORK, "compact": api.OP_PAGED_COMPACT, "chunk_scores": api.OP_PAGED_CHUNK_SCORES,
                  "chunk_attn": api.OP_PAGED_CHUNK_ATTN}[c["op"]]
            st["own"] = (api, sh, api.new_paged_workspace(sh, op))
    return st["own"]


def _run_own(st):
    c = st["case"]
    api, sh, kept = _handles(st)
    if c["op"] == "rotary":
        q, k = (api.rotary_bwd if c["bwd"] else api.rotary_fwd)(sh, st["q"], st["k"], kept, positions=st["pos"])
        return {"q": q, "k": k}
    caches = [st.get(n) for n in ("k8", "v8", "k_scale", "v_scale", "k_idx")]
    if c["op"] == "fork":
        moves = api.paged_fork(sh, st["src"], st["lens"], st["table"], st["ring"], st["free"], st["shares"], workspace=kept)
        api.paged_copy(sh, moves, *caches, workspace=kept)
        return _fork_outputs(st, moves)
    if c["op"] == "compact":
        p = api.paged_compact(sh, st["lens"], st["table"], st["shares"], workspace=kept)
        api.paged_copy(sh, p.moves, *caches, workspace=kept)
        return _compact_outputs(st, p.block_table, p.free_pages, p.free_state, p.shares, p.moves)
    if c["op"] == "chunk_scores":
        return api.paged_chunk_scores(sh, st["q_idx"], st["k_idx"], st["table"], st["starts"], st["pos"], workspace=kept)
    o, lse = api.paged_chunk_attn(sh, st["q"], st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["table"], st["starts"], st["pos"],
                                  sel_idx=st["sel"], workspace=kept)
    return {"o": o, "lse": lse}


def _cache_outputs(st):
    return {n: st[n] for n in ("k8", "v8", "k_scale", "v_scale", "k_idx")}


def _fork_outputs(st, moves):
    return {"lens": st["lens"], "table": st["table"], "ring": st["ring"], "free": st["free"], "shares": st["shares"], "moves": moves, **_cache_outputs(st)}


def _compact_outputs(st, table, ring, free, shares, moves):
    return {"table": table, "ring": ring, "free": free, "shares": shares, "moves": moves, **_cache_outputs(st)}


# ---------------------------------------------------------------- the plain forms
def _inv_freq(c, dev):
    """Radians a position of each pair of features, in 64 bits.  With a factor, pairs that turn less than once over the 8,192
    tokens that the model was first trained on turn slower by it, those that turn four times or more keep their speed, and those between go from one to the other."""
    f = float(c["base"]) ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
    if c["factor"] == 1:
        return f
    keep = ((8192 * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
    return f * (keep + (1 - keep) / c["factor"])


def _gain(c):
    return 1.0 if c["factor"] == 1 else 0.1 * math.log(c["factor"]) + 1


def _positions(st, dev):
    c = st["case"]
    return st["pos"].double() if st["pos"] is not None else (torch.arange(c["T"], device=dev) % c["N"]).double()


def _plain_turn(x, cos, sin, c):
    """x [T, H, d]: pairs of the first `rot` features turned, the others as they are."""
    f, half = x.float(), c["rot"] // 2
    a, b = (f[..., 0:c["rot"]:2], f[..., 1:c["rot"]:2]) if c["inter"] else (f[..., :half], f[..., half:c["rot"]])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], dim=3).flatten(2) if c["inter"] else torch.cat([u, v], dim=2)
    return torch.cat([y.bfloat16(), x[..., c["rot"]:]], dim=2)


def _plain_rotary(st):
    c, dev = st["case"], st["q"].device
    turn = _positions(st, dev)[:, None] * _inv_freq(c, dev)
    cos, sin = (_gain(c) * turn.cos()).float()[:, None], (_gain(c) * turn.sin()).float()[:, None]
    if c["bwd"]:
        sin = -sin
    return {"q": _plain_turn(st["q"], cos, sin, c), "k": _plain_turn(st["k"], cos, sin, c)}


def _plain_copy(st, a, b, rows):
    """The first `rows` tokens of pages a into pages b, with their scales."""
    keep = torch.arange(PAGE, device=a.device) < rows[:, None]
    for n in ("k8", "v8"):
        x = st[n].view(torch.uint8)
        x[b] = torch.where(keep[:, None, :, None], x[a], x[b])
    for n in ("k_scale", "v_scale"):
        st[n][b] = st[n][a]
    st["k_idx"][b] = torch.where(keep[:, :, None], st["k_idx"][a], st["k_idx"][b])


def _plain_fork(st):
    table, ring, shares, n_pages = st["table"], st["ring"], st["shares"], st["n_pages"]
    dev, (R, nb) = table.device, table.shape
    src, lens = st["src"].long(), st["lens"].long()
    head, count = st["free"][0].long(), st["free"][1].long()
    slot, col = torch.arange(R, device=dev), torch.arange(nb, device=dev)
    ended = src != slot
    goes_on = ended & (src >= 0)
    s = src.clamp(min=0)
    n = torch.where(goes_on, lens[s], torch.where(ended, 0, lens))
    full, rest = n // PAGE, n % PAGE
    theirs = table[s]
    gone = ended[:, None] & (col < _pages_of(lens)[:, None])
    kept = goes_on[:, None] & (col < full[:, None])
    # references to each page, less one
    out_of, into = torch.where(gone, table, n_pages).long(), torch.where(kept, theirs, n_pages).long()
    wide = torch.cat([shares, shares.new_zeros(1)]).long()
    wide.scatter_add_(0, out_of.reshape(-1), torch.full((R * nb,), -1, device=dev))
    wide.scatter_add_(0, into.reshape(-1), torch.ones(R * nb, dtype=torch.int64, device=dev))
    # pages without any go behind the free ones, in the order of slots and blocks
    flat = torch.arange(R * nb, device=dev)
    first = torch.full((n_pages + 1,), R * nb, device=dev).scatter_reduce_(0, out_of.reshape(-1), flat, "amin")
    free = gone & (wide[out_of] < 0) & (first[out_of] == flat.reshape(R, nb))
    order = free.reshape(-1).cumsum(0) - 1
    at = torch.where(free.reshape(-1), (head + count + order) % n_pages, n_pages)
    ring_out = torch.cat([ring, ring.new_zeros(1)]).scatter_(0, at, table.reshape(-1))[:-1]
    # a page of its own for a request whose tokens end inside one
    take = goes_on & (rest > 0)
    page = ring[(head + take.cumsum(0) - take.long()) % n_pages]
    moves = torch.stack([theirs.gather(1, full.clamp(max=nb - 1)[:, None])[:, 0].long(), page.long(), rest], dim=1)
    moves = torch.where(take[:, None], moves, torch.tensor([-1, -1, 0], device=dev))
    st["free"].copy_(torch.stack([(head + take.sum()) % n_pages, count - take.sum() + free.sum()]))
    shares.copy_(wide[:-1].clamp(min=0))
    st["lens"].copy_(n)
    table.copy_(torch.where(kept, theirs, torch.where(take[:, None] & (col == full[:, None]), page[:, None], table)))
    ring.copy_(ring_out)
    m = moves[st["moved"]]
    _plain_copy(st, m[:, 0], m[:, 1], m[:, 2])
    return _fork_outputs(st, moves.int())


def _plain_compact(st):
    table, n_pages, m = st["table"], st["n_pages"], st["n_moves"]
    dev = table.device
    mine = torch.arange(table.shape[1], device=dev) < _pages_of(st["lens"].long())[:, None]
    at = torch.where(mine, table, n_pages).long()
    used = torch.zeros(n_pages + 1, dtype=torch.bool, device=dev)
    used[at.reshape(-1)] = True
    used = used[:-1]
    u, page = used.sum(), torch.arange(n_pages, device=dev)
    a = torch.where(used & (page >= u), page, n_pages).sort().values[:m]
    b = torch.where(~used & (page < u), page, n_pages).sort().values[:m]
    to = torch.arange(n_pages + 1, device=dev)
    to[a] = b
    shares = torch.where(used, st["shares"], 0)
    shares[b] = shares[a]
    shares.masked_fill_(page >= u, 0)
    ring = torch.where(page < n_pages - u, u + page, -1)
    moves = torch.tensor([-1, -1, 0], device=dev).repeat(max(1, n_pages // 2), 1)
    moves[:m] = torch.stack([a, b, torch.full_like(a, PAGE)], dim=1)
    _plain_copy(st, a, b, moves[:m, 2])
    return _compact_outputs(st, torch.where(mine, to[at], table).int(), ring.int(), torch.stack([0 * u, n_pages - u]).int(), shares, moves.int())


def _padded(st, x):
    """x [T, ...] as [R, q, ...], and the place of each row in it."""
    i = torch.arange(st["case"]["q"], device=x.device)
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
    s = torch.matmul(qp, k.transpose(2, 3)).div_(math.sqrt(d))
    del k
    late = torch.arange(nb * PAGE, device=pos.device) > pp[:, :, None]
    s.view(R, Hkv, q, G, -1).masked_fill_(late[:, None, :, None], -math.inf)
    m = s.amax(3, keepdim=True)
    e = s.sub_(m).exp_()
    z = e.sum(3, keepdim=True)
    o = torch.matmul(e, pages(st["v8"], st["v_scale"], page, h).reshape(R, Hkv, nb * PAGE, d)) / z
    back = lambda x: x.reshape(R, Hkv, q, G, -1).permute(0, 2, 1, 3, 4)[req, i].reshape(T, Hq, -1)  # noqa: E731
    return {"o": back(o).bfloat16(), "lse": back(m + z.log())[..., 0].contiguous()}


def run(state):
    if own:
        return _run_own(state)
    return {"rotary": _plain_rotary, "fork": _plain_fork, "compact": _plain_compact, "chunk_scores": _plain_scores,
            "chunk_attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    H = c["Hq"] + c["Hkv"]
    token = 2 * c["Hkv"] * c["d"] + 2 * c["d_idx"]  # of the cache, without the scales
    if c["op"] == "rotary":
        return {"bytes": 4 * c["T"] * H * c["d"] + 4 * c["T"] * (not c["N"]), "flops": 3 * c["T"] * H * c["rot"]}
    if c["op"] == "fork":
        src, (lens, common) = _fork_src(c, np.random.RandomState(c["R"] * 7 + c["ctx"])), _fork_lens(c)
        ended = src != np.arange(c["R"])
        new = np.where(ended & (src >= 0), lens, 0)
        copied = (new % PAGE).sum() * token + 8 * c["Hkv"] * (new % PAGE > 0).sum()
        # a table entry read and one written for each page of a fork, one read for each page that is let go
        return {"bytes": int(2 * copied + 4 * (2 * _pages_of(new).sum() + _pages_of(lens)[ended].sum() + 4 * c["R"])), "flops": 0}
    if c["op"] == "compact":
        lens = _compact_lens(c)
        held = _pages_of(lens)
        used = int(held.sum() - int(held[:4].min()) // 2 * max(0, min(4, c["R"]) - 1))
        n_pages = int(used / c["live"]) + 3
        moved = used * (n_pages - used) / n_pages  # as many as pages lie at random
        return {"bytes": int(2 * moved * (PAGE * token + 8 * c["Hkv"]) + 8 * held.sum() + 8 * n_pages), "flops": 0}
    lens, q = _lens(c)
    T, (starts, req, pos) = int(q.sum()), _rows(lens, q)
    if c["op"] == "chunk_scores":
        return {"bytes": int(lens.sum()) * c["d_idx"] * 2 + T * c["Hkv"] * (c["d_idx"] * 2 + 4 * int(_pages_of(c["ctx"]))),
                "flops": 2 * int((pos + 1).sum()) * c["Hkv"] * c["d_idx"]}
    if c["sparse"]:
        nblk = np.minimum(pos // PAGE + 1, c["k"])
        seen = (nblk - 1) * PAGE + pos % PAGE + 1
    else:
        seen = pos + 1
    kv = int(np.minimum(np.bincount(req, seen), lens).sum())  # a request's rows share what they read
    return {"bytes": kv * c["Hkv"] * c["d"] * 2 + T * c["Hq"] * (c["d"] * 4 + 4), "flops": 4 * int(seen.sum()) * c["Hq"] * c["d"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotary(c, st):
    j = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(-2 * j / c["rot"] * math.log(c["base"]))
    gain = 1.0
    if c["factor"] != 1:
        turns = 8192 * f / (2 * math.pi)
        mix = torch.where(turns <= 1, 0.0, torch.where(turns >= 4, 1.0, (turns - 1) / 3))
        f = (1 - mix) * f / c["factor"] + mix * f
        gain = 0.1 * math.log(c["factor"]) + 1
    t = torch.arange(c["T"], device="cuda")
    pos = st["pos"].double() if st["pos"] is not None else (t - t // c["N"] * c["N"]).double()
    w = torch.polar(torch.full((c["T"], 1, c["rot"] // 2), gain, dtype=torch.float64, device="cuda"), (pos[:, None] * f)[:, None])
    w = w.conj() if c["bwd"] else w
    res = {}
    for n in ("q", "k"):
        x = st[n].double()
        y, r = x.clone(), c["rot"]
        z = w * (torch.complex(x[..., 0:r:2], x[..., 1:r:2]) if c["inter"] else torch.complex(x[..., :r // 2], x[..., r // 2:r]))
        if c["inter"]:
            y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
        else:
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        res[n] = y
    return res


def _exact_scores(c, st, lens, q):
    table, nb, t0 = st["table"].long(), st["table"].shape[1], 0
    res = torch.full((st["T"], c["Hkv"], nb), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        pos = st["pos"][t0:t0 + q[r]].long()
        for b in range(int(_pages_of(lens[r]))):
            k = st["k_idx"][table[r, b]].double()
            s = torch.einsum("tgd,nd->tgn", st["q_idx"][t0:t0 + q[r]].double(), k) * c["d_idx"] ** -0.5
            unseen = b * PAGE + torch.arange(PAGE, device="cuda") > pos[:, None]
            res[t0:t0 + q[r], :, b] = torch.where(unseen[:, None], -math.inf, s).amax(2)
        t0 += int(q[r])
    return res


def _exact_attn(c, st, lens, q):
    G, d, table = c["Hq"] // c["Hkv"], c["d"], st["table"].long()
    o = torch.zeros(st["T"], c["Hkv"], G, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["T"], c["Hkv"], G, dtype=torch.float64, device="cuda")
    x = st["q"].double().reshape(st["T"], c["Hkv"], G, d)

    def rows(codes, scales, page, g):
        return (codes.view(torch.uint8)[page, g].view(torch.float8_e4m3fn).double() * scales[page, g].double()[..., None, None]).flatten(-3, -2)

    t0 = 0
    for r in range(c["R"]):
        n, end = int(lens[r]), t0 + int(q[r])
        if st["sel"] is None:
            page = table[r, :int(_pages_of(n))]
            for g in range(c["Hkv"]):
                k, v = rows(st["k8"], st["k_scale"], page, g)[:n], rows(st["v8"], st["v_scale"], page, g)[:n]
                step = max(1, (1 << 28) // (G * n))
                for a in range(t0, end, step):
                    b = min(end, a + step)
                    s = torch.einsum("thd,nd->thn", x[a:b, g], k) / math.sqrt(d)
                    s.masked_fill_((torch.arange(n, device="cuda") > st["pos"][a:b, None])[:, None], -math.inf)
                    lse[a:b, g] = torch.logsumexp(s, 2)
                    o[a:b, g] = torch.einsum("thn,nd->thd", torch.exp(s - lse[a:b, g, :, None]), v)
        else:
            g = torch.arange(c["Hkv"], device="cuda")[:, None]
            for t in range(t0, end):
                block = st["sel"][t].long()
                seen = ((block[..., None] * PAGE + torch.arange(PAGE, device="cuda") <= st["pos"][t]) & (block >= 0)[..., None]).flatten(1)
                page = table[r, block.clamp(min=0)].clamp(min=0)
                s = torch.einsum("ghd,gnd->ghn", x[t], rows(st["k8"], st["k_scale"], page, g)) / math.sqrt(d)
                s = torch.where(seen[:, None], s, -math.inf)
                lse[t] = torch.logsumexp(s, 2)
                o[t] = torch.einsum("ghn,gnd->ghd", torch.exp(s - lse[t][..., None]), rows(st["v8"], st["v_scale"], page, g))
        t0 = end
    return {"o": o.reshape(st["T"], c["Hq"], d), "lse": lse.reshape(st["T"], c["Hq"])}


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    st = prepare(case, seed)
    if c["op"] == "rotary":
        return _exact_rotary(c, st)
    lens, q = _lens(c)
    order = np.random.RandomState(seed).permutation(c["R"])
    return (_exact_scores if c["op"] == "chunk_scores" else _exact_attn)(c, st, lens[order], q[order])
