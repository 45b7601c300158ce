"""The page-sharing, compaction, rotary and chunk operators from their
definitions, in numpy and 64 bits, and the error bounds their tests use."""
from __future__ import annotations

import numpy as np

from paged_ref import PAGE, e4m3_decode


def pages_of(n):
    return -(-int(n) // PAGE)


def fork(src, lens, table, ring, free, shares, fork_lens=None, held=None):
    """(lens, held, table, ring, free, shares, moves), one page after another."""
    R, n_pages = len(src), len(ring)
    had = [pages_of(n) for n in lens] if held is None else [int(h) for h in held]
    old, ring0 = table.copy(), ring.copy()
    lens, had_out, table, ring, shares = lens.copy(), list(had), table.copy(), ring.copy(), shares.copy()
    old_lens = lens.copy()
    refs = {}
    for p in range(n_pages):
        refs[p] = int(shares[p]) + 1
    head, count = (int(x) for x in free)
    dropped, taken = [], 0
    moves = np.tile(np.array([-1, -1, 0], np.int32), (R, 1))
    for r in range(R):
        if src[r] == r:
            continue
        for b in range(had[r]):
            refs[int(old[r, b])] -= 1
            dropped.append(int(old[r, b]))
    fresh = []
    for r in range(R):
        s = int(src[r])
        if s == r:
            continue
        n = 0 if s < 0 else int(old_lens[s] if fork_lens is None else fork_lens[r])
        for b in range(n // PAGE):
            table[r, b] = old[s, b]
            refs[int(old[s, b])] += 1
        if n % PAGE:
            page = int(ring0[(head + taken) % n_pages])
            taken += 1
            fresh.append(page)
            moves[r] = old[s, n // PAGE], page, n % PAGE
            table[r, n // PAGE] = page
        lens[r], had_out[r] = n, pages_of(n)
    back, seen = 0, set()
    for p in dropped:
        if refs[p] == 0 and p not in seen:
            seen.add(p)
            ring[(head + count + back) % n_pages] = p
            back += 1
    for p in range(n_pages):
        shares[p] = max(refs[p] - 1, 0)
    return (lens, np.array(had_out, np.int32), table, ring, np.array([(head + taken) % n_pages, count - taken + back], np.int32), shares, moves)


def compact(lens, table, n_pages, shares=None, held=None):
    """(table, ring, free, shares, moves)."""
    had = [pages_of(n) for n in lens] if held is None else held
    used = sorted({int(table[r, b]) for r in range(len(lens)) for b in range(had[r])})
    u = len(used)
    movers, inside = [p for p in used if p >= u], set(used)
    holes = [p for p in range(u) if p not in inside]
    to = dict(zip(movers, holes))
    out = table.copy()
    for r in range(len(lens)):
        for b in range(had[r]):
            out[r, b] = to.get(int(table[r, b]), int(table[r, b]))
    sh = None
    if shares is not None:
        sh = np.zeros(n_pages, np.int32)
        for p in used:
            sh[to.get(p, p)] = shares[p]
    ring = np.array(list(range(u, n_pages)) + [-1] * u, np.int32)
    moves = np.tile(np.array([-1, -1, 0], np.int32), (max(1, n_pages // 2), 1))
    for i, (a, b) in enumerate(to.items()):
        moves[i] = a, b, PAGE
    return out, ring, np.array([0, n_pages - u], np.int32), sh, moves


def rotary(x, pos, freqs, d_rot, interleaved, scale, backward):
    """x [T, H, d] float64 turned at pos [T]; freqs [d_rot/2] radians a position.  Rows of a negative position are NaN."""
    y = x.copy()
    i = np.arange(d_rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + d_rot // 2)
    w = pos[:, None] * freqs[None]
    c, s = (scale * f(w)[:, None] for f in (np.cos, np.sin))
    if backward:
        s = -s
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    y[pos < 0] = np.nan
    return y


def attn(q, k8, v8, ks, vs, table, req, pos, sel, scale):
    """o [T, Hq, d], lse [T, Hq] and the bounds of their errors.

    By the kernel's own arithmetic (d features, n visible tokens):
      scores  products of 8-bit significands are exact in fp32; sums of d of them, each step off by at most 2^-23
              of the sum of magnitudes: ds <= d 2^-23 sum|q k| scale, and a few roundings of the scaled score, s 2^-21
      exp     p relative 2 max ds + 2^-21 (exp2's error, the running maximum's factors)
      p       rounded to bf16, 2^-8 relative; to 2^-133 below (its least subnormal's half, over a reference of at least
              a tile's largest less 2^-9 of it)
      sums    n 2^-23 relative, as the tensor cores may cut instead of round
      o       rounded once to bf16, 2^-8 relative."""
    T, Hq, d = q.shape
    H = k8.shape[1]
    G = Hq // H
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    do, dl = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    kept = {}
    for t in range(T):
        if req[t] < 0 or pos[t] < 0:
            continue
        for h in range(H):
            blocks = np.arange(pos[t] // PAGE + 1) if sel is None else sel[t, h][sel[t, h] >= 0]
            if len(blocks) == 0:
                continue
            key = (int(req[t]), h, tuple(blocks))
            if key not in kept:
                pages = table[req[t], blocks]
                kept[key] = [(e4m3_decode(c[pages, h]) * s[pages, h].astype(np.float64)[:, None, None]).reshape(-1, d) for c, s in ((k8, ks), (v8, vs))]
            seen = ((blocks[:, None] * PAGE + np.arange(PAGE)) <= pos[t]).reshape(-1)
            K, V = (x[seen] for x in kept[key])
            n, x = len(K), slice(h * G, (h + 1) * G)
            s = q[t, x] @ K.T * scale
            ds = ((np.abs(q[t, x]) @ np.abs(K).T) * (d * 2.0 ** -23) * scale).max(1) + 2.0 ** -21 * np.abs(s).max(1)
            m = s.max(1)
            e = np.exp(s - m[:, None])
            z = e.sum(1)
            p = e / z[:, None]
            o[t, x], lse[t, x] = p @ V, m + np.log(z)
            rel = 2 * ds + 2.0 ** -8 + 2.0 ** -20 + 2 * n * 2.0 ** -23
            do[t, x] = rel[:, None] * (p @ np.abs(V)) + 2.0 ** -8 * np.abs(o[t, x]) + 1e-30
            dl[t, x] = ds + n * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(lse[t, x]) + np.abs(m))
    return o, lse, do, dl
