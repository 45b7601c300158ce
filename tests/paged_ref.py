"""The paged-cache operators from their definitions, in numpy and 64 bits, and
the error bounds their tests use."""
from __future__ import annotations

import numpy as np

PAGE = 128

# ------------------------------------------------------------------ e4m3
_POS = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(0x7F)])


def e4m3_decode(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.int64)
    v = np.where((c & 0x7F) == 0x7F, np.nan, _POS[np.minimum(c & 0x7F, 0x7E)])
    return np.where(c & 0x80, -v, v)


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest code, ties to the even one; |x| <= 448 or NaN."""
    a = np.abs(x)
    up = np.minimum(np.searchsorted(_POS, a), 0x7E)
    dn = np.maximum(up - 1, 0)
    du, dd = _POS[up] - a, a - _POS[dn]
    code = np.where(du < dd, up, np.where(dd < du, dn, np.where(up % 2 == 0, up, dn)))
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def scale_of(rows: np.ndarray) -> float:
    a = np.abs(rows[np.isfinite(rows)])
    amax = a.max() if a.size else 0.0
    if amax == 0:
        return 2.0 ** -112
    e = int(np.ceil(np.log2(amax / 448)))
    while 448 * 2.0 ** (e - 1) >= amax:
        e -= 1
    while 448 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** max(e, -112)


# ------------------------------------------------------------------ the operators
def plan(new, lens, table, ring, free, ended, T):
    """(table, ring, lens, free, q_starts, row_req, row_pos, slots, segs), one request after another."""
    R, n_pages = len(lens), len(ring)
    table, ring0, ring = table.copy(), ring, ring.copy()
    head, count = (int(x) for x in free)
    pages = lambda n: (n + PAGE - 1) // PAGE
    out_lens, starts, req, pos, slots, segs = [], [0], [], [], [], []
    back = taken = 0
    old = [0 if ended is not None and ended[r] else int(lens[r]) for r in range(R)]
    for r in range(R):
        if ended is not None and ended[r]:
            for j in range(pages(int(lens[r]))):
                ring[(head + count + back) % n_pages] = table[r, j]
                back += 1
    for r in range(R):
        n = int(new[r])
        for j in range(pages(old[r]), pages(old[r] + n)):
            table[r, j] = ring0[(head + taken) % n_pages]
            taken += 1
        for i in range(n):
            at = old[r] + i
            if i == 0 or at % PAGE == 0:
                segs.append(len(req))
            req.append(r)
            pos.append(at)
            slots.append(int(table[r, at // PAGE]) * PAGE + at % PAGE)
        out_lens.append(old[r] + n)
        starts.append(len(req))
    S = min(T, 2 * R + T // PAGE)
    pad = lambda x: np.array(x + [-1] * (T - len(x)), dtype=np.int32)
    segs = np.array(segs + [len(req)] * (S + 1 - len(segs)), dtype=np.int32)
    return (table, ring, np.array(out_lens, np.int32), np.array([(head + taken) % n_pages, count - taken + back], np.int32),
            np.array(starts, np.int32), pad(req), pad(pos), pad(slots), segs)


def append(new, slots, segs, codes, scales):
    """In place: new [T, H, d] into codes [n_pages, H, 128, d] (uint8) and scales [n_pages, H]."""
    for a, b in zip(segs[:-1], segs[1:]):
        if b <= a or slots[a] < 0:
            continue
        page, off = divmod(int(slots[a]), PAGE)
        for h in range(new.shape[1]):
            x = np.where(np.isfinite(new[a:b, h]), new[a:b, h], np.nan)
            s = scale_of(new[a:b, h])
            if off:
                had = float(scales[page, h])
                s = max(s, had)
                if s > had:
                    codes[page, h, :off] = e4m3_encode(e4m3_decode(codes[page, h, :off]) * had / s)
            codes[page, h, off:off + b - a] = e4m3_encode(x / s)
            scales[page, h] = s


def block_scores(q, k, table, req, pos, scale):
    """([T, H, nb] float64, the sums of |q k| * scale that bound its rounding)."""
    T, H, _ = q.shape
    nb = table.shape[1]
    out, mag = np.full((T, H, nb), -np.inf), np.zeros((T, H, nb))
    for t in range(T):
        if req[t] < 0:
            continue
        for c in range(min(nb, pos[t] // PAGE + 1)):
            rows = k[table[req[t], c], :max(0, min(PAGE, pos[t] - c * PAGE + 1))]
            out[t, :, c] = (q[t] @ rows.T).max(1) * scale
            mag[t, :, c] = (np.abs(q[t]) @ np.abs(rows).T).max(1) * scale
    return out, mag


def topk(scores, pos, k):
    T, H, _ = scores.shape
    out = np.full((T, H, k), -1, np.int32)
    for t in range(T):
        if pos[t] < 0:
            continue
        c0 = int(pos[t]) // PAGE
        for h in range(H):
            s = np.where(np.isnan(scores[t, h, :c0]), -np.inf, scores[t, h, :c0])
            best = np.lexsort((np.arange(c0), -s))[:k - 1]
            sel = np.sort(np.append(best, c0))
            out[t, h, :len(sel)] = sel
    return out


def attn(q, k8, v8, ks, vs, table, req, pos, sel, scale):
    """o [T, Hq, d], lse [T, Hq] and the bounds of their errors.

    Rounding in the kernel, by its own arithmetic (d features, n tokens):
      scores  fp32 sums of d products, each step off by at most 2^-23 of the
              sum of magnitudes, and the query's two-term split, off by 2^-23 of
              the row's largest scaled feature (448, at most twice its share):
              ds <= d 2^-23 sum|q k| scale + 2^-22 max|q| sum|k| scale
      exp     p relative 2 max ds + 2^-21 (exp2's error, the running maximum's factors)
      split   p relative 2^-8, or 2^-18 of the largest weight p vs (x = 16 p vs / reference is the sum of two e4m3
              terms, hi + lo / 16, off by 2^-8 x or half the least subnormal, 2^-10 / 16; the reference is at
              most the largest weight), on codes V / vs
      sums    n 2^-24 relative
      o       rounded once to bf16, 2^-8 relative."""
    T, Hq, d = q.shape
    H = k8.shape[1]
    G = Hq // H
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    do, dl = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for t in range(T):
        if req[t] < 0:
            continue
        for h in range(H):
            blocks = np.arange(pos[t] // PAGE + 1) if sel is None else sel[t, h][sel[t, h] >= 0]
            if len(blocks) == 0:
                continue
            pages = table[req[t], blocks]
            seen = ((blocks[:, None] * PAGE + np.arange(PAGE)) <= pos[t]).reshape(-1)
            K = (e4m3_decode(k8[pages, h]) * ks[pages, h].astype(np.float64)[:, None, None]).reshape(-1, d)[seen]
            V = (e4m3_decode(v8[pages, h]) * vs[pages, h].astype(np.float64)[:, None, None]).reshape(-1, d)[seen]
            sv = np.repeat(vs[pages, h].astype(np.float64), PAGE)[seen]
            n = len(K)
            for x in range(h * G, (h + 1) * G):
                s = K @ q[t, x] * scale
                ds = ((np.abs(K) @ np.abs(q[t, x])) * (d * 2.0 ** -23) + np.abs(K).sum(1) * np.abs(q[t, x]).max() * 2.0 ** -22) * scale
                ds = np.nanmax(ds) if not np.all(np.isnan(ds)) else np.nan
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                o[t, x], lse[t, x] = (e / z) @ V, m + np.log(z)
                rel = 2 * ds + 2.0 ** -8 + 2.0 ** -20 + 2 * n * 2.0 ** -24
                do[t, x] = rel * ((e / z) @ np.abs(V)) + 2.0 ** -18 * np.nanmax(e * sv) * np.abs(V / sv[:, None]).sum(0) / z + 2.0 ** -8 * np.abs(o[t, x]) + 1e-30
                dl[t, x] = ds + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(lse[t, x]) + abs(m))
    return o, lse, do, dl
