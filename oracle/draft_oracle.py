"""Plain numpy float64 forms of the operators of drafted tokens (test infrastructure).

Written from the definitions in ``include/qdq.h``; shares no code with the GPU path.
Only what the cache's codes are rounded by is computed in float32, because its definition is.
"""
from __future__ import annotations

import numpy as np

from .decode_oracle import BLOCK


def depths(parents):
    """Depth of each node, -1 where a node or one of its ancestors has no valid parent."""
    d = []
    for i, p in enumerate(parents):
        if p == -1:
            d.append(0)
        elif 0 <= p < i and d[p] >= 0:
            d.append(d[p] + 1)
        else:
            d.append(-1)
    return np.array(d)


def line(parents, i):
    """Node i and its ancestors."""
    out = [i]
    while parents[out[-1]] != -1:
        out.append(parents[out[-1]])
    return out[::-1]


def norm_turn(x, weight, eps, pos, freqs, interleaved):
    """x (n, heads, dim) of tokens at pos (n,): (result, sum of magnitudes of a pair's elements) in float64."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    y, mag = x.copy(), np.abs(x)
    if freqs is not None and len(freqs):
        r = len(freqs)
        a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
        t = (np.asarray(pos, np.float64)[:, None] * freqs.astype(np.float64))[:, None]
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
        mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def tree_attention(q, k, v, parents, scale, softcap=0.0, window=0, slopes=None):
    """One sequence's tree: q (n, heads, dim), its keys and values the last n of k and v (len, kv heads, dim).

    Returns what ``decode_oracle.attention`` does."""
    n, H, D = q.shape
    L, Hk, _ = k.shape
    base = L - n
    dep = depths(parents)
    out, av = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, mag, z = np.full((n, H), -np.inf), np.zeros((n, H)), np.zeros((n, H))
    big = np.abs(v).max(-1)
    big = np.pad(big, ((0, -L % BLOCK), (0, 0))).reshape(-1, BLOCK, Hk).max(1).repeat(BLOCK, 0)[:L]
    for i in range(n):
        if dep[i] < 0:
            out[i] = lse[i] = np.nan
            continue
        seen = [j for j in list(range(max(base, 0))) + [base + x for x in line(parents, i)] if j >= 0]
        at = np.array([j if j < base else base + dep[j - base] for j in seen], np.int64)
        far = base + dep[i] - at
        if window > 0:
            seen, far = [j for j, f in zip(seen, far) if f < window], far[far < window]
        if not len(seen):
            continue
        for h in range(H):
            kk, vv = k[seen, h * Hk // H], v[seen, h * Hk // H]
            x = scale * (kk @ q[i, h])
            mag[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x - slopes[h] * far
                mag[i, h] += np.abs(slopes[h] * far).max()
            m = x.max()
            p = np.exp(x - m)
            lse[i, h] = m + np.log(p.sum())
            p = p / p.sum()
            out[i, h] = p @ vv
            av[i, h] = p @ np.abs(vv)
            z[i, h] = (p * big[seen, h * Hk // H]).max()
    return out, lse, av, mag, z


def verify(logits, tokens, parents, uniform, draft, temperature):
    """One sequence: (path, next token, margin).  margin: how near any comparison was to its border, as a
    probability (a choice with a smaller margin than p is off by may go either way)."""
    n, V = logits.shape
    lo, hi = 0.0, float(np.float32(1) - np.float32(2.0 ** -24))
    u = None if uniform is None else np.clip(uniform.astype(np.float64), lo, hi)
    path, cur, margin = [0], 0, np.inf
    while True:
        x = logits[cur].astype(np.float64)
        if np.isnan(x).any() or not np.isfinite(x.max()):
            return path, -1, margin
        kids = [i for i in range(1, n) if parents[i] == cur]
        if temperature == 0:
            best = int(np.argmax(x))
            kids = [i for i in kids if tokens[i] == best][:1]
            if not kids:
                return path, best, margin
            cur = kids[0]
            path.append(cur)
            continue
        w = np.exp((x - x.max()) / temperature)
        w /= w.sum()
        went = None
        for i in kids:
            t = tokens[i]
            if not 0 <= t < V:
                continue
            if draft is None:
                q = np.zeros(V)
                q[t] = 1
                if w[t] == 0:
                    continue
            else:
                q = draft[cur].astype(np.float64)
            margin = min(margin, abs(u[i] * q[t] - w[t]) / max(q[t], 1e-30))
            if u[i] * q[t] < w[t]:
                went = i
                break
            rest = np.maximum(w - q, 0)
            if rest.sum() > 0:
                w = rest / rest.sum()
        if went is None:
            c = np.cumsum(w)
            t = u[0] * c[-1]
            at = min(int(np.searchsorted(c, t, side="right")), int(np.nonzero(w)[0][-1]))
            margin = min(margin, c[at] - t if at < np.nonzero(w)[0][-1] else np.inf, t - (c[at] - w[at]) if w[:at].any() else np.inf)
            return path, at, margin
        cur = went
        path.append(cur)


def keep(cache, table, kv_len, cu, path, accepted):
    """The definition of qdq_kv_keep on a ``decode_oracle.Cache``, block by block."""
    f = np.float32
    with np.errstate(all="ignore"):
        for s in range(len(kv_len)):
            n = cu[s + 1] - cu[s]
            old = kv_len[s] - n
            if n <= 0 or old < 0 or accepted[s] < 0:
                continue
            kept, last = [], -1
            for x in path[s][:accepted[s] + 1]:
                if not last < x < n:
                    break
                kept.append(x)
                last = x
            for p0 in range(old // BLOCK * BLOCK, old + len(kept), BLOCK):
                src = [p if p < old else old + kept[p - old] for p in range(p0, min(p0 + BLOCK, old + len(kept)))]
                if src == list(range(p0, p0 + len(src))):
                    continue

                def page(j):
                    slot = j // cache.page
                    ok = slot < table.shape[1] and 0 <= table[s, slot] < cache.raw.shape[0]
                    return int(table[s, slot]) if ok else None

                to = page(p0)
                for which in range(2):
                    for h in range(cache.n_kv):
                        codes, scales = [], []
                        for j in src:
                            pid, t = page(j), j % cache.page
                            codes.append(np.zeros(cache.dim, np.int8) if pid is None else cache._codes(pid, h, which)[t].copy())
                            scales.append(f("nan") if pid is None else cache._scales(pid, h, which)[t // BLOCK])
                        scales = np.array(scales, f)
                        top = f("nan") if np.isnan(scales).any() else scales.max()
                        if to is None:
                            continue
                        for i, (c, sc) in enumerate(zip(codes, scales)):
                            ratio = sc / top if top > 0 else f(0)
                            if src[i] == p0 + i and ratio == 1:
                                continue
                            cache._codes(to, h, which)[p0 % cache.page + i] = np.rint(c.astype(f) * ratio).astype(np.int8)
                        cache._scales(to, h, which)[p0 % cache.page // BLOCK] = top
