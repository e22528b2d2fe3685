"""Plain numpy float64 forms of the decode-step operators (test infrastructure).

Written from the definitions in ``include/qdq.h``; shares no code with the GPU path.
Only the cache's quantisation is computed in float32, because its definition is: every
quotient, product and maximum there is one float32 operation.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16


def record_bytes(page, dim):
    return (2 * page * dim + 8 * (page // BLOCK) + 127) // 128 * 128


def rms_norm(x, residual, weight, eps):
    """(y, h) in float64."""
    h = x.astype(np.float64)
    if residual is not None:
        h = h + residual.astype(np.float64)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight.astype(np.float64)
    return y, h


class Cache:
    """The pool as numpy bytes, read and written token by token."""

    def __init__(self, raw, page, n_kv, dim):
        self.page, self.n_kv, self.dim = page, n_kv, dim
        self.rec = record_bytes(page, dim)
        self.raw = raw.reshape(-1, n_kv, self.rec)

    def _codes(self, pid, h, which):
        a = which * self.page * self.dim
        return self.raw[pid, h, a:a + self.page * self.dim].view(np.int8).reshape(self.page, self.dim)

    def _scales(self, pid, h, which):
        nb = self.page // BLOCK
        a = 2 * self.page * self.dim + 4 * nb * which
        return self.raw[pid, h, a:a + 4 * nb].view(np.float32)

    def append(self, table, kv_len, cu, k, v):
        """The definition of qdq_kv_append, block by block."""
        f = np.float32
        with np.errstate(all="ignore"):
            for s in range(len(kv_len)):
                n = cu[s + 1] - cu[s]
                old = kv_len[s] - n
                if n <= 0 or old < 0:
                    continue
                for b in range(old // BLOCK, -(-kv_len[s] // BLOCK)):
                    p0 = b * BLOCK
                    slot = p0 // self.page
                    if slot >= table.shape[1] or not 0 <= table[s, slot] < self.raw.shape[0]:
                        continue
                    pid, t0 = table[s, slot], p0 % self.page
                    lo, hi = max(old, p0), min(kv_len[s], p0 + BLOCK)
                    for which, x in ((0, k), (1, v)):
                        for h in range(self.n_kv):
                            new = x[cu[s] + lo - old:cu[s] + hi - old, h].astype(f)
                            codes = self._codes(pid, h, which)[t0:t0 + BLOCK]
                            sc = self._scales(pid, h, which)
                            held = lo - p0
                            s_old = sc[t0 // BLOCK] if held else f(0)
                            m = np.abs(new).max()
                            s_new = f(m) / f(127)
                            if s_new < np.finfo(f).tiny:
                                s_new = f(0)
                            if not np.isfinite(m):
                                s_new = f("nan")
                            both = f("nan") if np.isnan(s_old) or np.isnan(s_new) else max(s_old, s_new)
                            inv = f(1) / both if both > 0 else f(0)
                            if held and not both == s_old:
                                again = s_old / both if both > 0 else f(0)
                                codes[:held] = np.rint(codes[:held].astype(f) * again).astype(np.int8)
                            c = np.rint(np.clip(new * inv, f(-127), f(127)))
                            codes[held:hi - p0] = np.where(np.isnan(c), 0, c).astype(np.int8)
                            sc[t0 // BLOCK] = both

    def read(self, table, s, start, n):
        """Values of n tokens of sequence s: two (n, heads, dim) float64 arrays; NaN where there is no page."""
        out = np.full((2, n, self.n_kv, self.dim), np.nan)
        with np.errstate(all="ignore"):
            for j in range(start, start + n):
                slot = j // self.page
                if slot >= table.shape[1] or not 0 <= table[s, slot] < self.raw.shape[0]:
                    continue
                for which in range(2):
                    for h in range(self.n_kv):
                        t = j % self.page
                        c = self._codes(table[s, slot], h, which)[t].astype(np.float32)
                        out[which, j - start, h] = c * self._scales(table[s, slot], h, which)[t // BLOCK]
        return out[0], out[1]


def attention(q, k, v, pos, scale, softcap=0.0, window=0, slopes=None):
    """One sequence.  q (n, heads, dim); k, v (len, kv heads, dim); pos (n,).

    Returns out (n, heads, dim), lse (n, heads), and for the error bounds abs_v = sum p |v| per
    output, a = the largest scale * sum |q||k| + |bias| over a row's visible tokens, and the largest
    p * max |v| of them (at least the largest p times 127 times the value scale, up to the block's largest code)."""
    n, H, D = q.shape
    L, Hk, _ = k.shape
    out = np.zeros((n, H, D))
    av = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    mag = np.zeros((n, H))
    z = np.zeros((n, H))
    big = np.abs(v).max(-1)
    pad = -L % BLOCK
    big = np.pad(big, ((0, pad), (0, 0))).reshape(-1, BLOCK, Hk).max(1).repeat(BLOCK, 0)[:L]  # a block's largest value: about 127 scales
    for i in range(n):
        lo = max(0, pos[i] - window + 1) if window > 0 else 0
        hi = min(L, pos[i] + 1)
        if hi <= lo:
            continue
        for h in range(H):
            kk, vv = k[lo:hi, h * Hk // H], v[lo:hi, h * Hk // H]
            x = scale * (kk @ q[i, h])
            mag[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                far = pos[i] - np.arange(lo, hi)
                x = x - slopes[h] * far
                mag[i, h] += np.abs(slopes[h] * far).max()
            m = x.max()
            p = np.exp(x - m)
            lse[i, h] = m + np.log(p.sum())
            p = p / p.sum()
            out[i, h] = p @ vv
            av[i, h] = p @ np.abs(vv)
            z[i, h] = (p * big[lo:hi, h * Hk // H]).max()
    return out, lse, av, mag, z


def logprobs(x, tokens, k):
    """(logprob, entropy, top_index, top_logprob) of rows of logits, float64."""
    x64 = x.astype(np.float64)
    R, n = x.shape
    lp = np.full(R, np.nan)
    ent = np.full(R, np.nan)
    ti = np.zeros((R, k), np.int64)
    tl = np.full((R, k), np.nan)
    for r in range(R):
        row = x64[r]
        nan = np.isnan(row)
        # NaN first, then larger first, equal by smaller index
        order = np.lexsort((np.arange(n), np.where(nan, 0.0, -row), ~nan))[:k]
        ti[r] = order
        m = row.max() if not nan.any() else np.nan
        if not np.isfinite(m):
            continue
        e = np.exp(row - m)
        lse = m + np.log(e.sum())
        p = e / e.sum()
        ent[r] = -(p[p > 0] * (row[p > 0] - lse)).sum()
        if 0 <= tokens[r] < n:
            lp[r] = row[tokens[r]] - lse
        tl[r] = row[order] - lse
    return lp, ent, ti, tl
