"""Drafted tokens next to borders: results that no other call and no rounding may change.

Bounds (u = 2^-24), beside those of test_gpu_drafts.py.  A row's sum of weights Z holds each chunk's likeliest token and the joins
of chunks as pairs of f32; the other tokens' weights are f32: an exponent h (in bits) is off by |h| 2^-23, which is |h| ln 2 2^-23
of the weight, exp2 by 2^-22, and a chunk's sum by 22 u: 2^-18 of what those tokens have, where |h| is at most 20.
* what rejected drafts without probabilities leave is summed from the tokens that are left wherever less than half of the last
  such sum remains, likely tokens as pairs, the others as above with |h| up to 42 (a draft that leaves less than 2^-24 is never
  rejected): 2 (22 u + 2^-22 + 42 ln 2 2^-23) < 2^-16 of itself; 2^-15 below.
* a child's p is a pair: its weight to 2^-30, Z as above.  Where all tokens but the likeliest of their chunks share less
  than 2^-9.9, p is within 2^-27.9 of itself, and so is p - b q of p + b q.
"""
import numpy as np
import pytest

from oracle import draft_oracle as dref
from test_gpu_decode_ops import _dt, _filled, _i32, _np, _t, attn_kernel  # noqa: F401
from test_gpu_drafts import _cu, _parents, _tree, _verify

pytestmark = pytest.mark.gpu


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nodes,heads,n_kv,dim,dtype,softcap,window,bias,wide", [
    (26, 32, 8, 128, "bf16", 0, 0, False, 60),   # 104 rows: the tensor cores' fourth warp has 8 of them and 24 of no node
    (13, 24, 8, 128, "f16", 0, 0, False, 60),
    (13, 24, 8, 64, "f32", 0, 900, False, 32),
    (20, 4, 4, 64, "f16", 0, 50, False, 16),     # 16 rows to a tile of the decode kernel, the second with 12 of no node
    (20, 4, 4, 128, "f32", 0, 50, True, 32),
    (21, 8, 4, 64, "bf16", 30.0, 40, True, 32),
    (37, 4, 2, 192, "bf16", 0, 70, False, 60),
])
def test_a_tree_does_not_depend_on_the_call_before(cuda_lib, nodes, heads, n_kv, dim, dtype, softcap, window, bias, wide):
    # Rows past a tree's last share warps with its rows, and these move their references together: with scores that grow by 2^6 to
    # 2^14 behind the first tile another call's tree, left in shared memory, would show in the rounding.
    import torch
    rng = np.random.default_rng(nodes + dim)
    seqs, page, most = 8, 64, 64
    lens = [2000 + 150 * s for s in range(seqs)]
    raw, table, _ = _filled(rng, lens, page, n_kv, dim)
    slopes = _t((2.0 ** -rng.uniform(1, 8, heads)).astype(np.float32)) if bias else None
    q = _t(wide * dim ** -0.5 * rng.standard_normal((seqs * most, heads, dim)).astype(np.float32), _dt(dtype))
    parents = [_parents(rng, nodes) for _ in lens]
    ws = cuda_lib.kv_attention_workspace(seqs, most, max(lens), heads, n_kv, dim)

    def run(n, par):
        return _tree(cuda_lib, raw, table, lens, [n] * seqs, q[:n * seqs], heads, n_kv, dim, page, par, softcap=softcap, window=window,
                     slopes=slopes, max_kv=max(lens), max_q=most, workspace=ws)

    seen = []
    x, norm = torch.ones(4096, 8192, device="cuda", dtype=torch.bfloat16), torch.ones(8192, device="cuda")
    for before in (np.full(most, 99), _parents(rng, most, "chain"), _parents(rng, most, "star"), -1.0, 1.0):
        if isinstance(before, float):  # rows that pass through the norm's shared memory
            cuda_lib.rms_norm((x * before), norm, torch.empty_like(x), 4096, 8192)
        else:
            run(most, [before] * seqs)
        seen.append(run(nodes, parents))
        assert torch.isfinite(seen[-1][0]).all()
    for out, lse in seen[1:]:
        assert torch.equal(out, seen[0][0]) and torch.equal(lse, seen[0][1])


def _stars(x, tokens, u, probs=None, max_rows=None):
    """A star for each row of x (the rows of its drafts are zeros): what test_gpu_drafts._verify takes."""
    seqs, m, n = tokens.shape[0], tokens.shape[1], x.shape[1]
    rows = np.zeros((seqs, m, n), np.float32)
    rows[:, 0] = x
    q = None
    if probs is not None:
        q = np.full((seqs, m, n), 1 / n, np.float32)
        q[:, 0] = probs
        q = q.reshape(-1, n)
    return dict(x=_t(rows.reshape(-1, n)), tokens=tokens.reshape(-1), parents=[np.array([-1] + [0] * (m - 1))] * seqs,
                u=u.astype(np.float32).reshape(-1), probs=q, cu=_cu([m] * seqs), nodes=[m] * seqs, n=n, temperature=1.0, kind="star")


def _accepted(w):
    """What the oracle accepts, by sequence."""
    x, m = _np(w["x"]), w["nodes"][0]
    return [dref.verify(x[s * m:s * m + m], w["tokens"][s * m:s * m + m], list(w["parents"][s]), w["u"][s * m:s * m + m].astype(np.float64),
                        None if w["probs"] is None else w["probs"][s * m:s * m + m], 1.0)[0][1:] for s in range(len(w["nodes"]))]


@pytest.mark.parametrize("n,at,max_rows", [(3000, [5, 9, 1500, 2999, 7], None), (3000, [0, 1030, 2050, 1, 2], None),
                                           (30001, [5, 9, 15000, 30000, 7], None), (30001, [5, 9, 15000, 30000, 7], 64)])
def test_what_rejected_likely_drafts_leave(cuda_lib, n, at, max_rows):
    # Drafts without probabilities: the likeliest tokens in order, all but the last refused, which is 2^-15 from its border.  The
    # first has up to 1 - 10^-6 of the probability.  (64 rows: the bound from which on rows are read when they are reached.)
    rng = np.random.default_rng(n + at[1])
    x, tokens, u, want = [], [], [], []
    for gap in (2.0, 5.0, 8.0, 11.0, 14.0):
        for last in range(5):
            for side in (-1, 1):
                for _ in range(1 if n > 3000 else 4):
                    row = (-gap - np.log(n) - 1 + 0.5 * rng.standard_normal(n)).astype(np.float32)
                    row[at] = (np.array([0.0] + [-gap] * 4) + 0.3 * rng.standard_normal(5)).astype(np.float32)
                    e = np.exp(row.astype(np.float64))
                    numbers = np.full(6, 0.5)
                    for i in range(last + 1):
                        w = e[at[i]] / e.sum()
                        numbers[1 + i] = w + 0.5 * (1 - w) if i < last else min(w * (1 + side * 2.0 ** -15), 1 - 2.0 ** -24)
                        e[at[i]] = 0
                    x.append(row)
                    tokens.append([0] + at[:last + 1] + [-1] * (4 - last))
                    u.append(numbers)
                    want.append([] if side > 0 and numbers[1 + last] > w else [last + 1])
    w = _stars(np.array(x), np.array(tokens), np.array(u))
    assert _accepted(w) == want
    assert max_rows is None or len(x) * max_rows * n * 4 > 128 << 20
    acc, path, nxt = _verify(cuda_lib, w, max_rows=max_rows)
    assert [p[1:a + 1].tolist() for p, a in zip(path, acc)] == want
    assert (nxt >= 0).all()


@pytest.mark.parametrize("n,max_rows", [(5000, None), (30001, None), (30001, 64)])
def test_drafts_that_the_target_nearly_has(cuda_lib, n, max_rows):
    # Probabilities that are the target's but for 2 * 10^-4 to 2 * 10^-3 of themselves.  The first draft is refused; the second
    # is 2^-13 from its border, or refused and the third is.  p - b q is 6 * 10^-5 there and S 2.7 * 10^-4: both are off by 2^-14
    # of themselves together.
    rng = np.random.default_rng(n)
    at = [10, 1500, 2600, 3700]
    x, probs, tokens, u, want = [], [], [], [], []
    for k in range(40):
        row = (np.log(1e-3 / n) - 0.3 + 0.5 * rng.standard_normal(n)).astype(np.float32)
        row[at] = np.log([0.3, 0.3, 0.25, 0.15]) + 0.02 * rng.standard_normal(4)
        p = np.exp(row.astype(np.float64))
        p /= p.sum()
        assert p.sum() - p[at].sum() < 2.0 ** -9.9
        q = 1.01 * p
        q[at] = p[at] * [1.5, 1 - 2e-4, 1 - 8e-4, 1 - 2e-3]
        q = q.astype(np.float32)
        side, last, w, numbers = (-1, 1)[k % 2], 1 + k // 2 % 2, p, np.full(4, 0.5)
        for i in range(last + 1):
            border = w[at[i]] / float(q[at[i]])
            numbers[1 + i] = border + 0.5 * (1 - border) if i < last else border * (1 + side * 2.0 ** -13)
            w = np.maximum(w - q, 0)
            w /= w.sum()
        x.append(row)
        probs.append(q)
        tokens.append([0] + at[:last + 1] + [-1] * (2 - last))
        u.append(numbers)
        want.append([] if side > 0 else [last + 1])
    w = _stars(np.array(x), np.array(tokens), np.array(u), np.array(probs))
    assert (np.array(u) < 1).all() and _accepted(w) == want
    assert max_rows is None or len(x) * max_rows * n * 4 > 128 << 20
    acc, path, nxt = _verify(cuda_lib, w, max_rows=max_rows)
    assert [p[1:a + 1].tolist() for p, a in zip(path, acc)] == want


@pytest.mark.parametrize("drafts", [True, False])
def test_a_draft_far_below_the_likeliest(cuda_lib, drafts):
    # p of 10^-20 to 10^-29: its number is 2^-21 from the border
    rng = np.random.default_rng(8)
    n, seqs = 3000, 60
    x = np.full((seqs, n), -90.0, np.float32)
    x[:, 1234] = rng.standard_normal(seqs)
    x[:, 77] = x[:, 1234] - rng.uniform(45, 66, seqs)
    p = np.exp(x.astype(np.float64) - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    side = np.where(np.arange(seqs) % 2 == 0, -1, 1)
    probs = None
    if drafts:
        probs = np.full((seqs, n), 1 / n, np.float32)
        probs[:, 77] = 2.0 ** -10
    u = np.stack([np.full(seqs, 0.5), p[:, 77] / (2.0 ** -10 if drafts else 1) * (1 + side * 2.0 ** -21)], 1)
    w = _stars(x, np.tile([0, 77], (seqs, 1)), u, probs)
    want = [[1] if s < 0 else [] for s in side]
    assert _accepted(w) == want
    acc, path, nxt = _verify(cuda_lib, w)
    assert [q[1:a + 1].tolist() for q, a in zip(path, acc)] == want


def test_a_row_that_is_finite_gives_a_token(cuda_lib):
    # Two likely tokens of one chunk whose drafts' probabilities are the target's to an f32's rounding: what a rejection leaves is
    # nothing, or less than the rounding of one of them.
    rng = np.random.default_rng(13)
    seqs, n = 4000, 64
    x = np.full((seqs, n), -np.inf, np.float32)
    x[:, 3], x[:, 40] = 1.0, rng.uniform(-2, 1, seqs)
    p = np.exp(x.astype(np.float64) - 1)
    p /= p.sum(1, keepdims=True)
    probs = p.astype(np.float32)
    probs[:, 3] *= np.float32(1.001)
    step = rng.integers(-2, 3, seqs)
    for k in (-2, -1, 1, 2):
        for _ in range(abs(k)):
            probs[step == k, 40] = np.nextafter(probs[step == k, 40], np.float32(np.inf if k > 0 else 0))
    u = np.stack([rng.random(seqs), np.full(seqs, 1 - 2.0 ** -24)], 1)
    w = _stars(x, np.tile([0, 3], (seqs, 1)), u, probs)
    acc, path, nxt = _verify(cuda_lib, w)
    assert (acc == 0).all()
    assert np.isin(nxt, [3, 40]).all()


@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 17, 2 ** 30, -2 ** 31])
def test_keep_of_a_length_far_past_the_pages(cuda_lib, far):
    # such a sequence's tokens have no pages: nothing of it is written, and the others' paths are kept
    import torch
    rng = np.random.default_rng(1)
    page, n_kv, dim = 16, 2, 64
    lens, nodes = [40, 40, 50], [10, 9, 12]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    paths, acc = [[0, 3, 5, 9], [0, 2, 4, 8], [0, 1, 7, 11]], [3, 3, 3]
    want = raw.clone()
    cuda_lib.kv_keep(want, _i32(table), _i32(lens), _i32(_cu(nodes)), _i32(paths), _i32([3, -1, 3]), n_kv, dim, page)
    lens[1] = far
    cuda_lib.kv_keep(raw, _i32(table), _i32(lens), _i32(_cu(nodes)), _i32(paths), _i32(acc), n_kv, dim, page)
    assert torch.equal(raw, want)
