"""Drafted tokens next to borders: results that no other call and no rounding may change."""
import numpy as np
import pytest

from test_gpu_decode_ops import _dt, _filled, _t, attn_kernel  # noqa: F401
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
