"""The debug build (-DQDQ_CHECKS) of the drafted tokens' operators: every guard holds on valid inputs.

The guards cover the cache records that are written, the parts, chunks and paths in workspaces and shared memory.  Each
operator runs through both builds, which must agree bit for bit, and the status word must stay 0.
"""
import numpy as np
import pytest

import test_gpu_drafts as drafts
from test_gpu_checked_decode import _i32, _same, checked  # noqa: F401

pytestmark = pytest.mark.gpu


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# (lengths before, new, heads, cache heads, dim, page, type, kind)
APPEND = [
    ([0, 37, 15], [1, 1, 1], 6, 2, 128, 16, "f32", None),
    ([0, 37, 15], [9, 30, 2], 6, 2, 64, 48, "bf16", "tree"),
    ([0, 37, 15, 3], [64, 30, 61, 0], 6, 2, 96, 16, "f16", "forest"),
    ([100, 3], [300, 171], 5, 3, 192, 64, "bf16", None),
    ([100, 3], [64, 171], 5, 3, 256, 16, "f32", None),
]


@pytest.mark.parametrize("old,new,heads,n_kv,dim,page,dtype,kind", APPEND)
def test_checked_append_rope(cuda_lib, checked, old, new, heads, n_kv, dim, page, dtype, kind):  # noqa: F811
    def run():
        r = drafts._append_rope(cuda_lib, np.random.default_rng(dim), old, new, heads, n_kv, dim, page, dtype, dim, False, True, kind)
        return [r["raw"], r["out"]]

    _same(cuda_lib, checked, run)


# (lengths, nodes, heads, cache heads, dim, page, type)
TREE = [
    ([777], [13], 24, 8, 128, 64, "f32"),
    ([3000, 64, 500, 20], [64, 64, 7, 20], 16, 2, 64, 16, "bf16"),
    ([20000, 100], [40, 9], 32, 8, 128, 64, "f16"),
    ([5000, 100], [33, 33], 8, 2, 256, 32, "bf16"),
    ([5000, 100, 70], [2, 33, 1], 8, 2, 192, 16, "f32"),
]


@pytest.mark.parametrize("lens,nodes,heads,n_kv,dim,page,dtype", TREE)
def test_checked_tree_attention(cuda_lib, checked, lens, nodes, heads, n_kv, dim, page, dtype):  # noqa: F811
    import torch
    rng = np.random.default_rng(dim)
    raw, table, _ = drafts._filled(rng, lens, page, n_kv, dim)
    q = _t(rng.standard_normal((sum(nodes), heads, dim)).astype(np.float32)).to(drafts._dt(dtype))
    par = _i32(np.concatenate([drafts._parents(rng, n) for n in nodes]))
    tab, kv_len, cu = _i32(table), _i32(lens), _i32(drafts._cu(nodes))

    def run():
        out, lse = torch.empty_like(q), torch.empty(sum(nodes), heads, device="cuda")
        ws = cuda_lib.kv_attention_workspace(len(lens), max(nodes), max(lens), heads, n_kv, dim)
        cuda_lib.kv_tree_attention(raw, tab, kv_len, q, out, ws, heads, n_kv, dim, page, max(lens), cu, max(nodes), par, lse=lse)
        return [out, lse]

    _same(cuda_lib, checked, run)


@pytest.mark.parametrize("nodes,n,kind,probs,temperature,dtype,most", [
    ([1, 2, 6, 0, 3], 1023, "chain", True, 1.0, "f32", 6),
    ([5, 9, 64], 5001, "tree", False, 1.0, "f16", 64),
    ([6, 5, 4], 50000, "tree", True, 1.0, "bf16", 6),
    ([6, 5, 4] * 6, 60001, "tree", True, 1.0, "f32", 40),
    ([6, 5, 4] * 6, 60001, "tree", False, 1.0, "f32", 40),
    ([6, 5, 4] * 6, 60001, "tree", True, 0.0, "f32", 40),
    ([2, 1, 4] * 16, 30001, "tree", True, 1.0, "bf16", 50),
])
def test_checked_verify(cuda_lib, checked, nodes, n, kind, probs, temperature, dtype, most):  # noqa: F811
    w = drafts._problem(np.random.default_rng(n), nodes, n, kind, probs, temperature, dtype)
    _same(cuda_lib, checked, lambda: [_t(np.asarray(x)) for x in drafts._verify(cuda_lib, w, max_rows=most)])


def test_checked_keep(cuda_lib, checked):  # noqa: F811
    rng = np.random.default_rng(4)
    lens, new, page, n_kv, dim = [40, 64, 77], [40, 20, 9], 16, 2, 96
    raw, table, _ = drafts._filled(rng, lens, page, n_kv, dim)
    path, acc = _i32([[0, 3, 30, 39], [2, 3, 17, -1], [0, -1, -1, -1]]), _i32([3, 2, 0])

    def run():
        mine = raw.clone()
        cuda_lib.kv_keep(mine, _i32(table), _i32(lens), _i32(drafts._cu(new)), path, acc, n_kv, dim, page)
        return [mine]

    _same(cuda_lib, checked, run)
