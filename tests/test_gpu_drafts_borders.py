"""Drafted tokens next to borders: results that no other call may change."""
import numpy as np
import pytest

from test_gpu_decode_ops import _dt, _filled, _t, attn_kernel  # noqa: F401
from test_gpu_drafts import _parents, _tree

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
