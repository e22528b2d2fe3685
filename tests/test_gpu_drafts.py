"""GPU parity of the operators of drafted tokens against the float64 forms of ``oracle.draft_oracle``.

Bounds (u = 2^-24, the f32 unit roundoff; e = the output type's: 2^-24, 2^-11, 2^-8):
* norm and rotation: a head's sum of squares is folded over at most 8 products per lane and 5 shuffles, so it is off by
  13 u, the root's reciprocal by half of that and 4 u, and two products follow: 13 u.  The angle reaches cos and sin as
  an f32 fraction of half a turn (off by 2^-25 of it: pi u), which are off by 2 u themselves: 8 u of the pair's
  magnitudes, and two products and a sum round by 3 u: |y - y_ref| <= 24 u (|a| + |b|) + e |y_ref|; 32 u below.
* cached keys and values: the code is within half a step s of the value and the step within 40 u of max / 127, so a value
  is off by s (1/2 + 127 * 40 u) and what the value itself was; a token that the block held before moves by another
  half a step where the step grew.
* attention: the bounds of test_gpu_decode_ops.py, whose kernels these are.
* verification: probabilities are off by 2^-22 (exponent), 2^-23 (its factor's rest) and the f32 sums of 1024 terms in 32
  lanes (2^-19 at most), relative, 2^-18 together: choices whose margin (as a
  probability) is above 2^-17 are equal.  Among thousands of unlikely tokens a number is often nearer than that to a border.
* kept tokens: codes and scales are equal (the definition is in f32 operations).
"""
import numpy as np
import pytest

from oracle import decode_oracle as ref
from oracle import draft_oracle as dref
from test_gpu_decode_ops import (EPS, U, _check_attention, _dt, _filled, _i32, _np, _pool, _t, _tables, _values, _within,  # noqa: F401
                                 attn_kernel)

pytestmark = pytest.mark.gpu

MARGIN = 2.0 ** -17


def _parents(rng, n, kind="tree"):
    if n == 0:
        return np.zeros(0, np.int64)
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "forest":  # several roots
        return np.array([-1 if rng.random() < 0.3 else rng.integers(-1, i) for i in range(n)], np.int64)
    if kind == "star":
        return np.array([-1] + [0] * (n - 1))
    return np.array([-1] + [i - 1 if rng.random() < 0.5 else rng.integers(0, i) for i in range(1, n)])


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


# ------------------------------------------------------------------ norm, rotation and append

ROPE = [
    # cached before, new, heads, kv heads, dim, page, dtype, turned, interleaved, norm, kind of tree (None: no parents)
    ([0], [1], 1, 1, 64, 16, "f32", 64, False, True, None),
    ([776], [1], 24, 8, 128, 64, "f32", 128, False, True, None),
    ([5, 0, 31, 16], [1] * 4, 6, 2, 128, 32, "bf16", 128, True, True, None),
    ([5, 0, 31, 16, 47], [3, 0, 17, 16, 1], 3, 1, 96, 16, "f16", 96, False, True, None),
    ([100, 7], [200, 33], 4, 2, 192, 48, "f32", 192, False, True, None),
    ([100, 7], [200, 33], 4, 2, 192, 48, "bf16", 64, True, False, None),
    ([0, 9], [70, 130], 8, 8, 256, 32, "f32", 256, False, False, None),
    ([0, 9], [70, 130], 2, 1, 256, 32, "f16", 128, False, True, None),
    ([12, 1], [50, 64], 7, 1, 64, 128, "bf16", 32, False, True, "tree"),
    ([1000, 3, 0, 15], [26, 64, 1, 5], 8, 2, 128, 64, "f32", 128, False, True, "tree"),
    ([30, 40], [64, 9], 8, 4, 128, 16, "f16", 8, True, True, "forest"),
    ([33, 5], [20, 31], 2, 2, 64, 16, "f32", 64, True, False, "star"),
    ([300], [900], 24, 8, 128, 64, "bf16", 128, False, False, None),
]


def _append_rope(qdq, rng, old, new, heads, n_kv, dim, page, dtype, turned, interleaved, norm, kind, far=0, base=10000.0):
    lens = [a + b for a, b in zip(old, new)]
    raw, table, c = _filled(rng, old, page, n_kv, dim, n_pages=sum(-(-n // page) for n in lens) + 3)
    table = np.pad(table, ((0, 0), (0, 3 + max(-(-n // page) for n in lens) - table.shape[1])), constant_values=-1)
    free = [p for p in range(c.raw.shape[0]) if p not in table]
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            if table[s, i] < 0:
                table[s, i] = free.pop()
    cu = _cu(new)
    q = _t(1.5 * rng.standard_normal((cu[-1], heads, dim)).astype(np.float32), _dt(dtype))
    k = _t(1.5 * rng.standard_normal((cu[-1], n_kv, dim)).astype(np.float32), _dt(dtype))
    v = _t(rng.standard_normal((cu[-1], n_kv, dim)).astype(np.float32), _dt(dtype))
    qw = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norm else None
    kw = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norm else None
    freqs = (base ** (-np.arange(turned // 2) * 2 / max(turned, 1))).astype(np.float32) if turned else None
    parents = None if kind is None else np.concatenate([_parents(rng, n, kind) for n in new]).astype(np.int32)
    import torch
    out = torch.full_like(q, 5.0)
    single = all(n == 1 for n in new)
    qdq.kv_append_rope(raw, _i32(table), _i32(lens), q, out, k, v, heads, n_kv, dim, page, None if freqs is None else _t(freqs),
                       interleaved, None if qw is None else _t(qw), None if kw is None else _t(kw), 1e-6,
                       cu_new=None if single else _i32(cu), max_new=max(new), parent=None if parents is None else _i32(parents))
    return dict(raw=raw, table=table, c=c, lens=lens, cu=cu, q=q, k=k, v=v, qw=qw, kw=kw, freqs=freqs, parents=parents, out=out)


def _check_rope(r, old, new, n_kv, dim, page, dtype, interleaved):
    got = ref.Cache(r["raw"].cpu().numpy(), page, n_kv, dim)
    untouched = np.ones(got.raw.shape, bool)
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    for s in range(len(new)):
        if new[s] == 0:
            continue
        a, b = r["cu"][s], r["cu"][s + 1]
        dep = np.arange(new[s]) if r["parents"] is None else dref.depths(r["parents"][a:b])
        pos = old[s] + dep
        y, mag = dref.norm_turn(_np(r["q"])[a:b], r["qw"], 1e-6, pos, r["freqs"], interleaved)
        _within(_np(r["out"])[a:b], y, 32 * U * mag + EPS[dtype] * np.abs(y) + tiny)
        yk, mk = dref.norm_turn(_np(r["k"])[a:b], r["kw"], 1e-6, pos, r["freqs"], interleaved)
        vals = {0: (yk, 32 * U * mk), 1: (_np(r["v"])[a:b], np.zeros_like(yk))}
        before, after = _values(r["c"], r["table"], s, old[s]), _values(got, r["table"], s, r["lens"][s])
        for b0 in range(old[s] // 16 * 16, r["lens"][s], 16):
            held, end = max(old[s] - b0, 0), min(r["lens"][s] - b0, 16)
            pid, t0 = r["table"][s, b0 // page], b0 % page
            for h in range(n_kv):
                untouched[pid, h, (t0 * dim):(t0 + end) * dim] = False
                untouched[pid, h, (page + t0) * dim:(page + t0 + end) * dim] = False
                for which in range(2):
                    at = 2 * page * dim + 4 * (which * (page // 16) + t0 // 16)
                    untouched[pid, h, at:at + 4] = False
                    new_vals, off = (x[b0 + held - old[s]:b0 + end - old[s], h] for x in vals[which])
                    s_old = float(r["c"]._scales(pid, h, which)[t0 // 16]) if held else 0.0
                    step = max(s_old, np.abs(new_vals).max() / 127)
                    g = after[which][b0:b0 + end, h]
                    _within(g[held:], new_vals, step * (0.5 + 127 * 40 * U) + off)
                    if held:
                        grown = 0.5 * step if step > s_old * (1 - 64 * U) else 0
                        _within(g[:held], before[which][b0:b0 + held, h], grown + 127 * 40 * U * step)
    assert np.array_equal(got.raw[untouched], r["c"].raw[untouched])  # nothing else is written


@pytest.mark.parametrize("old,new,heads,n_kv,dim,page,dtype,turned,interleaved,norm,kind", ROPE)
def test_append_rope(cuda_lib, old, new, heads, n_kv, dim, page, dtype, turned, interleaved, norm, kind):
    rng = np.random.default_rng(sum(old) + sum(new) + dim + heads)
    r = _append_rope(cuda_lib, rng, old, new, heads, n_kv, dim, page, dtype, turned, interleaved, norm, kind)
    _check_rope(r, old, new, n_kv, dim, page, dtype, interleaved)


@pytest.mark.parametrize("dim,page,dtype,new", [(64, 16, "f32", [5, 0, 33]), (96, 48, "bf16", [17, 1, 16]), (128, 64, "f16", [1, 1, 1]),
                                                (192, 32, "f32", [2, 40, 1]), (256, 16, "bf16", [9, 31, 64])])
def test_append_rope_without_norm_and_rotation_is_append(cuda_lib, dim, page, dtype, new):
    # bit for bit, and the queries as they are
    import torch
    rng = np.random.default_rng(dim)
    n_kv, heads = 2, 6
    old = [20, 7, 16]
    r = _append_rope(cuda_lib, rng, old, new, heads, n_kv, dim, page, dtype, 0, False, False, None)
    assert torch.equal(r["out"], r["q"])
    want = _t(r["c"].raw.reshape(r["raw"].shape))
    cuda_lib.kv_append(want, _i32(r["table"]), _i32(r["lens"]), r["k"], r["v"], n_kv, dim, page, cu_new=_i32(r["cu"]), max_new=max(new))
    assert torch.equal(want, r["raw"])


@pytest.mark.parametrize("pos", [1 << 16, 1 << 20, 4194303])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_at_far_positions(cuda_lib, pos, interleaved):
    # an f32 angle would be off by up to a tenth of a radian here
    import torch
    rng = np.random.default_rng(pos)
    dim, heads, page = 128, 4, 128
    raw = _pool(2, page, 1, dim)
    table = np.full((1, pos // page + 1), -1, np.int32)
    table[0, -1] = 1
    q = _t(rng.standard_normal((1, heads, dim)).astype(np.float32))
    k = _t(rng.standard_normal((1, 1, dim)).astype(np.float32))
    freqs = np.concatenate([[1.0, 0.5], 500000.0 ** (-np.arange(2, 64) / 64)]).astype(np.float32)
    out = torch.empty_like(q)
    n = pos % 16 + 1  # the block's tokens before the last come first, so that it holds them
    cuda_lib.kv_append(raw, _i32(table), _i32([pos + 1]), k.expand(n, 1, dim).contiguous(), k.expand(n, 1, dim).contiguous(), 1, dim, page,
                       cu_new=_i32([0, n]), max_new=n)
    cuda_lib.kv_append_rope(raw, _i32(table), _i32([pos + 1]), q, out, k, k, heads, 1, dim, page, _t(freqs), interleaved)
    y, mag = dref.norm_turn(_np(q), None, 0, [pos], freqs, interleaved)
    _within(_np(out), y, 32 * U * mag + U * np.abs(y))


def test_append_rope_of_keys_and_values_alone(cuda_lib):
    import torch
    rng = np.random.default_rng(5)
    r = _append_rope(cuda_lib, rng, [20, 3], [9, 30], 4, 2, 128, 32, "bf16", 128, False, True, "tree")
    want = _t(r["c"].raw.reshape(r["raw"].shape))
    cuda_lib.kv_append_rope(want, _i32(r["table"]), _i32(r["lens"]), None, None, r["k"], r["v"], 0, 2, 128, 32, _t(r["freqs"]),
                            False, None, _t(r["kw"]), cu_new=_i32(r["cu"]), max_new=30, parent=_i32(r["parents"]))
    assert torch.equal(want, r["raw"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_rope_of_slices_of_one_buffer_and_in_place(cuda_lib, dtype):
    # q, k and v as a fused projection leaves them; queries turned where they lie
    import torch
    rng = np.random.default_rng(8)
    heads, n_kv, dim, page = 6, 2, 64, 16
    r = _append_rope(cuda_lib, rng, [20, 3], [9, 30], heads, n_kv, dim, page, dtype, 64, False, True, "tree")
    rows = r["cu"][-1]
    buf = torch.full((rows + 1, heads + 2 * n_kv + 1, dim), 7.0, device="cuda", dtype=_dt(dtype))
    q, k, v = buf[:rows, :heads], buf[:rows, heads:heads + n_kv], buf[:rows, heads + n_kv:heads + 2 * n_kv]
    q.copy_(r["q"])
    k.copy_(r["k"])
    v.copy_(r["v"])
    raw = _t(r["c"].raw.reshape(r["raw"].shape))
    cuda_lib.kv_append_rope(raw, _i32(r["table"]), _i32(r["lens"]), q, q, k, v, heads, n_kv, dim, page, _t(r["freqs"]), False,
                            _t(r["qw"]), _t(r["kw"]), cu_new=_i32(r["cu"]), max_new=30, parent=_i32(r["parents"]))
    assert torch.equal(raw, r["raw"]) and torch.equal(q, r["out"]) and torch.equal(k, r["k"]) and torch.equal(v, r["v"])
    assert (buf[rows] == 7).all() and (buf[:, -1] == 7).all()


def test_append_rope_of_what_is_no_tree_or_no_sequence(cuda_lib):
    # parents that are not earlier, and their descendants; more new tokens than there are; no page; freqs that are no numbers
    import torch
    rng = np.random.default_rng(9)
    heads, n_kv, dim, page = 2, 1, 64, 16
    raw = _pool(8, page, n_kv, dim)
    before = raw.clone()
    table = [[0, 1], [2, 3], [-1, 4], [5, 6]]
    new = [6, 5, 6, 3]
    cu = _cu(new)
    parents = [-1, 0, 3, 0, 2, -2] + [-1, 0, 1, 2, 3] + [-1, 0, 0, 1, 1, 2] + [-1, 0, 0]
    q, k, v = (_t(rng.standard_normal((cu[-1], n, dim)).astype(np.float32)) for n in (heads, n_kv, n_kv))
    freqs = np.ones(32, np.float32)
    out = torch.full_like(q, 5.0)
    cuda_lib.kv_append_rope(raw, _i32(table), _i32([6, 3, 6, 3]), q, out, k, v, heads, n_kv, dim, page, _t(freqs), cu_new=_i32(cu),
                            max_new=6, parent=_i32(parents))
    got = np.isnan(_np(out)).all((1, 2))
    assert got.tolist() == [False, False, True, False, True, True] + [True] * 5 + [False] * 9
    assert np.isfinite(_np(out)[~got]).all()
    assert torch.equal(raw[2:5], before[2:5])  # nothing appended, and nothing without a page
    kk, vv = torch.zeros(6, n_kv, dim, device="cuda"), torch.zeros(6, n_kv, dim, device="cuda")
    cuda_lib.kv_read(raw, _i32(table[:1]), None, _i32([0, 6]), kk, vv, n_kv, dim, page, 6)
    assert torch.isnan(kk).all() and torch.isfinite(vv).all()
    freqs[3] = np.inf
    cuda_lib.kv_append_rope(raw, _i32(table[3:]), _i32([3]), q[17:], out[17:], k[17:], v[17:], heads, n_kv, dim, page, _t(freqs),
                            cu_new=_i32([0, 3]), max_new=3)
    assert np.isnan(_np(out)[17:, :, [3, 35]]).all() and np.isfinite(np.delete(_np(out)[17:], [3, 35], 2)).all()


def test_append_rope_of_tokens_past_max_new(cuda_lib):
    import torch
    rng = np.random.default_rng(4)
    heads, n_kv, dim, page = 2, 1, 128, 16
    raw = _pool(8, page, n_kv, dim)
    table = _i32([[0, 1, 2], [3, 4, 5]])
    q, k, v = (_t(rng.standard_normal((40, n, dim)).astype(np.float32)) for n in (heads, n_kv, n_kv))
    out = torch.full_like(q, 5.0)
    freqs = _t(np.ones(64, np.float32))
    cuda_lib.kv_append_rope(raw, table, _i32([33, 7]), q, out, k, v, heads, n_kv, dim, page, freqs, cu_new=_i32([0, 33, 40]), max_new=18)
    assert (out[18:33] == 5).all() and not (out[:18] == 5).any() and not (out[33:] == 5).any()
    want = _pool(8, page, n_kv, dim)
    cuda_lib.kv_append_rope(want, table, _i32([18, 7]), torch.cat([q[:18], q[33:]]), torch.empty(25, heads, dim, device="cuda"),
                            torch.cat([k[:18], k[33:]]), torch.cat([v[:18], v[33:]]), heads, n_kv, dim, page, freqs,
                            cu_new=_i32([0, 18, 25]), max_new=18)
    assert torch.equal(raw, want)


# ------------------------------------------------------------------ tree attention

def _tree(qdq, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents, softcap=0.0, window=0, slopes=None, max_kv=None,
          max_q=None, workspace=None):
    import torch
    out, lse = torch.full_like(q, 5.0), torch.full((q.shape[0], heads), 5.0, device="cuda")
    max_q = max_q or int(max(nodes))
    max_kv = max_kv if max_kv is not None else int(max(lens))
    ws = workspace if workspace is not None else qdq.kv_attention_workspace(len(lens), max_q, max_kv, heads, n_kv, dim)
    qdq.kv_tree_attention(raw, _i32(table), _i32(lens), q, out, ws, heads, n_kv, dim, page, max_kv, _i32(_cu(nodes)), max_q,
                          _i32(np.concatenate(parents)), softcap=softcap, window=window, slopes=slopes, lse=lse)
    return out, lse


def _check_tree(c, table, lens, nodes, parents, q, out, lse, dtype, scale, softcap, window, slopes):
    cu = _cu(nodes)
    qn, on, ln = _np(q), _np(out), _np(lse)
    for s, n in enumerate(lens):
        if nodes[s] == 0:
            continue
        k, v = _values(c, table, s, n)
        a, b = cu[s], cu[s + 1]
        o, l, av, mag, z = dref.tree_attention(qn[a:b], k, v, list(parents[s]), scale, softcap, window, None if slopes is None else _np(slopes))
        d = 2.0 ** -18 * mag + 2.0 ** -20 * (1 + softcap)
        tiny = 2.0 ** -25 if dtype == "f16" else 0
        _within(on[a:b], o, ((2 * d + 2.0 ** -17 + (0 if dtype == "f32" else 2.0 ** -11))[..., None] * av + EPS[dtype] * np.abs(o) + tiny
                             + 2.0 ** -39 * n * z[..., None]))
        with np.errstate(invalid="ignore"):
            _within(ln[a:b], l, d + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(np.isinf(l), 0, l)))


TREE = [
    # lens, nodes, heads, kv heads, dim, page, dtype, softcap, window, bias, kind
    ([1], [1], 1, 1, 64, 16, "f32", 0, 0, False, "tree"),
    ([7], [7], 2, 1, 128, 16, "f32", 0, 0, False, "tree"),            # nothing before the tree
    ([64, 80], [64, 64], 4, 2, 64, 16, "bf16", 0, 0, False, "forest"),
    ([777], [13], 24, 8, 128, 64, "f32", 0, 0, False, "tree"),
    ([300, 0, 17, 40], [5, 0, 17, 1], 6, 2, 128, 32, "f16", 0, 0, True, "tree"),
    ([300, 129, 70], [3, 31, 40], 7, 1, 96, 48, "f32", 30.0, 0, False, "forest"),
    ([300, 129, 70], [33, 31, 64], 4, 4, 256, 32, "f16", 0, 37, True, "tree"),
    ([300, 129, 70], [33, 64, 64], 4, 4, 256, 32, "f32", 0, 5, True, "chain"),
    ([50, 65], [5, 64], 10, 2, 192, 16, "bf16", 20.0, 16, True, "tree"),
    ([1500, 333], [64, 63], 12, 4, 128, 64, "f32", 0, 0, False, "tree"),
    ([1500, 90, 257], [64, 40, 1], 16, 2, 128, 16, "bf16", 0, 0, False, "tree"),
    ([513, 700], [64, 50], 16, 1, 64, 32, "f32", 30.0, 200, True, "tree"),
    ([513, 700], [64, 50], 16, 1, 64, 32, "f16", 0, 1, False, "tree"),
    ([1000, 80], [64, 64], 8, 2, 192, 48, "f32", 0, 0, True, "forest"),
    ([9000, 300], [48, 5], 4, 1, 128, 32, "bf16", 0, 0, False, "tree"),
    ([9000, 300], [48, 64], 4, 1, 64, 32, "f32", 0, 8000, False, "star"),
    ([6000, 100, 2100], [2, 3, 1], 9, 3, 64, 16, "f16", 0, 2, False, "tree"),
    ([400, 81], [26, 64], 3, 1, 96, 16, "bf16", 0, 0, False, "chain"),
]


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("lens,nodes,heads,n_kv,dim,page,dtype,softcap,window,bias,kind", TREE)
def test_tree_attention(cuda_lib, lens, nodes, heads, n_kv, dim, page, dtype, softcap, window, bias, kind):
    rng = np.random.default_rng(sum(lens) + heads + dim)
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    q = _t(1.5 * rng.standard_normal((sum(nodes), heads, dim)).astype(np.float32), _dt(dtype))
    parents = [_parents(rng, n, kind) for n in nodes]
    slopes = _t((2.0 ** -np.linspace(1, 8, heads)).astype(np.float32)) if bias else None
    out, lse = _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents, softcap, window, slopes)
    _check_tree(c, table, lens, nodes, parents, q, out, lse, dtype, dim ** -0.5, softcap, window, slopes)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("dtype,softcap,window,bias", [("f32", 0, 0, False), ("bf16", 30.0, 50, True)])
def test_a_chain_is_causal_attention(cuda_lib, dtype, softcap, window, bias):
    rng = np.random.default_rng(2)
    lens, nodes, heads, n_kv, dim, page = [500, 64, 90], [64, 64, 7], 8, 2, 128, 16
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    q = _t(1.5 * rng.standard_normal((sum(nodes), heads, dim)).astype(np.float32), _dt(dtype))
    slopes = _t((2.0 ** -np.linspace(1, 8, heads)).astype(np.float32)) if bias else None
    out, lse = _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, [_parents(rng, n, "chain") for n in nodes], softcap,
                     window, slopes)
    _check_attention(c, table, lens, nodes, q, out, lse, dtype, dim ** -0.5, softcap, window, slopes)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("heads,n_kv", [(2, 2), (16, 1)])
def test_tree_attention_of_what_is_no_tree(cuda_lib, heads, n_kv):
    # a node without a valid parent and its descendants are NaN, the others are not; and so is a sequence with more rows
    # than max_q (in its first max_q), with a length out of range, or a page that is not there
    import torch
    rng = np.random.default_rng(3)
    lens, nodes, dim, page = [100, 90, 70, 60], [8, 20, 8, 8], 64, 16
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    q = _t(rng.standard_normal((sum(nodes), heads, dim)).astype(np.float32), _dt("bf16"))
    parents = [np.array([-1, 0, 1, 5, 3, 2, -7, 6]), _parents(rng, 20), _parents(rng, 8), _parents(rng, 8)]
    table[3, 1] = 1 << 29
    out, lse = _tree(cuda_lib, raw, table, [100, 90, 71 + 1000, 60], nodes, q, heads, n_kv, dim, page, parents, max_kv=200, max_q=16)
    nan = np.isnan(_np(out)).all((1, 2))
    assert nan[:8].tolist() == [False, False, False, True, True, False, True, True]
    assert nan[8:24].all() and (out[24:28] == 5).all()
    assert nan[28:36].all() and nan[36:].all() and np.array_equal(np.isnan(_np(lse)).all(1), nan)
    good = [0, 1, 2, 5]
    k, v = _values(c, table, 0, 100)
    o = dref.tree_attention(_np(q)[:8], k, v, [-1, 0, 1, 0, 0, 2, 0, 0], dim ** -0.5)[0]
    assert np.abs(_np(out)[good] - o[good]).max() < 2.0 ** -5 * np.abs(o).max()
    torch.cuda.synchronize()


@pytest.mark.usefixtures("attn_kernel")
def test_hidden_drafts_do_not_reach_a_row(cuda_lib):
    # NaN scales and queries of one branch stay in it (a block of its own)
    rng = np.random.default_rng(6)
    heads, n_kv, dim, page = 12, 1, 128, 16
    lens, nodes = [96], [48]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    c._scales(table[0, 4], 0, 0)[0] = np.nan   # tokens 64 .. 79: nodes 16 .. 31
    c._scales(table[0, 5], 0, 1)[0] = np.nan   # tokens 80 .. 95: nodes 32 .. 47
    raw = _t(c.raw.reshape(raw.shape))
    parents = [np.array([-1] + list(range(15)) + [15] + list(range(16, 31)) + [15] + list(range(32, 47)))]
    q = _t(rng.standard_normal((48, heads, dim)).astype(np.float32), _dt("f16"))
    out, lse = _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents)
    assert np.isfinite(_np(out)[:16]).all() and np.isnan(_np(out)[16:]).all()
    assert np.isfinite(_np(lse)[:16]).all() and np.isnan(_np(lse)[16:32]).all()


@pytest.mark.usefixtures("attn_kernel")
def test_trees_share_a_workspace_and_repeat(cuda_lib):
    # calls of other shapes, of attention without trees and of log probabilities between them
    import torch
    rng = np.random.default_rng(7)
    heads, n_kv, dim, page = 8, 2, 64, 16
    lens, nodes = [5000, 17, 3000, 64], [64, 3, 30, 64]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    q = _t(rng.standard_normal((sum(nodes), heads, dim)).astype(np.float32), _dt("bf16"))
    parents = [_parents(rng, n) for n in nodes]
    ws = cuda_lib.kv_attention_workspace(8, 64, 5000, heads, n_kv, dim)
    first = _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents, max_kv=5000, workspace=ws)
    x = torch.randn(3, 5000, device="cuda")
    for window in (0, 40, 0):
        _tree(cuda_lib, raw, table[2:], lens[2:], nodes[2:], q[67:], heads, n_kv, dim, page, parents[2:], window=window, max_kv=5000,
              workspace=ws)
        cuda_lib.kv_attention(raw, _i32(table), _i32(lens), q[:4], torch.empty_like(q[:4]), ws, heads, n_kv, dim, page, 5000)
        cuda_lib.token_logprobs(x, None, None, torch.empty(3, device="cuda"), 3, 5000, ws)
        cuda_lib.verify_drafts(x, None, torch.rand(3, device="cuda"), _i32([0] * 3), _i32([[0]] * 3), _i32([0] * 3), 5000, ws)
        again = _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents, max_kv=5000, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("n_seqs,nq,heads,n_kv,dim,max_kv", [(1, 64, 8, 1, 64, 3000), (3, 17, 2, 2, 128, 70000), (40, 5, 8, 8, 64, 900),
                                                             (2, 64, 16, 1, 128, 20000)])
def test_tree_workspace_is_enough_for_any_window(cuda_lib, n_seqs, nq, heads, n_kv, dim, max_kv):
    # (refused with QDQ_ERR_SCRATCH else); lengths at the bound, results against the call without a window that hides
    import torch
    rng = np.random.default_rng(nq)
    page = 64
    n_pages = -(-max_kv // page)
    raw = torch.zeros(n_pages, n_kv, ref.record_bytes(page, dim), dtype=torch.uint8, device="cuda")
    raw[:, :, :2 * page * dim] = torch.randint(0, 200, (n_pages, n_kv, 2 * page * dim), device="cuda", dtype=torch.uint8)
    raw.view(torch.float32)[:, :, page * dim // 2:] = 1 / 64
    table = np.tile(np.arange(n_pages, dtype=np.int32), (n_seqs, 1))  # all sequences read the same pages
    lens, nodes = [max_kv] * n_seqs, [nq] * n_seqs
    q = _t(rng.standard_normal((n_seqs * nq, heads, dim)).astype(np.float32), _dt("bf16"))
    parents = [_parents(rng, nq) for _ in lens]
    ws = cuda_lib.kv_attention_workspace(n_seqs, nq, max_kv, heads, n_kv, dim)
    run = lambda w: _tree(cuda_lib, raw, table, lens, nodes, q, heads, n_kv, dim, page, parents, window=w, workspace=ws)  # noqa: E731
    all_, lse = run(0)
    for window in (1, 17, max_kv // 3, max_kv - nq, max_kv - 1, max_kv, (1 << 31) - 1):
        out, l = run(window)
        assert torch.isfinite(out).all() and torch.isfinite(l).all() and (l <= lse + 2.0 ** -12).all()
        if window >= max_kv:
            assert torch.equal(out, all_)
    out, _ = run(1)  # a node sees itself alone: its value
    k, v = (torch.empty(nq, n_kv, dim, device="cuda") for _ in range(2))
    cuda_lib.kv_read(raw, _i32(table[:1]), _i32([max_kv - nq]), _i32([0, nq]), k, v, n_kv, dim, page, nq)
    want = v.repeat_interleave(heads // n_kv, 1).repeat(n_seqs, 1, 1)
    assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -11).all()


# ------------------------------------------------------------------ verification

def _peaked(rng, rows, n, peaks=16):
    x = 2.5 * rng.standard_normal((rows, n))
    for r in range(rows):
        x[r, rng.integers(0, n, peaks)] = np.log(n) + 3 + 2 * rng.standard_normal(peaks)
    return x.astype(np.float32)


def _softmax(x, t=1.0):
    e = np.exp((x - x.max(-1, keepdims=True)) / t)
    return e / e.sum(-1, keepdims=True)


def _problem(rng, nodes, n, kind, drafts, temperature, dtype):
    import torch
    rows = sum(nodes)
    x = _t(_peaked(rng, rows, n), _dt(dtype))
    xn = _np(x)
    p = _softmax(xn + 0.8 * rng.standard_normal(xn.shape), temperature or 1.0)
    parents = [_parents(rng, m, kind) for m in nodes]
    cu, tokens = _cu(nodes), np.zeros(rows, np.int64)
    for s, par in enumerate(parents):
        for i, up in enumerate(par):
            if up < 0:
                continue
            if drafts:
                tokens[cu[s] + i] = rng.choice(n, p=p[cu[s] + up] / p[cu[s] + up].sum())
            else:
                rank = int((par[:i] == up).sum())
                tokens[cu[s] + i] = np.argsort(-p[cu[s] + up])[min(rank, n - 1)]
    u = rng.random(rows).astype(np.float32)
    probs = p.astype(np.float32) if drafts else None
    return dict(x=x, tokens=tokens, parents=parents, u=u, probs=probs, cu=cu, nodes=nodes, n=n, temperature=temperature, kind=kind)


def _verify(qdq, w, max_rows=None, cu=True, **over):
    import torch
    a = dict(w, **over)
    seqs = len(a["nodes"])
    max_rows = max_rows or max(1, max(a["nodes"]))
    acc, path, nxt = (torch.full(shape, -9, dtype=torch.int32, device="cuda") for shape in ((seqs,), (seqs, max_rows), (seqs,)))
    ws = qdq.verify_drafts_workspace(seqs, max_rows, a["n"])
    probs = a["probs"]
    qdq.verify_drafts(a["x"], None if a["tokens"] is None else _i32(a["tokens"]), None if a["u"] is None else _t(a["u"]), acc, path, nxt,
                      a["n"], ws, cu=_i32(a["cu"]) if cu else None, max_rows=max_rows,
                      parent=None if a["kind"] == "chain" or a["parents"] is None else _i32(np.concatenate(a["parents"])),
                      draft_probs=probs if probs is None or not isinstance(probs, np.ndarray) else _t(probs), temperature=a["temperature"])
    return _np(acc), _np(path), _np(nxt)


def _check_verify(w, got):
    """Equal to the oracle; where a choice is nearer to its border than MARGIN, to the oracle with that number moved over it.

    (Probabilities that are off by a share of at most MARGIN / 2 move the two sides of a comparison by at most that
    share of 1, which is what moving the number by MARGIN does; far from every border they change nothing.)"""
    acc, path, nxt = got
    x = _np(w["x"])
    for s, m in enumerate(w["nodes"]):
        a, b = w["cu"][s], w["cu"][s + 1]
        if m == 0:
            assert acc[s] == -1 and nxt[s] == -1 and (path[s] == -1).all()
            continue
        u = None if w["u"] is None else w["u"][a:b].astype(np.float64)

        def outcome(u):
            want, token, margin = dref.verify(x[a:b], w["tokens"][a:b], list(w["parents"][s]), u, None if w["probs"] is None else w["probs"][a:b],
                                              w["temperature"])
            return (want + [-1] * (path.shape[1] - len(want)), len(want) - 1, token), margin

        want, margin = outcome(u)
        mine = (path[s].tolist(), acc[s], nxt[s])
        if margin < MARGIN and mine != want:
            moved = [np.where(np.arange(m) == i, u + d, u) for i in range(m) for d in (-MARGIN, MARGIN)]
            assert mine in [outcome(v)[0] for v in moved], (s, mine, want, margin)
        else:
            assert mine == want, (s, margin)


VERIFY = [
    # nodes, n, kind, drafts with probabilities, temperature, dtype
    ([1], 1, "chain", True, 1.0, "f32"),
    ([4, 0, 1, 7], 5, "tree", False, 1.0, "f32"),
    ([1, 2, 6, 0, 3], 1023, "chain", True, 1.0, "f32"),
    ([8] * 20, 1025, "chain", True, 0.7, "bf16"),
    ([5, 9, 64, 33], 5000, "tree", True, 1.0, "f32"),
    ([5, 9, 64, 33], 5001, "tree", True, 1.3, "f16"),
    ([5, 9, 64, 33], 4999, "tree", False, 1.0, "f32"),
    ([64] * 6, 3001, "star", True, 1.0, "bf16"),
    ([64] * 6, 3001, "star", False, 1.0, "f32"),
    ([6, 5, 4], 128256, "chain", True, 1.0, "f32"),
    ([6, 5, 14], 128256, "tree", False, 0.8, "bf16"),
    ([12, 3, 20], 30001, "tree", True, 0.0, "bf16"),
    ([12, 3, 20], 30003, "tree", False, 0.0, "f32"),
    ([1] * 40, 50001, "chain", True, 1.0, "f16"),
]


@pytest.mark.parametrize("nodes,n,kind,drafts,temperature,dtype", VERIFY)
def test_verify(cuda_lib, nodes, n, kind, drafts, temperature, dtype):
    rng = np.random.default_rng(sum(nodes) + n)
    for _ in range(3):
        w = _problem(rng, nodes, n, kind, drafts, temperature, dtype)
        _check_verify(w, _verify(cuda_lib, w))


def test_verify_rejects_down_to_what_is_left(cuda_lib):
    # every draft of a star is refused (numbers just below 1, drafts that the target hardly has), child after child
    rng = np.random.default_rng(1)
    w = _problem(rng, [9, 9, 9], 2000, "star", True, 1.0, "f32")
    w["u"][:] = np.float32(0.9999)
    w["u"][::9] = rng.random(3)
    w["probs"] = _softmax(rng.standard_normal(w["probs"].shape)).astype(np.float32)
    got = _verify(cuda_lib, w)
    _check_verify(w, got)
    assert (got[0] <= 1).all()
    w["probs"] = None
    w["tokens"] = rng.integers(0, 2000, 27)
    w["tokens"][5] = w["tokens"][4]      # the same draft twice
    w["tokens"][3], w["tokens"][12] = -1, 2000   # no tokens
    got = _verify(cuda_lib, w)
    _check_verify(w, got)


def test_verify_first_and_last_numbers(cuda_lib):
    # u = 0 accepts whatever has a probability and draws the first token that has one; u = 1 and more draw the last
    import torch
    n = 5000
    x = np.full((4, n), -np.inf, np.float32)
    x[:, 100:4000:7] = 0.0
    w = dict(x=_t(x), tokens=np.array([0, 100, 0, 101]), parents=[np.array([-1, 0])] * 2, u=np.zeros(4, np.float32), probs=None,
             cu=np.array([0, 2, 4]), nodes=[2, 2], n=n, temperature=1.0, kind="tree")
    acc, path, nxt = _verify(cuda_lib, w)
    assert acc.tolist() == [1, 0] and nxt.tolist() == [100, 100]
    for u in (1.0, 2.0, np.float32(1) - np.float32(2.0 ** -24)):
        w["u"] = np.full(4, u, np.float32)
        acc, path, nxt = _verify(cuda_lib, w)
        assert acc.tolist() == [0, 0] and nxt.tolist() == [3999, 3999]  # 100 is lost in the first, 3999 the last that is left
    w["u"] = np.full(4, np.nan, np.float32)
    assert ((0 <= _verify(cuda_lib, w)[2]) & (_verify(cuda_lib, w)[2] < n)).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("temperature", [1.0, 0.0])
def test_verify_rows_that_are_not_finite(cuda_lib, temperature):
    rng = np.random.default_rng(2)
    n = 3000
    for value in (np.nan, np.inf, -np.inf):
        w = _problem(rng, [2, 2, 2], n, "chain", True, temperature, "f32")
        x = w["x"].cpu().numpy()
        if value == -np.inf:
            x[[0, 3]] = value
        else:
            x[0, 7] = x[3, 2999] = value
        for s in range(3):  # drafts that are accepted where they can be
            w["tokens"][2 * s + 1] = int(np.argmax(x[2 * s]))
            w["probs"][2 * s, w["tokens"][2 * s + 1]] = 1e-6
        w["x"], w["u"] = _t(x), np.full(6, 1e-3, np.float32)
        acc, path, nxt = _verify(cuda_lib, w)
        assert acc.tolist() == [0, 1, 1] and nxt[0] == -1 and nxt[1] == -1 and 0 <= nxt[2] < n
        assert path.tolist() == [[0, -1], [0, 1], [0, 1]]


def test_verify_masked_logits_and_tiny_temperatures(cuda_lib):
    # masks of -inf and of the type's lowest value; a temperature that leaves one token
    import torch
    rng = np.random.default_rng(3)
    for dtype in ("f32", "f16", "bf16"):
        for low in (-np.inf, float(torch.finfo(_dt(dtype)).min)):
            w = _problem(rng, [5, 5, 5, 5], 4001, "tree", True, 1.0, dtype)
            x = w["x"].clone()
            x[:, 1::2] = low
            w["x"] = x
            got = _verify(cuda_lib, w)
            _check_verify(w, got)
            assert (got[2] % 2 == 0).all()
    w = _problem(rng, [5, 5], 4001, "tree", False, 1e-6, "f32")
    best = _np(w["x"]).argmax(1)
    acc, path, nxt = _verify(cuda_lib, w)
    for s in range(2):
        assert nxt[s] == best[w["cu"][s] + path[s][acc[s]]]


@pytest.mark.parametrize("offset,pad,dtype", [(0, 0, "f32"), (1, 3, "f32"), (3, 1, "bf16"), (0, 5, "f16"), (7, 9, "bf16")])
def test_verify_strided_rows(cuda_lib, offset, pad, dtype):
    # rows at every alignment inside wider buffers, whose other elements would win
    import torch
    rng = np.random.default_rng(offset + pad)
    n = 4097
    w = _problem(rng, [4, 7, 1, 5], n, "tree", True, 1.0, dtype)
    rows = sum(w["nodes"])
    buf = torch.full((rows * (n + pad) + offset,), 100.0, device="cuda", dtype=_dt(dtype))
    x = buf[offset:].as_strided((rows, n), (n + pad, 1))
    x.copy_(w["x"])
    pb = torch.full((rows * (n + pad) + offset,), 100.0, device="cuda")
    probs = pb[offset:].as_strided((rows, n), (n + pad, 1))
    probs.copy_(_t(w["probs"]))
    _check_verify(w, _verify(cuda_lib, dict(w, x=x, probs=probs)))


def test_verify_without_drafts(cuda_lib):
    # one row per sequence: the next token alone
    rng = np.random.default_rng(5)
    w = _problem(rng, [1] * 200, 1500, "chain", False, 0.9, "f32")
    _check_verify(w, _verify(cuda_lib, dict(w, tokens=None, probs=None), cu=False))


def test_verify_rows_past_max_rows_do_not_count(cuda_lib):
    rng = np.random.default_rng(6)
    w = _problem(rng, [12, 3, 9], 2000, "tree", True, 1.0, "f32")
    got = _verify(cuda_lib, w, max_rows=5)
    cut = dict(w, nodes=[5, 3, 5])
    cut["parents"] = [p[:5] for p in w["parents"]]
    for s, (a, m) in enumerate(zip(w["cu"], cut["nodes"])):
        want, token, margin = dref.verify(_np(w["x"])[a:a + m], w["tokens"][a:a + m], list(cut["parents"][s]), w["u"][a:a + m], w["probs"][a:a + m], 1.0)
        assert margin > MARGIN and got[0][s] == len(want) - 1 and got[2][s] == token and got[1][s].tolist() == want + [-1] * (5 - len(want))


def test_verify_parents_that_are_none(cuda_lib):
    # a node whose parent is not earlier is not reached
    rng = np.random.default_rng(7)
    w = _problem(rng, [6], 900, "tree", False, 1.0, "f32")
    best = int(_np(w["x"])[0].argmax())
    w["tokens"][:] = best
    w["u"][:] = 0
    w["parents"] = [np.array([-1, 1, 5, -3, 64, 0])]
    acc, path, _ = _verify(cuda_lib, w)
    assert acc.tolist() == [1] and path[0].tolist() == [0, 5, -1, -1, -1, -1]


@pytest.mark.parametrize("drafts", [True, False])
def test_the_emitted_token_has_the_targets_distribution(cuda_lib, drafts):
    # 40000 sequences of one target: how often a token comes first is binomial; 5.5 deviations for 12 tokens
    import torch
    S, n, m = 40000, 12, 4
    g = torch.Generator(device="cuda").manual_seed(3)
    p, q = (torch.randn(n, device="cuda", generator=g) for _ in range(2))
    q = torch.softmax(q, 0)
    x = (2 * p).expand(S * m, n).contiguous()
    target = torch.softmax(2 * p.double(), 0).cpu().numpy()
    tokens = torch.multinomial(q.expand(S * m, n), 1, generator=g)[:, 0].to(torch.int32)
    parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda").repeat(S)
    u = torch.rand(S * m, device="cuda", generator=g)
    acc, path, nxt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((S,), (S, m), (S,)))
    cuda_lib.verify_drafts(x, tokens, u, acc, path, nxt, n, cuda_lib.verify_drafts_workspace(S, m, n),
                           cu=torch.arange(0, S * m + 1, m, dtype=torch.int32, device="cuda"), max_rows=m, parent=parents,
                           draft_probs=q.expand(S * m, n).contiguous() if drafts else None)
    assert set(acc.tolist()) == {0, 1}
    drafted = tokens.view(S, m).gather(1, path[:, 1:2].clamp(min=0).long())[:, 0]
    first = torch.where(acc > 0, drafted, nxt)
    got = torch.bincount(first.long(), minlength=n).cpu().numpy()
    if not drafts:  # drafts drawn at random all the same: what is emitted has the target's distribution for any drafts
        pass
    assert (np.abs(got - S * target) <= 5.5 * np.sqrt(S * target * (1 - target))).all()


# ------------------------------------------------------------------ kept paths

def _same_cache(raw, c):
    """Equal bytes, but for the payload of a scale that is NaN."""
    got = raw.cpu().numpy().reshape(c.raw.shape)
    codes = 2 * c.page * c.dim
    scales = slice(codes, codes + 8 * (c.page // 16))
    a, b = (np.ascontiguousarray(x[:, :, scales]).view(np.float32) for x in (got, c.raw))
    assert np.array_equal(got[:, :, :codes], c.raw[:, :, :codes]) and np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("page,n_kv,dim", [(16, 1, 64), (48, 3, 96), (64, 2, 128), (32, 2, 192), (16, 2, 256)])
def test_keep(cuda_lib, page, n_kv, dim):
    # bit for bit: paths of every kind, across blocks and pages
    rng = np.random.default_rng(page + dim)
    old = [0, 5, 31, 16, 100, 47, 7, 20, 3]
    new = [1, 20, 64, 9, 40, 33, 64, 12, 30]
    lens = [a + b for a, b in zip(old, new)]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    paths = [[0], [0, 3, 19], [0] + list(range(30, 64)), list(range(9)), [0, 39], [32], [0, 1, 2, 3, 4, 50, 51, 63], [4, 5, 6], [0, 2, 29]]
    width = 40
    p = np.full((9, width), -1)
    for s, x in enumerate(paths):
        p[s, :len(x)] = x
    acc = [len(x) - 1 for x in paths]
    acc[7] = -1                      # nothing kept
    p[8, 1:3] = [5, 5]               # not growing: the path ends before the second 5
    dref.keep(c, table, lens, _cu(new), p.tolist(), acc)
    cuda_lib.kv_keep(raw, _i32(table), _i32(lens), _i32(_cu(new)), _i32(p), _i32(acc), n_kv, dim, page)
    _same_cache(raw, c)


def test_keep_paths_that_are_none(cuda_lib):
    # nodes past the new tokens or before the first, more accepted than the path has, more new tokens than there are, missing pages
    rng = np.random.default_rng(11)
    page, n_kv, dim = 16, 2, 64
    lens, new = [40, 40, 40, 20, 60, 60], [10, 10, 10, 30, 40, 40]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    p = [[0, 3, 10, 4], [-1, 2, 3, 4], [1, 3, 5, 9], [0, 1, 2, 3], [0, 20, 21, 39], [0, 5, 6, 7]]
    acc = [3, 3, 100, 3, 3, 3]
    table[4, 2] = -1   # a source
    table[5, 1] = 77   # a destination
    dref.keep(c, table, lens, _cu(new), p, acc)
    cuda_lib.kv_keep(raw, _i32(table), _i32(lens), _i32(_cu(new)), _i32(p), _i32(acc), n_kv, dim, page)
    _same_cache(raw, c)


def test_keep_scales_that_are_zero_or_nan(cuda_lib):
    rng = np.random.default_rng(12)
    page, n_kv, dim = 16, 1, 128
    lens, new = [40, 40, 40], [30, 30, 30]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    for s, value in enumerate((0.0, np.nan, 1e30)):
        c._scales(table[s, 1], 0, 0)[0] = value
    c._scales(table[0, 0], 0, 1)[0] = c._scales(table[0, 1], 0, 1)[0] = 0.0
    raw = _t(c.raw.reshape(raw.shape))
    p = [[0, 8, 9, 25]] * 3
    dref.keep(c, table, lens, _cu(new), p, [3] * 3)
    cuda_lib.kv_keep(raw, _i32(table), _i32(lens), _i32(_cu(new)), _i32(p), _i32([3] * 3), n_kv, dim, page)
    _same_cache(raw, c)


# ------------------------------------------------------------------ many tokens, many rows: the kernels that large calls take

# A warp keeps its tokens from 6 new tokens of a sequence and 160 of the batch on.
ROPE_MANY = [
    ([0, 3, 17, 40], [64, 9, 33, 50], 5, 3, 64, 16, "f32", 64, False, True, "tree"),
    ([0, 3, 17, 40], [64, 0, 33, 1], 9, 2, 96, 48, "bf16", 96, True, True, "forest"),
    ([7, 3, 15], [60, 64, 64], 17, 1, 128, 16, "f16", 56, False, True, "star"),
    ([100, 31, 0], [64, 64, 40], 2, 9, 192, 64, "f32", 8, True, False, "tree"),
    ([100, 31, 0], [64, 64, 40], 8, 2, 256, 32, "bf16", 256, False, True, "chain"),
    ([1, 2, 3, 4, 5] * 8, [6, 1, 0, 5, 3] * 8, 24, 8, 128, 64, "f32", 128, False, True, None),
    ([160, 2], [161, 1], 0, 2, 64, 16, "bf16", 64, False, True, None),
    ([15], [162], 1, 1, 64, 16, "f16", 0, False, False, None),
]


@pytest.mark.parametrize("old,new,heads,n_kv,dim,page,dtype,turned,interleaved,norm,kind", ROPE_MANY)
def test_append_rope_of_many_tokens(cuda_lib, old, new, heads, n_kv, dim, page, dtype, turned, interleaved, norm, kind):
    rng = np.random.default_rng(sum(old) + dim + heads)
    if heads == 0:  # keys and values alone: as with one head of queries
        r = [_append_rope(cuda_lib, np.random.default_rng(5), old, new, h, n_kv, dim, page, dtype, turned, interleaved, norm, kind)
             for h in (1,)][0]
        raw, _, _ = _filled(np.random.default_rng(5), old, page, n_kv, dim, n_pages=r["raw"].shape[0])
        cuda_lib.kv_append_rope(raw, _i32(r["table"]), _i32(r["lens"]), None, None, r["k"], r["v"], 0, n_kv, dim, page, _t(r["freqs"]),
                                interleaved, None, _t(r["kw"]), 1e-6, cu_new=_i32(r["cu"]), max_new=max(new))
        assert np.array_equal(raw.cpu().numpy(), r["raw"].cpu().numpy())
        return
    r = _append_rope(cuda_lib, rng, old, new, heads, n_kv, dim, page, dtype, turned, interleaved, norm, kind)
    _check_rope(r, old, new, n_kv, dim, page, dtype, interleaved)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_rope_of_many_tokens_is_that_of_few(cuda_lib, dim):
    # one batch at once, and its sequences one by one (other kernels): the cache bit for bit, missing pages, a sequence that has
    # more new tokens than tokens and nodes without a parent among them
    import torch
    rng = np.random.default_rng(dim)
    heads, n_kv, page, seqs, m = 6, 2, 16, 8, 24
    old = [int(x) for x in rng.integers(0, 60, seqs)]
    lens = [x + m for x in old]
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    lens[3] = m - 1
    table[4, (old[4] + m - 1) // page] = -1
    parents = np.concatenate([_parents(rng, m) for _ in range(seqs)]).astype(np.int32)
    parents[5 * m + 10] = 12
    parents[6 * m + 3] = -2
    q, k, v = (_t(rng.standard_normal((seqs * m, h, dim)).astype(np.float32)) for h in (heads, n_kv, n_kv))
    freqs, w = _t((10000.0 ** (-np.arange(dim // 2) * 2 / dim)).astype(np.float32)), _t(rng.uniform(0.5, 1.5, dim).astype(np.float32))
    whole, single = raw.clone(), raw.clone()
    outs = [torch.full_like(q, 5.0) for _ in range(2)]
    cuda_lib.kv_append_rope(whole, _i32(table), _i32(lens), q, outs[0], k, v, heads, n_kv, dim, page, freqs, q_weight=w, k_weight=w,
                            cu_new=_i32(np.arange(seqs + 1) * m), max_new=m, parent=_i32(parents))
    for s in range(seqs):
        at = slice(s * m, s * m + m)
        cuda_lib.kv_append_rope(single, _i32(table[s:s + 1]), _i32(lens[s:s + 1]), q[at], outs[1][at], k[at], v[at], heads, n_kv, dim, page,
                                freqs, q_weight=w, k_weight=w, cu_new=_i32([0, m]), max_new=m, parent=_i32(parents[at]))
    assert torch.isnan(outs[0][3 * m:4 * m]).all() and torch.isnan(outs[0][5 * m + 10]).all() and torch.isnan(outs[0][6 * m + 3]).all()
    assert torch.equal(torch.isnan(outs[0]), torch.isnan(outs[1])) and torch.equal(outs[0].nan_to_num(), outs[1].nan_to_num())
    _same_cache(whole, ref.Cache(single.cpu().numpy(), page, n_kv, dim))


# The walk reads the rows that it reaches where 128 MiB of logits could be rows (a bound by max_rows); more than two CTAs to
# an SM at 8 to a sequence make it 4.
VERIFY_MANY = [
    ([5, 9, 64, 1, 0, 6, 20, 3, 2, 7, 4, 30], 60001, "tree", True, 1.0, "f32"),
    ([5, 9, 64, 1, 0, 6, 20, 3, 2, 7, 4, 30], 120003, "tree", False, 0.8, "bf16"),
    ([40, 9, 33, 1, 0, 6, 20, 3, 2, 7, 4, 30], 120000, "star", True, 1.0, "f16"),
    ([40, 9, 33, 1, 0, 6, 20, 3, 2, 7, 4, 30], 90000, "star", False, 1.0, "f32"),
    ([5, 9, 64, 1, 0, 6, 20, 3, 2, 7, 4, 30], 100001, "tree", True, 0.0, "bf16"),
    ([3, 1, 2, 0, 5] * 9 + [40], 30001, "chain", True, 1.0, "f32"),
    ([3, 1, 2, 0, 5] * 9 + [40], 40001, "tree", False, 1.0, "f16"),
    ([3, 1, 2, 0, 5] * 9 + [40], 30007, "tree", False, 0.0, "f32"),
    ([3, 1, 2, 0, 5] * 9, 20001, "chain", True, 1.0, "f32"),
    ([3, 1, 2, 0, 5] * 9, 18001, "tree", True, 1.2, "bf16"),
]


@pytest.mark.parametrize("nodes,n,kind,drafts,temperature,dtype", VERIFY_MANY)
def test_verify_many_rows(cuda_lib, nodes, n, kind, drafts, temperature, dtype):
    rng = np.random.default_rng(n)
    w = _problem(rng, nodes, n, kind, drafts, temperature, dtype)
    _check_verify(w, _verify(cuda_lib, w))


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_verify_many_rows_that_are_not_finite(cuda_lib, temperature):
    # a NaN, +inf or a row of -inf at the root, at a draft that is reached and at one that is not
    import torch
    rng = np.random.default_rng(3)
    seqs, m, n = 40, 21, 45000
    x = torch.randn(seqs * m, n, device="cuda")
    tokens = rng.integers(0, n, seqs * m)
    for s in range(seqs):
        x[s * m, tokens[s * m + 1]] = 60.0  # the first draft is accepted
    x[0, 44999] = float("nan")
    x[m, 0] = float("inf")
    x[2 * m] = float("-inf")
    x[3 * m + 1, 30000] = float("nan")
    x[4 * m + 1] = float("-inf")
    x[5 * m + 2] = float("nan")
    parents = np.tile(np.concatenate([[-1, 0], np.zeros(m - 2, int)]), (seqs, 1))
    w = dict(x=x, tokens=tokens, parents=list(parents), u=rng.random(seqs * m).astype(np.float32), probs=None, cu=_cu([m] * seqs),
             nodes=[m] * seqs, n=n, temperature=temperature, kind="tree")
    acc, path, nxt = _verify(cuda_lib, w)
    assert acc.tolist() == [0, 0, 0] + [1] * (seqs - 3)
    assert (nxt[:5] == -1).all() and (nxt[5:] >= 0).all() and (nxt < n).all()
    assert (path[:3, 1:] == -1).all() and (path[3:, 1] == 1).all()


def test_verify_many_rows_by_either_way(cuda_lib):
    # rows past the sequences' own make the bound large: the same problem read at once and row by row, with masked logits
    import torch
    rng = np.random.default_rng(9)
    w = _problem(rng, [6, 3, 9, 12, 1, 7], 50000, "tree", True, 1.0, "f32")
    w["x"][:, rng.choice(50000, 20000, replace=False)] = torch.finfo(torch.float32).min
    w["x"][:, 7::11] = float("-inf")
    few, many = _verify(cuda_lib, w), _verify(cuda_lib, w, max_rows=64)
    assert 6 * 64 * 50000 * 4 <= 128 << 20 < 12 * 64 * 50000 * 4
    w2 = dict(w, nodes=w["nodes"] * 2, parents=w["parents"] * 2, cu=_cu(w["nodes"] * 2), tokens=np.tile(w["tokens"], 2), u=np.tile(w["u"], 2),
              x=w["x"].repeat(2, 1), probs=np.tile(w["probs"], (2, 1)))
    lazy = _verify(cuda_lib, w2, max_rows=64)
    for a, b in ((few[0], many[0]), (few[2], many[2]), (np.tile(few[0], 2), lazy[0]), (np.tile(few[2], 2), lazy[2]),
                 (np.tile(many[1], (2, 1)), lazy[1])):
        assert np.array_equal(a, b)


def test_verify_replayed_graphs_share_a_workspace(cuda_lib):
    # clusters and all rows at once, captured into graphs with one workspace, replayed in turns with other inputs
    import torch
    rng = np.random.default_rng(77)
    shapes = [([6, 3, 9, 12], 40000, True, 12), ([6, 3, 9, 12, 1, 7] * 2, 50000, False, 64), ([5] * 40, 20001, True, 5), ([4, 7], 3001, True, 7)]
    first, second = ([_problem(rng, nodes, n, "tree", drafts, 1.0, "f32") for nodes, n, drafts, _ in shapes] for _ in range(2))
    ws = torch.zeros(max(cuda_lib.verify_drafts_workspace_bytes(len(x[0]), x[3], x[1]) for x in shapes), dtype=torch.uint8, device="cuda")
    runs = []
    for w, x in zip(first, shapes):
        seqs = len(x[0])
        acc, path, nxt = (torch.full(shape, -9, dtype=torch.int32, device="cuda") for shape in ((seqs,), (seqs, x[3]), (seqs,)))
        ins = dict(x=w["x"].clone(), tokens=_i32(w["tokens"]), u=_t(w["u"]), parent=_i32(np.concatenate(w["parents"])),
                   probs=None if w["probs"] is None else _t(w["probs"]))

        def call(ins=ins, acc=acc, path=path, nxt=nxt, w=w, x=x, cu=_i32(w["cu"])):
            cuda_lib.verify_drafts(ins["x"], ins["tokens"], ins["u"], acc, path, nxt, x[1], ws, cu=cu, max_rows=x[3], parent=ins["parent"],
                                   draft_probs=ins["probs"])

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, ins, (acc, path, nxt), call))  # (the call holds cu)
    for problems in (second, first):
        for (_, ins, outs, _), w in zip(runs, problems):
            ins["x"].copy_(w["x"])
            ins["tokens"].copy_(_i32(w["tokens"]))
            ins["u"].copy_(_t(w["u"]))
            ins["parent"].copy_(_i32(np.concatenate(w["parents"])))
            if ins["probs"] is not None:
                ins["probs"].copy_(_t(w["probs"]))
            for t in outs:
                t.fill_(-9)
        for graph, _, _, _ in runs:
            graph.replay()
        torch.cuda.synchronize()
        for (_, _, outs, _), w in zip(runs, problems):
            _check_verify(w, tuple(_np(t) for t in outs))


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_drafted_tokens(cuda_lib, dtype, graph):
    """Append with rotation, tree attention, verification and the kept path as one step, eager or replayed from a graph.

    After each step the sequences go on from the accepted path, so the cache's tokens, seen in order, are those of an
    undrafted run: the kept keys are the given ones at their positions (within the steps of the scales they went through),
    a row of the tree equals the row of causal attention over its line, and the next step appends behind them."""
    import torch
    rng = np.random.default_rng(21)
    heads, n_kv, dim, page, n = 6, 2, 64, 16, 700
    seqs, m, steps = 3, 9, 3
    old = [30, 1, 15]
    raw, table, c = _filled(rng, old, page, n_kv, dim, n_pages=30)
    table = np.arange(30).reshape(3, 10).astype(np.int32)
    raw = torch.zeros(30, n_kv, ref.record_bytes(page, dim), dtype=torch.uint8, device="cuda")
    dt = _dt(dtype)
    freqs = _t((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    first = [torch.randn(sum(old), x, dim, device="cuda").to(dt) for x in (n_kv, n_kv)]
    cuda_lib.kv_append_rope(raw, _i32(table), _i32(old), None, None, *first, 0, n_kv, dim, page, freqs, cu_new=_i32(_cu(old)), max_new=30)
    kv_len = _i32([x + m for x in old])
    parents = np.array([-1, 0, 0, 1, 1, 3, 2, 6, 5])
    par, cu, tab = _i32(np.tile(parents, seqs)), _i32(np.arange(seqs + 1) * m), _i32(table)
    f = lambda h: torch.empty(seqs * m, h, dim, device="cuda", dtype=dt)  # noqa: E731
    q, k, v, qo, out = f(heads), f(n_kv), f(n_kv), f(heads), f(heads)
    lse = torch.empty(seqs * m, heads, device="cuda")
    logits, u = torch.empty(seqs * m, n, device="cuda"), torch.empty(seqs * m, device="cuda")
    tokens = torch.empty(seqs * m, dtype=torch.int32, device="cuda")
    acc, path, nxt = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((seqs,), (seqs, m), (seqs,)))
    ws = cuda_lib.kv_attention_workspace(seqs, m, 160, heads, n_kv, dim)
    vws = cuda_lib.verify_drafts_workspace(seqs, m, n)

    def step():
        cuda_lib.kv_append_rope(raw, tab, kv_len, q, qo, k, v, heads, n_kv, dim, page, freqs, cu_new=cu, max_new=m, parent=par)
        cuda_lib.kv_tree_attention(raw, tab, kv_len, qo, out, ws, heads, n_kv, dim, page, 160, cu, m, par, lse=lse)
        cuda_lib.verify_drafts(logits, tokens, u, acc, path, nxt, n, vws, cu=cu, max_rows=m, parent=par)
        cuda_lib.kv_keep(raw, tab, kv_len, cu, path, acc, n_kv, dim, page)
        kv_len.add_(acc + 1)  # behind the kept tokens and the next step's

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
        tokens.copy_(torch.randint(0, n, tokens.shape, device="cuda", generator=g))
        # the drafts on the way 0, 1, 3, 5, 8 are the likely tokens
        for s in range(seqs):
            for a, b in ((0, 1), (1, 3), (3, 5), (5, 8)):
                logits[s * m + a, tokens[s * m + b].long()] = 9.0
        u.copy_(torch.rand(u.shape, device="cuda", generator=g))

    replay = None
    if graph:
        keep_raw, keep_len = raw.clone(), kv_len.clone()
        fill(0)
        step()
        torch.cuda.synchronize()
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            step()
        raw.copy_(keep_raw)
        kv_len.copy_(keep_len)
    lengths = list(old)
    truth = [[list(_np(first[w])[_cu(old)[s]:_cu(old)[s + 1]]) for s in range(seqs)] for w in range(2)]
    total = 0
    for t in range(steps):
        fill(t)
        before = raw.clone()
        replay.replay() if graph else step()
        torch.cuda.synchronize()
        a, p = _np(acc), _np(path)
        total += a.sum()
        cache = ref.Cache(raw.cpu().numpy(), page, n_kv, dim)
        for s in range(seqs):
            rows = [s * m + x for x in p[s][:a[s] + 1]]
            want, tok, margin = dref.verify(_np(logits)[s * m:(s + 1) * m], _np(tokens)[s * m:(s + 1) * m], list(parents), _np(u)[s * m:(s + 1) * m], None, 1.0)
            assert margin > MARGIN and [x - s * m for x in rows] == want and _np(nxt)[s] == tok
            # the tree's rows against causal attention over their line, in float64 from the cache as it was
            whole = before.clone()
            cuda_lib.kv_append_rope(whole, tab[s:s + 1], _i32([lengths[s] + m]), q[s * m:(s + 1) * m], torch.empty_like(q[:m]),
                                    k[s * m:(s + 1) * m], v[s * m:(s + 1) * m], heads, n_kv, dim, page, freqs, cu_new=_i32([0, m]),
                                    max_new=m, parent=_i32(parents))
            kk, vv = _values(ref.Cache(whole.cpu().numpy(), page, n_kv, dim), table, s, lengths[s] + m)
            for i in range(m):
                line = list(range(lengths[s])) + [lengths[s] + x for x in dref.line(list(parents), i)]
                o, l, av, mag, z = ref.attention(_np(qo)[s * m + i][None], kk[line], vv[line], np.array([len(line) - 1]), dim ** -0.5)
                d = 2.0 ** -18 * mag + 2.0 ** -20
                bound = (2 * d + 2.0 ** -17 + 2.0 ** -11)[..., None] * av + EPS[dtype] * np.abs(o) + 2.0 ** -39 * len(line) * z[..., None]
                _within(_np(out)[s * m + i][None], o, bound)
            for w, x in ((0, k), (1, v)):
                truth[w][s] += list(_np(x)[rows])
            lengths[s] += len(rows)
            got = _values(cache, table, s, lengths[s])
            pos = np.arange(lengths[s])
            keys = dref.norm_turn(np.array(truth[0][s]), None, 0, pos, _np(freqs), False)[0]
            for w, y in ((0, keys), (1, np.array(truth[1][s]))):
                for b in range(0, lengths[s], 16):
                    for h in range(n_kv):
                        sc = float(cache._scales(table[s, b // page], h, w)[b % page // 16])
                        # half a step for the first rounding and for each of up to `steps` times that a block's scale grew or a
                        # token moved (twice a step), at steps not above the last one
                        assert np.abs(got[w][b:b + 16, h] - y[b:b + 16, h]).max() <= sc * (0.5 * (1 + 2 * steps) + 0.01)
    assert total > 0 and _np(kv_len).tolist() == [x + m for x in lengths]
    assert cuda_lib.pipeline_timeouts() == 0


def test_calls_on_other_streams(cuda_lib):
    # two streams with workspaces of their own at once, and a stream that waits for what wrote its inputs
    import torch
    rng = np.random.default_rng(31)
    w = [_problem(rng, [6] * 30, 20000, "tree", i == 0, 1.0, "f32") for i in range(2)]
    want = [_verify(cuda_lib, x) for x in w]
    streams = [torch.cuda.Stream() for _ in w]
    args = []
    for x in w:
        acc, path, nxt = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((30,), (30, 6), (30,)))
        args.append((x["x"], _i32(x["tokens"]), _t(x["u"]), acc, path, nxt, 20000, cuda_lib.verify_drafts_workspace(30, 6, 20000),
                     _i32(x["cu"]), 6, _i32(np.concatenate(x["parents"])), None if x["probs"] is None else _t(x["probs"])))
    torch.cuda.synchronize()
    for _ in range(5):
        for a, st in zip(args, streams):
            with torch.cuda.stream(st):
                cuda_lib.verify_drafts(*a)
    torch.cuda.synchronize()
    for a, (acc, path, nxt) in zip(args, want):
        assert np.array_equal(_np(a[3]), acc) and np.array_equal(_np(a[4]), path) and np.array_equal(_np(a[5]), nxt)
