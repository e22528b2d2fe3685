"""Refusals and sizes of the operators of drafted tokens (no GPU: fake, never dereferenced addresses), and their oracle."""
import numpy as np
import pytest

from oracle import decode_oracle as ref
from oracle import draft_oracle as dref
from test_decode_ops_host import _at, qdq  # noqa: F401


def test_append_rope_refusals(qdq):  # noqa: F811
    f = qdq.lib().qdq_kv_append_rope
    p, t, ln, cu, par, q, o, k, v, qw, kw, fr = (_at(i) for i in range(12))

    def call(p=p, n_pages=4, page=16, n_kv=2, dim=64, t=t, width=3, ln=ln, cu=cu, par=par, seqs=2, most=5, heads=4, q=q, qs=256, o=o, os=256,
             k=k, ks=128, v=v, vs=128, qw=qw, kw=kw, eps=1e-6, fr=fr, n_rot=64, inter=0, type=0):
        return f(p, n_pages, page, n_kv, dim, t, width, ln, cu, par, seqs, most, heads, q, qs, o, os, k, ks, v, vs, qw, kw, eps, fr, n_rot, inter,
                 type, None)

    for name in ("p", "t", "ln", "k", "v", "q", "o"):
        assert call(**{name: None}) == qdq.QDQ_ERR_NULL, name
    for bad in (dict(n_pages=0), dict(page=24), dict(n_kv=0), dict(width=0), dict(seqs=-1), dict(most=-1), dict(cu=None), dict(heads=-1),
                dict(eps=-1.0), dict(eps=float("nan")), dict(type=3), dict(n_rot=0), dict(n_rot=12), dict(n_rot=72), dict(n_rot=-8),
                dict(inter=2), dict(qs=255), dict(os=128), dict(ks=64), dict(vs=127)):
        assert call(**bad) == qdq.QDQ_ERR_DIMS, bad
    for bad in (dict(dim=80), dict(most=65), dict(page=1 << 17)):
        assert call(**bad) == qdq.QDQ_ERR_UNSUPPORTED, bad
    for bad in (dict(p=p + 64), dict(t=t + 2), dict(ln=ln + 1), dict(cu=cu + 2), dict(par=par + 1), dict(fr=fr + 2), dict(qw=qw + 4),
                dict(kw=kw + 8), dict(q=q + 8), dict(o=o + 4), dict(k=k + 2), dict(qs=258), dict(vs=130)):
        assert call(**bad) == qdq.QDQ_ERR_ALIGN, bad
    for bad in (dict(o=k), dict(o=v), dict(k=p), dict(o=p), dict(o=q + 16), dict(o=q, os=512), dict(ln=p), dict(cu=p), dict(par=p + 128),
                dict(o=qw), dict(fr=o), dict(kw=p), dict(q=p)):
        assert call(**bad) == qdq.QDQ_ERR_ALIAS, bad
    # nothing to do: whatever the addresses; other arguments are still checked
    for nothing in (dict(seqs=0), dict(most=0)):
        assert call(p=None, t=None, ln=None, k=None, v=None, q=None, o=None, **nothing) == qdq.QDQ_OK
        assert call(n_rot=12, **nothing) == qdq.QDQ_ERR_DIMS
    assert call(seqs=0, n_rot=12, fr=None) == qdq.QDQ_OK           # nothing is turned: n_rot does not count
    assert call(seqs=0, heads=0, q=None, o=None, qs=0, os=0) == qdq.QDQ_OK
    assert call(most=0, par=None, cu=None) == qdq.QDQ_ERR_DIMS     # one token each: max_new 1
    assert call(seqs=0, most=1000, par=None) == qdq.QDQ_OK         # more than a tree's nodes without parents


def test_tree_attention_refusals(qdq):  # noqa: F811
    f = qdq.lib().qdq_kv_tree_attention
    p, t, ln, cu, par, q, o, lse, sl, ws = (_at(i) for i in range(10))

    def call(p=p, page=16, dim=64, t=t, ln=ln, cu=cu, par=par, seqs=2, most=5, kv=48, heads=4, q=q, qs=256, o=o, os=256, lse=lse, sl=sl,
             scale=0.125, cap=0.0, window=0, type=0, ws=ws, wb=0):
        return f(p, 4, page, 2, dim, t, 3, ln, cu, par, seqs, most, kv, heads, q, qs, o, os, lse, sl, scale, cap, window, type, ws, wb, None)

    for name in ("p", "t", "ln", "cu", "par", "q", "o", "ws"):
        assert call(**{name: None}) == qdq.QDQ_ERR_NULL, name
    for bad in (dict(most=-1), dict(heads=3), dict(window=-1), dict(cap=-1.0), dict(scale=float("inf")), dict(type=5), dict(qs=64), dict(kv=-1)):
        assert call(**bad) == qdq.QDQ_ERR_DIMS, bad
    for bad in (dict(most=65), dict(dim=72), dict(kv=qdq.QDQ_MAX_KV_LEN + 1)):
        assert call(**bad) == qdq.QDQ_ERR_UNSUPPORTED, bad
    for bad in (dict(par=par + 2), dict(q=q + 4), dict(ws=ws + 128), dict(lse=lse + 1)):
        assert call(**bad) == qdq.QDQ_ERR_ALIGN, bad
    for bad in (dict(par=o), dict(par=ws, wb=64), dict(q=o), dict(lse=o)):
        assert call(**bad) == qdq.QDQ_ERR_ALIAS, bad
    for nothing in (dict(seqs=0), dict(most=0)):
        assert call(p=None, t=None, ln=None, cu=None, par=None, q=None, o=None, ws=None, **nothing) == qdq.QDQ_OK


def test_verify_refusals(qdq):  # noqa: F811
    f = qdq.lib().qdq_verify_drafts
    x, tok, cu, par, dp, u, acc, path, nxt, ws = (_at(i) for i in range(10))
    need = qdq.verify_drafts_workspace_bytes(3, 5, 1000)

    def call(x=x, stride=1000, type=0, tok=tok, cu=cu, par=par, seqs=3, rows=5, n=1000, dp=dp, ds=1000, u=u, temp=1.0, acc=acc, path=path,
             nxt=nxt, ws=ws, wb=need - 1):
        return f(x, stride, type, tok, cu, par, seqs, rows, n, dp, ds, u, temp, acc, path, nxt, ws, wb, None)

    for name in ("x", "tok", "u", "acc", "path", "nxt", "ws"):
        assert call(**{name: None}) == qdq.QDQ_ERR_NULL, name
    for bad in (dict(type=-1), dict(seqs=-1), dict(rows=0), dict(n=0), dict(stride=999), dict(ds=999), dict(cu=None), dict(temp=-1.0),
                dict(temp=float("nan")), dict(temp=1e-7), dict(temp=float("inf"))):
        assert call(**bad) == qdq.QDQ_ERR_DIMS, bad
    assert call(rows=65) == qdq.QDQ_ERR_UNSUPPORTED
    assert call(n=(1 << 30) + 1, stride=1 << 31, ds=1 << 31) == qdq.QDQ_ERR_UNSUPPORTED
    for bad in (dict(x=x + 2), dict(tok=tok + 1), dict(cu=cu + 2), dict(par=par + 3), dict(dp=dp + 1), dict(u=u + 2), dict(acc=acc + 2),
                dict(path=path + 1), dict(nxt=nxt + 2), dict(ws=ws + 16)):
        assert call(**bad) == qdq.QDQ_ERR_ALIGN, bad
    for bad in (dict(acc=nxt), dict(path=x), dict(nxt=tok), dict(acc=cu + 4), dict(ws=dp), dict(path=u), dict(acc=par)):
        assert call(**bad) == qdq.QDQ_ERR_ALIAS, bad
    assert call() == qdq.QDQ_ERR_SCRATCH
    assert call(x=None, tok=None, u=None, acc=None, path=None, nxt=None, ws=None, seqs=0) == qdq.QDQ_OK
    assert call(u=None, temp=0.0) == qdq.QDQ_ERR_SCRATCH     # the best token: no numbers needed
    assert call(tok=None, rows=1) == qdq.QDQ_ERR_SCRATCH     # no drafts


def test_verify_workspace(qdq):  # noqa: F811
    f = qdq.verify_drafts_workspace_bytes
    assert f(0, 1, 10) == f(1, 0, 10) == f(1, 65, 10) == f(1, 1, 0) == f(1, 1, (1 << 30) + 1) == 0
    for n in (1, 1017, 1018, 1024, 128256, 1 << 30):
        for seqs, rows in ((1, 1), (3, 64)):
            chunks = -(-(n + 7) // 1024)
            b = f(seqs, rows, n)
            assert b % 256 == 0 and b - b // 8 // 256 * 256 >= seqs * chunks * (8 * rows + 4)


def test_keep_refusals(qdq):  # noqa: F811
    f = qdq.lib().qdq_kv_keep
    p, t, ln, cu, path, acc = (_at(i) for i in range(6))

    def call(p=p, n_pages=4, page=16, n_kv=2, dim=64, t=t, width=3, ln=ln, cu=cu, seqs=2, path=path, stride=5, acc=acc):
        return f(p, n_pages, page, n_kv, dim, t, width, ln, cu, seqs, path, stride, acc, None)

    for name in ("p", "t", "ln", "cu", "path", "acc"):
        assert call(**{name: None}) == qdq.QDQ_ERR_NULL, name
    for bad in (dict(n_pages=0), dict(page=8), dict(n_kv=0), dict(width=0), dict(seqs=-1), dict(stride=0)):
        assert call(**bad) == qdq.QDQ_ERR_DIMS, bad
    assert call(dim=48) == qdq.QDQ_ERR_UNSUPPORTED
    for bad in (dict(p=p + 16), dict(t=t + 1), dict(ln=ln + 2), dict(cu=cu + 2), dict(path=path + 1), dict(acc=acc + 3)):
        assert call(**bad) == qdq.QDQ_ERR_ALIGN, bad
    for bad in (dict(acc=p), dict(path=p), dict(cu=p + 64), dict(ln=p), dict(t=p)):
        assert call(**bad) == qdq.QDQ_ERR_ALIAS, bad
    assert call(p=None, t=None, ln=None, cu=None, path=None, acc=None, seqs=0) == qdq.QDQ_OK


def _short_calls(qdq, device):  # noqa: F811
    """Calls whose tensors are right but for one that holds less than the call reads or writes."""
    import torch

    def f(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)

    def i(*shape):
        return f(*shape, dtype=torch.int32)

    pages, table, ws = f(3, 2176, dtype=torch.uint8), i(2, 1), f(1 << 22, dtype=torch.uint8)

    def rope(n=i(2), q=f(2, 128), o=f(2, 128), k=f(2, 64), v=f(2, 64), qw=f(64), kw=f(64), cu=None, par=None):
        qdq.kv_append_rope(pages, table, n, q, o, k, v, 2, 1, 64, 16, f(32), False, qw, kw, cu_new=cu, parent=par)

    def tree(n=i(2), q=f(2, 128), o=f(2, 128), cu=i(3), sl=f(2), ws=ws):
        qdq.kv_tree_attention(pages, table, n, q, o, ws, 2, 1, 64, 16, 16, cu, 1, i(2), slopes=sl)

    def verify(x=f(2, 64), tok=i(2), u=f(2), acc=i(2), path=i(2, 1), nxt=i(2), cu=None, dp=f(2, 64), par=None, ws=ws):
        qdq.verify_drafts(x, tok, u, acc, path, nxt, 64, ws, cu=cu, draft_probs=dp, parent=par)

    def keep(n=i(2), cu=i(3), path=i(2, 3), acc=i(2)):
        qdq.kv_keep(pages, table, n, cu, path, acc, 1, 64, 16)

    wide = f(1 << 22, 2, dtype=torch.uint8)[:, 0]
    return {rope: dict(n=i(1), q=f(1, 128), o=f(2, 64), k=f(1, 64), v=f(2, 32), qw=f(63), kw=f(32), cu=i(2), par=i(1)),
            tree: dict(n=i(1), q=f(2, 64), o=f(2, 64), cu=i(2), sl=f(1), ws=wide),
            verify: dict(x=f(1, 64), tok=i(1), u=f(1), path=i(1, 1), nxt=i(1), cu=i(2), dp=f(2, 63), par=i(1), ws=wide),
            keep: dict(n=i(1), cu=i(2), path=i(1, 3), acc=i(1))}


def test_binding_refuses_short_tensors(qdq, monkeypatch):  # noqa: F811
    monkeypatch.setattr(qdq, "_cuda", lambda name, t: None if t is None else t.data_ptr())
    for call, short in _short_calls(qdq, "cpu").items():
        for name, tensor in short.items():
            with pytest.raises(ValueError, match="expected"):
                call(**{name: tensor})


def test_binding_refuses_other_types(qdq):  # noqa: F811
    import torch
    x, i = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        qdq.verify_drafts(x.double(), i, x[:, 0], i, i[:, None], i, 64, x)
    with pytest.raises(TypeError):
        qdq.verify_drafts(x, i.long(), x[0, :2], i, i[:, None].contiguous(), i, 64, x)
    with pytest.raises(TypeError):
        qdq.kv_keep(torch.zeros(3, 2176, dtype=torch.uint8), torch.zeros(2, 1), i, i, i[:, None], i, 1, 64, 16)


@pytest.mark.gpu
def test_binding_refuses_short_tensors_of_the_device(cuda_lib):
    # whole tensors run; short ones are refused as on the host, by the ordinary path too
    import torch
    for call, short in _short_calls(cuda_lib, "cuda").items():
        call()
        for name, tensor in short.items():
            with pytest.raises(ValueError, match="expected"):
                call(**{name: tensor})
    torch.cuda.synchronize()


# ------------------------------------------------------------------ the oracle itself

def test_oracle_rotation():
    x = np.array([[[3.0, 4.0, 1.0, 2.0, 7.0, 9.0]]])
    quarter = np.array([np.pi / 2, np.pi])
    y, _ = dref.norm_turn(x, None, 0, [1], quarter, True)
    assert np.allclose(y, [[[-4, 3, -1, -2, 7, 9]]])
    y, _ = dref.norm_turn(x, None, 0, [1], quarter, False)
    assert np.allclose(y, [[[-1, -4, 3, -2, 7, 9]]])
    assert np.allclose(dref.norm_turn(x, np.full(6, 2.0), 0, [0], quarter, True)[0], 2 * x / np.sqrt((x * x).mean()))


def test_oracle_trees():
    assert dref.depths([-1, 0, 0, 2, 9, 4, -1, 6]).tolist() == [0, 1, 1, 2, -1, -1, 0, 1]
    assert dref.line([-1, 0, 0, 2], 3) == [0, 2, 3]
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    a = dref.tree_attention(q, k, v, [-1, 0, 1, 2, 3], 0.3, 0, 4, np.array([0.1, 0.2]))
    b = ref.attention(q, k, v, np.arange(4, 9), 0.3, 0, 4, np.array([0.1, 0.2]))
    for x, y in zip(a, b):
        assert np.allclose(x, y)
    alone = dref.tree_attention(q[:2], k[-2:], v[-2:], [-1, -1], 0.3)[0]
    assert np.allclose(alone, v[-2:])  # two roots and nothing before them: each sees itself


def test_oracle_verification():
    x = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [0.3, 0.3, 0.4]]))
    q = np.array([[0.2, 0.6, 0.2]] * 3)
    # drafted 1 has p / q = 1/2: accepted below it, else w = (0.3, 0, 0) / 0.3
    assert dref.verify(x[:2], [0, 1], [-1, 0], np.array([0.85, 0.49]), q, 1.0)[:2] == ([0, 1], 2)
    assert dref.verify(x[:2], [0, 1], [-1, 0], np.array([0.99, 0.51]), q, 1.0)[:2] == ([0], 0)
    # without probabilities: 1 accepted below 0.3; then 0 below 0.5 / 0.7; then 2 is left
    assert dref.verify(x, [0, 1, 0], [-1, 0, 0], np.array([0.0, 0.31, 0.72]), None, 1.0)[:2] == ([0], 2)
    assert dref.verify(x, [0, 1, 0], [-1, 0, 0], np.array([0.65, 0.31, 0.71]), None, 1.0)[:2] == ([0, 2], 2)
    assert dref.verify(x, [0, 0, 2], [-1, 0, 1], None, None, 0)[:2] == ([0, 1, 2], 2)


def test_oracle_kept_path():
    raw = np.zeros((2, 1, ref.record_bytes(16, 64)), np.uint8)
    c = ref.Cache(raw, 16, 1, 64)
    table = np.array([[1, 0]])
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((20, 1, 64)).astype(np.float32), rng.standard_normal((20, 1, 64)).astype(np.float32)
    c.append(table, [20], [0, 20], k, v)
    before = c.read(table, 0, 0, 20)
    dref.keep(c, table, [20], [0, 10], [[0, 4, 9]], [2])
    after = c.read(table, 0, 0, 13)
    step = np.abs(before).max() / 127
    for a, b in zip(after, before):
        assert np.abs(a - b[list(range(10)) + [10, 14, 19]]).max() <= step
