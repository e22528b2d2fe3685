"""Refusals and sizes of the decode-step operators (no GPU: fake, never dereferenced addresses)."""
import pytest

GOOD = 0x10000000


def _at(i):
    return GOOD + (i << 28)


@pytest.fixture(scope="module")
def qdq():
    from ggml_quantized_dequant_gb300 import _build
    import ggml_quantized_dequant_gb300 as q
    _build.build()
    q.load()
    return q


def test_rms_norm_refusals(qdq):
    f = qdq.lib().qdq_rms_norm
    x, r, w, s, o, q8 = (_at(i) for i in range(6))

    def call(x=x, r=r, w=w, s=s, o=o, q8=q8, type=0, rows=4, n=256, xs=256, rs=256, ss=256, os=256, eps=1e-5):
        return f(x, r, w, s, o, q8, type, rows, n, xs, rs, ss, os, eps, None)

    assert call(x=None) == qdq.QDQ_ERR_NULL
    assert call(o=None, q8=None) == qdq.QDQ_ERR_NULL
    assert call(type=3) == qdq.QDQ_ERR_DIMS
    assert call(rows=-1) == qdq.QDQ_ERR_DIMS
    assert call(n=0) == qdq.QDQ_ERR_DIMS
    assert call(n=250) == qdq.QDQ_ERR_DIMS                      # Q8_0 needs whole blocks
    assert call(xs=255) == qdq.QDQ_ERR_DIMS
    assert call(ss=255) == qdq.QDQ_ERR_DIMS
    assert call(eps=-1.0) == qdq.QDQ_ERR_DIMS
    assert call(eps=float("nan")) == qdq.QDQ_ERR_DIMS
    assert call(n=1 << 16, xs=1 << 16, rs=1 << 16, ss=1 << 16, os=1 << 16) == qdq.QDQ_ERR_UNSUPPORTED
    assert call(x=x + 2) == qdq.QDQ_ERR_ALIGN
    assert call(x=x + 1, type=2) == qdq.QDQ_ERR_ALIGN
    assert call(w=w + 2) == qdq.QDQ_ERR_ALIGN
    assert call(q8=q8 + 8) == qdq.QDQ_ERR_ALIGN
    assert call(o=x + 16) == qdq.QDQ_ERR_ALIAS                   # not exactly x
    assert call(o=x, os=512) == qdq.QDQ_ERR_ALIAS                # x with another stride
    assert call(s=o) == qdq.QDQ_ERR_ALIAS
    assert call(s=w) == qdq.QDQ_ERR_ALIAS
    assert call(q8=x) == qdq.QDQ_ERR_ALIAS
    assert call(rows=0) == qdq.QDQ_OK
    assert call(rows=0, o=x, s=r) == qdq.QDQ_OK                  # in place


def test_rows_that_overlap_by_one_element_are_refused(qdq):
    # slices of one wide buffer that share an element, at either end, and rows of different strides among one another
    n, st = 256, 512
    norm = qdq.lib().qdq_rms_norm
    for off, os in ((n - 1, st), (st - n + 1, st), (-(n - 1), st), (-(st - n + 1), st), (1, st), (n, st + 8)):
        assert norm(_at(0), None, None, None, _at(0) + 4 * off, None, 0, 4, n, st, 0, 0, os, 1e-5, None) == qdq.QDQ_ERR_ALIAS, off
    attend = qdq.lib().qdq_kv_attention
    p, t, ln, q, ws = (_at(i) for i in range(1, 6))
    for off in (252, 260, -252, -260, 4):  # q and out: 256 of 512 elements
        assert attend(p, 4, 16, 2, 64, t, 3, ln, None, 2, 1, 48, 4, q, 512, q + 4 * off, 512, None, None, 0.125, 0.0, 0, 0, ws, 0,
                      None) == qdq.QDQ_ERR_ALIAS, off


def test_nothing_to_do_needs_no_pointers(qdq):
    # no rows, sequences, tokens or queries: OK whatever the (empty) tensors' addresses; other arguments are still checked
    lib, ok = qdq.lib(), qdq.QDQ_OK
    assert lib.qdq_rms_norm(None, None, None, None, None, None, 0, 0, 64, 64, 0, 0, 0, 1e-5, None) == ok
    assert lib.qdq_rms_norm(None, None, None, None, None, None, 3, 0, 64, 64, 0, 0, 0, 1e-5, None) == qdq.QDQ_ERR_DIMS
    for seqs, most in ((0, 5), (2, 0)):
        for f in (lib.qdq_kv_append, lib.qdq_kv_read):
            assert f(_at(0), 4, 16, 2, 64, _at(1), 3, None, _at(2), seqs, most, None, None, 128, 128, 0, None) == ok
            assert f(None, 4, 16, 2, 64, None, 3, None, _at(2), seqs, most, None, None, 128, 128, 0, None) == ok
            assert f(None, 4, 24, 2, 64, None, 3, None, _at(2), seqs, most, None, None, 128, 128, 0, None) == qdq.QDQ_ERR_DIMS
        assert lib.qdq_kv_attention(None, 4, 16, 2, 64, None, 3, None, _at(2), seqs, most, 48, 4, None, 256, None, 256, None, None,
                                    0.125, 0.0, 0, 0, None, 0, None) == ok
        assert lib.qdq_kv_attention(None, 4, 16, 2, 64, None, 3, None, _at(2), seqs, most, 48, 3, None, 256, None, 256, None, None,
                                    0.125, 0.0, 0, 0, None, 0, None) == qdq.QDQ_ERR_DIMS
    assert lib.qdq_token_logprobs(None, 1000, 0, _at(0), 0, 1000, 5, None, None, None, None, None, 0, None) == ok
    assert lib.qdq_token_logprobs(None, 1000, 0, _at(0), 0, 1000, 1001, None, None, None, None, None, 0, None) == qdq.QDQ_ERR_DIMS


def test_page_bytes(qdq):
    assert qdq.kv_page_bytes(64, 8, 128) == 8 * 16512             # 16384 codes + 32 bytes of scales, to 128
    assert qdq.kv_page_bytes(16, 1, 64) == 2176
    for bad in ((15, 1, 64), (24, 1, 64), (16, 0, 64), (16, 1, 80), (0, 1, 64)):
        assert qdq.kv_page_bytes(*bad) == 0


def test_append_and_read_refusals(qdq):
    lib = qdq.lib()
    p, t, n, cu, k, v = (_at(i) for i in range(6))

    def append(p=p, pages=4, page=16, heads=2, dim=64, t=t, ts=3, n=n, cu=cu, seqs=2, most=5, k=k, v=v, ks=128, vs=128, type=0):
        return lib.qdq_kv_append(p, pages, page, heads, dim, t, ts, n, cu, seqs, most, k, v, ks, vs, type, None)

    def read(p=p, pages=4, page=16, heads=2, dim=64, t=t, ts=3, start=n, cu=cu, seqs=2, most=5, k=k, v=v, ks=128, vs=128, type=0):
        return lib.qdq_kv_read(p, pages, page, heads, dim, t, ts, start, cu, seqs, most, k, v, ks, vs, type, None)

    for call in (append, read):
        assert call(p=None) == qdq.QDQ_ERR_NULL
        assert call(t=None) == qdq.QDQ_ERR_NULL
        assert call(k=None) == qdq.QDQ_ERR_NULL
        assert call(pages=0) == qdq.QDQ_ERR_DIMS
        assert call(page=24) == qdq.QDQ_ERR_DIMS
        assert call(heads=0) == qdq.QDQ_ERR_DIMS
        assert call(ts=0) == qdq.QDQ_ERR_DIMS
        assert call(seqs=-1) == qdq.QDQ_ERR_DIMS
        assert call(most=-1) == qdq.QDQ_ERR_DIMS
        assert call(type=7) == qdq.QDQ_ERR_DIMS
        assert call(ks=127) == qdq.QDQ_ERR_DIMS
        assert call(dim=80, ks=160, vs=160) == qdq.QDQ_ERR_UNSUPPORTED
        assert call(p=p + 64) == qdq.QDQ_ERR_ALIGN
        assert call(t=t + 2) == qdq.QDQ_ERR_ALIGN
        assert call(v=v + 8) == qdq.QDQ_ERR_ALIGN
        assert call(vs=130) == qdq.QDQ_ERR_ALIGN
        assert call(ks=132, type=1) == qdq.QDQ_ERR_ALIGN
        assert call(k=p + 128) == qdq.QDQ_ERR_ALIAS
        assert call(seqs=0) == qdq.QDQ_OK
        assert call(most=0) == qdq.QDQ_OK
    assert append(cu=None) == qdq.QDQ_ERR_DIMS                    # one token each needs max_new 1
    assert append(n=None) == qdq.QDQ_ERR_NULL
    assert append(t=p) == qdq.QDQ_ERR_ALIAS
    assert read(cu=None) == qdq.QDQ_ERR_NULL
    assert read(k=v) == qdq.QDQ_ERR_ALIAS


def test_attention_refusals(qdq):
    f = qdq.lib().qdq_kv_attention
    p, t, n, cu, q, o, lse, sl, ws = (_at(i) for i in range(9))

    def call(p=p, pages=4, page=16, heads=2, dim=64, t=t, ts=3, n=n, cu=cu, seqs=2, most=5, kv=48, nh=4, q=q, qs=256, o=o, os=256,
             lse=lse, sl=sl, scale=0.125, cap=0.0, win=0, type=0, ws=ws, wb=1 << 24):
        return f(p, pages, page, heads, dim, t, ts, n, cu, seqs, most, kv, nh, q, qs, o, os, lse, sl, scale, cap, win, type, ws, wb, None)

    for name in ("p", "t", "n", "q", "o", "ws"):
        assert call(**{name: None}) == qdq.QDQ_ERR_NULL
    assert call(nh=3) == qdq.QDQ_ERR_DIMS
    assert call(kv=-1) == qdq.QDQ_ERR_DIMS
    assert call(win=-1) == qdq.QDQ_ERR_DIMS
    assert call(cap=-1.0) == qdq.QDQ_ERR_DIMS
    assert call(scale=float("inf")) == qdq.QDQ_ERR_DIMS
    assert call(cu=None) == qdq.QDQ_ERR_DIMS
    assert call(qs=255) == qdq.QDQ_ERR_DIMS
    assert call(type=-1) == qdq.QDQ_ERR_DIMS
    assert call(dim=72, qs=288, os=288) == qdq.QDQ_ERR_UNSUPPORTED
    assert call(kv=(1 << 30) + 1) == qdq.QDQ_ERR_UNSUPPORTED
    assert call(q=q + 4) == qdq.QDQ_ERR_ALIGN
    assert call(ws=ws + 16) == qdq.QDQ_ERR_ALIGN
    assert call(os=258) == qdq.QDQ_ERR_ALIGN
    assert call(o=q) == qdq.QDQ_ERR_ALIAS
    assert call(o=p + 256) == qdq.QDQ_ERR_ALIAS
    assert call(lse=o) == qdq.QDQ_ERR_ALIAS
    assert call(ws=q) == qdq.QDQ_ERR_ALIAS
    assert call(sl=o) == qdq.QDQ_ERR_ALIAS
    assert call(seqs=0) == qdq.QDQ_OK
    assert call(most=0) == qdq.QDQ_OK
    assert qdq.kv_attention_workspace_bytes(1, 1, 100, 3, 2, 64) == 0
    assert qdq.kv_attention_workspace_bytes(1, 1, 100, 4, 2, 72) == 0


def test_logprobs_refusals(qdq):
    f = qdq.lib().qdq_token_logprobs
    x, t, lp, en, ti, tl, ws = (_at(i) for i in range(7))

    def call(x=x, st=1000, type=0, t=t, rows=3, n=1000, k=5, lp=lp, en=en, ti=ti, tl=tl, ws=ws, wb=1 << 24):
        return f(x, st, type, t, rows, n, k, lp, en, ti, tl, ws, wb, None)

    assert call(x=None) == qdq.QDQ_ERR_NULL
    assert call(t=None) == qdq.QDQ_ERR_NULL                       # a log probability needs its token
    assert call(lp=None) == qdq.QDQ_ERR_NULL
    assert call(ti=None) == qdq.QDQ_ERR_NULL
    assert call(ws=None) == qdq.QDQ_ERR_NULL
    assert call(st=999) == qdq.QDQ_ERR_DIMS
    assert call(k=-1) == qdq.QDQ_ERR_DIMS
    assert call(n=4, k=5) == qdq.QDQ_ERR_DIMS
    assert call(type=9) == qdq.QDQ_ERR_DIMS
    assert call(k=65) == qdq.QDQ_ERR_UNSUPPORTED
    assert call(x=x + 2) == qdq.QDQ_ERR_ALIGN
    assert call(lp=lp + 2) == qdq.QDQ_ERR_ALIGN
    assert call(ws=ws + 128) == qdq.QDQ_ERR_ALIGN
    assert call(lp=x + 4) == qdq.QDQ_ERR_ALIAS
    assert call(tl=ti) == qdq.QDQ_ERR_ALIAS
    assert call(en=t) == qdq.QDQ_ERR_ALIAS
    assert call(rows=0) == qdq.QDQ_OK
    assert qdq.token_logprobs_workspace_bytes(3, 1000, 65) == 0


def test_binding_refuses_wrong_tensors(qdq):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        qdq.rms_norm(x, None, x.half(), 4, 64)
    with pytest.raises(TypeError):
        qdq.rms_norm(x.double(), None, x.double(), 4, 64)
    with pytest.raises(TypeError):
        qdq.rms_norm(x, torch.zeros(64).half(), x, 4, 64)
    with pytest.raises(ValueError):
        qdq.rms_norm(x, None, x, 4, 63)
    with pytest.raises(ValueError):
        qdq.rms_norm(x.t().contiguous().t(), None, torch.zeros(4, 64), 4, 64)
    with pytest.raises(TypeError):
        qdq.token_logprobs(x, torch.zeros(4, dtype=torch.int64), torch.zeros(4), None, 4, 64, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(TypeError):
        qdq.rms_norm(x, None, x.clone(), 4, 64)  # not on the device
    pages = torch.zeros(3, 2176, dtype=torch.uint8)
    table = torch.zeros(1, 2, dtype=torch.int64)
    with pytest.raises(TypeError):
        qdq.kv_append(pages, table, torch.zeros(1, dtype=torch.int32), x, x, 1, 64, 16)
    with pytest.raises(ValueError):
        qdq.kv_append(pages[:, 1:], table.int(), torch.zeros(1, dtype=torch.int32), x, x, 1, 64, 16)


def test_binding_without_the_c_marshalling(qdq, monkeypatch, tmp_path):
    # not built, or not loadable: the Python code makes the calls (and refuses a host tensor)
    import torch
    x = torch.zeros(4, 64)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(qdq, "_PKG", str(tmp_path))
    for content in (None, b"not a library"):
        if content:
            (tmp_path / "_fastcall.so").write_bytes(content)
        monkeypatch.setattr(qdq, "_fast_lib", None)
        monkeypatch.setattr(qdq, "_fast", None)
        for _ in range(2):
            with pytest.raises(TypeError, match="CUDA tensor"):
                qdq.rms_norm(x, None, x.clone(), 4, 64)


def test_build_without_python_headers(qdq, monkeypatch, tmp_path):
    import sysconfig

    from ggml_quantized_dequant_gb300 import _build
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    monkeypatch.setattr(_build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    assert _build.build_fastcall() is None
    assert _build.build() == _build.LIB and not (tmp_path / "_fastcall.so").exists()


def _short_calls(qdq, device):
    """Calls whose tensors are right but for one that holds less than the call reads or writes."""
    import torch

    def f(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device=device)

    def i(*shape):
        return f(*shape, dtype=torch.int32)

    def norm(x=f(4, 64), w=f(64), o=f(4, 64), r=f(4, 64), s=f(4, 64), q=f(4 * 2 * 34, dtype=torch.uint8)):
        qdq.rms_norm(x, w, o, 4, 64, residual=r, sum_out=s, q8_out=q)

    pages, table, ws = f(3, 2176, dtype=torch.uint8), i(2, 1), f(1 << 22, dtype=torch.uint8)

    def append(n=i(2), k=f(2, 64), v=f(2, 64), cu=None):
        qdq.kv_append(pages, table, n, k, v, 1, 64, 16, cu_new=cu, max_new=1)

    def read(start=i(2), cu=i(3), k=f(2, 64), v=f(2, 64)):
        qdq.kv_read(pages, table, start, cu, k, v, 1, 64, 16, 1)

    def attention(n=i(2), q=f(2, 128), o=f(2, 128), cu=None, sl=f(2), lse=f(2, 2), ws=ws):
        qdq.kv_attention(pages, table, n, q, o, ws, 2, 1, 64, 16, 16, cu_q=cu, slopes=sl, lse=lse)

    def logprobs(x=f(4, 64), t=i(4), lp=f(4), en=f(4), k=3, ti=i(4, 3), tl=f(4, 3), ws=ws):
        qdq.token_logprobs(x, t, lp, en, 4, 64, ws, k, ti, tl)

    return {norm: dict(x=f(3, 64), w=f(63), o=f(3, 64), r=f(3, 64), s=f(3, 64), q=f(4 * 2 * 34 - 1, dtype=torch.uint8)),
            append: dict(n=i(1), k=f(1, 64), v=f(1, 64), cu=i(2)), read: dict(start=i(1), cu=i(2)),
            attention: dict(n=i(1), q=f(1, 128), o=f(1, 128), cu=i(2), sl=f(1), lse=f(1, 2), ws=f(1 << 22, 2, dtype=torch.uint8)[:, 0]),
            logprobs: dict(x=f(3, 64), t=i(3), lp=f(3), en=f(3), ti=i(3, 3), tl=f(3, 3), ws=f(1 << 22, 2, dtype=torch.uint8)[:, 0])}


def test_binding_refuses_short_tensors(qdq, monkeypatch):
    # (host tensors in the place of the device's: every call is refused before anything is launched)
    monkeypatch.setattr(qdq, "_cuda", lambda name, t: None if t is None else t.data_ptr())
    for call, short in _short_calls(qdq, "cpu").items():
        for name, tensor in short.items():
            with pytest.raises(ValueError, match="expected"):
                call(**{name: tensor})


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


def test_attention_kernel_option(qdq):
    assert qdq.set_option(qdq.QDQ_OPT_ATTN_KERNEL, 2) == 0
    assert qdq.lib().qdq_set_option(qdq.QDQ_OPT_ATTN_KERNEL, 3) == qdq.QDQ_ERR_DIMS
    assert qdq.lib().qdq_set_option(qdq.QDQ_OPT_ATTN_KERNEL, -1) == qdq.QDQ_ERR_DIMS
    assert qdq.set_option(qdq.QDQ_OPT_ATTN_KERNEL, 0) == 2
