"""The debug build (-DQDQ_CHECKS) of the decode-step operators: every guard holds on valid inputs.

The guards cover the parts and tickets in the caller's workspace, the blocks of a split and the lists in shared memory.
Each operator runs through both builds, which must agree bit for bit, and the status word must stay 0.
"""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def checked(cuda_lib):
    from ggml_quantized_dequant_gb300 import _build
    dbg = ctypes.CDLL(_build.build(checks=True))
    for name, (res, args) in cuda_lib.SIGNATURES.items():
        fn = getattr(dbg, name)
        fn.restype, fn.argtypes = res, args
    assert dbg.qdq_checks_enabled() == 1 and dbg.qdq_check_status() == 0
    return dbg


def _same(qdq, dbg, run):
    import torch
    want = [t.clone() for t in run()]
    normal, qdq._lib = qdq._lib, dbg
    try:
        got = run()
        torch.cuda.synchronize()
        assert dbg.qdq_check_status() == 0 and dbg.qdq_pipeline_timeouts() == 0
    finally:
        qdq._lib = normal
    for a, b in zip(want, got):
        assert a.dtype == b.dtype and np.array_equal(*(t.contiguous().view(torch.uint8).cpu().numpy() for t in (a, b)))


def _i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,n,dtype", [(1, 3072, "float32"), (700, 8192, "bfloat16"), (10000, 320, "float16"), (3, 20000, "float32")])
def test_checked_norm(cuda_lib, checked, rows, n, dtype):
    import torch
    x = torch.randn(rows, n, device="cuda").to(getattr(torch, dtype))
    w = torch.randn(n, device="cuda")

    def run():
        out, total = torch.empty_like(x), torch.empty_like(x)
        q8 = torch.zeros(cuda_lib.q8_0_packed_bytes(rows, n), dtype=torch.uint8, device="cuda")
        cuda_lib.rms_norm(x, w, out, rows, n, residual=x.flip(0).contiguous(), sum_out=total, q8_out=q8)
        return [out, total, q8]

    _same(cuda_lib, checked, run)


# (lengths, queries, heads, cache heads, dims, type, bound, cap and bias)
ATTENTION = [
    ([777], [1], 24, 8, 128, "float32", 777, False),
    ([20000], [1], 4, 2, 64, "bfloat16", 20000, False),
    (list(range(1, 3000, 63)), [1] * 48, 8, 8, 64, "float32", 3000, True),
    ([6000, 30, 1, 2000] * 4 + [1, 7, 900], [1, 0, 1, 1] * 4 + [0, 0, 1], 8, 8, 128, "float32", 8000, False),
    ([4000, 30, 1, 2000, 9] * 3, [2, 1, 1, 5, 0] * 3, 12, 4, 96, "float16", 9000, True),
    ([700, 2000, 40], [300, 129, 40], 6, 2, 128, "bfloat16", 2000, False),
    ([700, 2000, 40], [300, 129, 40], 6, 2, 64, "float32", 2000, True),
    ([1500, 90], [130, 90], 4, 2, 256, "bfloat16", 1500, False),
    ([1500, 90], [130, 90], 4, 2, 192, "float32", 1500, False),
]


@pytest.mark.parametrize("lens,nq,heads,n_kv,dim,dtype,bound,bent", ATTENTION)
def test_checked_cache_and_attention(cuda_lib, checked, lens, nq, heads, n_kv, dim, dtype, bound, bent):
    import torch
    page, dt = 32, getattr(torch, dtype)
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(need)), -1)
    for s, (m, at) in enumerate(zip(need, np.cumsum([0] + need))):
        table[s, :m] = at + np.arange(m)
    total, cu = sum(lens), np.cumsum([0] + lens)
    k, v = (torch.randn(total, n_kv, dim, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(sum(nq), heads, dim, device="cuda").to(dt)
    slopes = torch.rand(heads, device="cuda") / 16 if bent else None

    def run():
        pages = cuda_lib.kv_pages(sum(need), page, n_kv, dim)
        cuda_lib.kv_append(pages, _i32(table), _i32(lens), k, v, n_kv, dim, page, cu_new=_i32(cu), max_new=max(lens))
        kk, vv = torch.empty_like(k), torch.empty_like(v)
        cuda_lib.kv_read(pages, _i32(table), None, _i32(cu), kk, vv, n_kv, dim, page, max(lens))
        made = [pages, kk, vv]
        ws = cuda_lib.kv_attention_workspace(len(lens), max(nq), bound, heads, n_kv, dim)
        for window in (0, 150):
            out, lse = torch.zeros_like(q), torch.zeros(len(q), heads, device="cuda")
            cuda_lib.kv_attention(pages, _i32(table), _i32(lens), q, out, ws, heads, n_kv, dim, page, bound,
                                  cu_q=_i32(np.cumsum([0] + nq)), max_q=max(nq), softcap=20.0 if bent else 0.0, window=window,
                                  slopes=slopes, lse=lse)
            made += [out, lse]
        return made

    for kernel in (0, 1, 2):
        cuda_lib.set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, kernel)
        checked.qdq_set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, kernel)
        try:
            _same(cuda_lib, checked, run)
        finally:
            cuda_lib.set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, 0)
            checked.qdq_set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, 0)


@pytest.mark.parametrize("rows,n,k,dtype", [(1, 128256, 20, "float32"), (40, 30001, 64, "bfloat16"), (700, 5000, 5, "float16"),
                                            (3, 50000, 0, "float32")])
def test_checked_logprobs(cuda_lib, checked, rows, n, k, dtype):
    import torch
    x = torch.randn(rows, n, device="cuda").to(getattr(torch, dtype))
    x[-1, 3:] = float("-inf")  # fewer logits than alternatives: every list fills
    tokens = _i32(np.arange(rows) % n)

    def run():
        lp, ent = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
        ti, tl = torch.zeros(rows, k, dtype=torch.int32, device="cuda"), torch.zeros(rows, k, device="cuda")
        cuda_lib.token_logprobs(x, tokens, lp, ent, rows, n, cuda_lib.token_logprobs_workspace(rows, n, k), k, ti, tl)
        return [lp, ent, ti, tl]

    _same(cuda_lib, checked, run)
