"""GPU parity of the decode-step operators against the float64 forms of ``oracle.decode_oracle``.

Bounds (u = 2^-24, the f32 unit roundoff; e = the output type's: 2^-24, 2^-11, 2^-8):
* norm: a sum of squares folded over at most 32 products per thread and two warp folds has relative
  error <= 64 u, the root half of it, and three roundings follow: |y - y_ref| <= (64 u + e) |y_ref|.
* cache codes and scales: equal (the definition is in f32 operations); values read back: one rounding.
* attention: a score's products are exact in two f16 parts of the query (relative remainder 2^-22) and
  summed by at most 16 instructions of one truncation each, so it is off by at most
  d = 2^-18 a + 2^-20 with a = scale * sum |q||k| + |bias| (+ 2^-20 cap for the tanh); probabilities
  are off by a relative 2 d + 2^-20 before and after normalisation, and the sums over tokens by 2^-18;
  the f16 parts of a probability times its value scale end at 2^-39 of the row's largest such product
  (z = max p s, a code is at most 127, and the tokens of a sum share the row's total of p):
  |o - o_ref| <= (2 d + 2^-17) sum p|v| + 2^-39 127 n z + e |o_ref|,  |lse - ref| <= d + 2^-18 + 2^-22 |lse|;
  with 16-bit activations the probabilities are rounded to f16 once where a tile has more than 8
  rows: + 2^-11 sum p|v|.
* log probabilities: the running sum of a thread has at most n / 256 + 64 additions and an exponent
  is off by 2^-22 (|x| + 1): |lp - ref| <= t with t = (n / 256 + 64) u + 2^-21 (max |x| + 1), the entropy
  by t (4 + 2 H).
"""
import numpy as np
import pytest

from oracle import decode_oracle as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _dt(t):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[t]


def _t(a, dtype=None):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return x if dtype is None else x.to(dtype)


def _np(t):
    import torch
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _within(got, want, bound):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isnan(want) | (got == want) | (np.abs(got - want) <= bound)
    assert ok.all(), "worst excess %g" % np.nanmax(np.where(ok, 0, np.abs(got - want) / np.maximum(bound, 1e-300)))


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("rows,n,dtype,residual", [
    (1, 1, "f32", False), (3, 31, "f32", True), (1, 3072, "f32", True), (5, 3072, "f16", True), (200, 160, "bf16", True),
    (2, 8193, "f32", True), (3, 8192, "bf16", False), (170, 8200, "f16", True), (2, 20001, "bf16", True),
    (2, 32768, "f32", True), (153, 32767, "bf16", False), (1, 16384, "f16", True), (153, 1, "f16", True)])
def test_norm(cuda_lib, rows, n, dtype, residual):
    import torch
    rng = np.random.default_rng(rows * 7 + n)
    x = _t(rng.standard_normal((rows, n)).astype(np.float32), _dt(dtype))
    r = _t(3 * rng.standard_normal((rows, n)).astype(np.float32), _dt(dtype)) if residual else None
    w = _t(rng.standard_normal(n).astype(np.float32))
    out, total = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    cuda_lib.rms_norm(x, w, out, rows, n, 1e-5, residual=r, sum_out=total)
    y, h = ref.rms_norm(_np(x), None if r is None else _np(r), _np(w), 1e-5)
    _within(_np(out), y, (64 * U + EPS[dtype]) * np.abs(y) + (2.0 ** -25 if dtype == "f16" else 0))
    _within(_np(total), h, EPS[dtype] * np.abs(h) + (2.0 ** -25 if dtype == "f16" else 0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (4, 3), (8, 8), (0, 12)])
def test_norm_strided_and_in_place(cuda_lib, dtype, offset, pad):
    # rows inside a wider buffer at every alignment; the sum over the residual, the norm over x; no weight
    import torch
    rows, n = 7, 264
    rng = np.random.default_rng(offset * 31 + pad)
    buf = _t(rng.standard_normal((2, rows * (n + pad) + offset)).astype(np.float32), _dt(dtype))
    before = buf.clone()
    x = buf[0, offset:].as_strided((rows, n), (n + pad, 1))
    r = buf[1, offset:].as_strided((rows, n), (n + pad, 1))
    y, h = ref.rms_norm(_np(x), _np(r), None, 1e-6)
    cuda_lib.rms_norm(x, None, x, rows, n, 1e-6, residual=r, sum_out=r)
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    _within(_np(x), y, (64 * U + EPS[dtype]) * np.abs(y) + tiny)
    _within(_np(r), h, EPS[dtype] * np.abs(h) + tiny)
    mask = torch.ones_like(buf, dtype=torch.bool)
    for i in range(2):
        mask[i, offset:].as_strided((rows, n), (n + pad, 1)).fill_(False)
    assert torch.equal(buf[mask], before[mask])  # nothing between the rows is written


@pytest.mark.parametrize("rows,n,dtype", [(1, 32, "f32"), (9, 3072, "f32"), (300, 96, "bf16"), (3, 8224, "f16"), (2, 32768, "f32")])
def test_norm_to_q8_0(cuda_lib, rows, n, dtype):
    import torch
    rng = np.random.default_rng(rows + n)
    x = _t(rng.standard_normal((rows, n)).astype(np.float32), _dt(dtype))
    x[0, :32] = 0  # a block of zeros
    w = _t(rng.standard_normal(n).astype(np.float32))
    out = torch.empty_like(x)
    packed = torch.full((cuda_lib.q8_0_packed_bytes(rows, n),), 0x55, dtype=torch.uint8, device="cuda")
    cuda_lib.rms_norm(x, w, out, rows, n, 1e-5, q8_out=packed)
    y, _ = ref.rms_norm(_np(x), None, _np(w), 1e-5)
    _within(_np(out), y, (64 * U + EPS[dtype]) * np.abs(y) + (2.0 ** -25 if dtype == "f16" else 0))
    val = torch.empty(rows, n, device="cuda")
    cuda_lib.q8_0_dequant(packed, val, rows, n)  # the packed form is an ordinary Q8_0 matrix
    m = np.abs(y.reshape(rows, -1, 32)).max(-1, keepdims=True)
    # half a step of d = f16(m / 127), the clamp at 127 d (d may round down by 2^-11), and d below the f16 normals
    step = (m / 127 * (0.5 + 127 * 2.0 ** -11) * (1 + 2.0 ** -10) + 128 * 2.0 ** -25) * np.ones((1, 1, 32))
    _within(_np(val), y, step.reshape(rows, n) + 64 * U * np.abs(y))
    assert (_np(val)[0, :32] == 0).all()


@pytest.mark.parametrize("rows,n,dtype,residual,pad", [
    (650, 8192, "bf16", True, 0), (1251, 7160, "f16", True, 8), (611, 5600, "f32", False, 4), (620, 8192, "f32", True, 0),
    (9800, 96, "bf16", True, 0), (20001, 8, "f16", False, 8), (9729, 384, "f32", True, 0), (10001, 320, "f16", True, 32)])
def test_norm_many_rows(cuda_lib, rows, n, dtype, residual, pad):
    # CTAs that take several rows: strided, in place, with every output
    import torch
    rng = np.random.default_rng(rows + n)
    buf = _t(rng.standard_normal((2, rows * (n + pad))).astype(np.float32), _dt(dtype))
    x, r = (b.as_strided((rows, n), (n + pad, 1)) for b in buf)
    w = _t(rng.standard_normal(n).astype(np.float32))
    y, h = ref.rms_norm(_np(x), _np(r) if residual else None, _np(w), 1e-5)
    before = buf.clone()
    q8 = n % 32 == 0
    packed = torch.full((cuda_lib.q8_0_packed_bytes(rows, n),), 0x55, dtype=torch.uint8, device="cuda") if q8 else None
    cuda_lib.rms_norm(x, w, x, rows, n, 1e-5, residual=r if residual else None, sum_out=r, q8_out=packed)
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    _within(_np(x), y, (64 * U + EPS[dtype]) * np.abs(y) + tiny)
    _within(_np(r), h, EPS[dtype] * np.abs(h) + tiny)
    mask = torch.ones_like(buf, dtype=torch.bool)
    for m in mask:
        m.as_strided((rows, n), (n + pad, 1)).fill_(False)
    assert torch.equal(buf[mask], before[mask])
    if q8:
        val = torch.empty(rows, n, device="cuda")
        cuda_lib.q8_0_dequant(packed, val, rows, n)
        m = np.abs(y.reshape(rows, -1, 32)).max(-1, keepdims=True)
        step = (m / 127 * (0.5 + 127 * 2.0 ** -11) * (1 + 2.0 ** -10) + 128 * 2.0 ** -25) * np.ones((1, 1, 32))
        _within(_np(val), y, step.reshape(rows, n) + 64 * U * np.abs(y))


@pytest.mark.parametrize("rows,n,dtype", [(1536, 3072, "f32"), (4096, 8192, "bf16"), (256, 1024, "f16"), (20224, 256, "bf16")])
def test_norm_to_q8_0_is_the_next_calls_matrix(cuda_lib, rows, n, dtype):
    # the projections read their weights ahead of the wait for the call before: the norm must have written them by then
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = [torch.randn(rows, n, device="cuda", generator=g).to(_dt(dtype)) for _ in range(4)]
    v = torch.randn(8, n, device="cuda", generator=g)
    packed = torch.zeros(cuda_lib.q8_0_packed_bytes(rows, n), dtype=torch.uint8, device="cuda")
    ws = torch.empty(cuda_lib.gemm_batch_workspace_bytes(8, rows, n), dtype=torch.uint8, device="cuda")
    outs = {"one": torch.empty(1, rows, device="cuda"), "few": torch.empty(3, rows, device="cuda"),
            "batch": torch.empty(8, rows, device="cuda")}

    def call(how):
        if how == "batch":
            cuda_lib.q8_0_gemm_batch(packed, v, outs[how], ws, rows, n, 8)
        else:
            cuda_lib.q8_0_gemv(packed, v, outs[how], rows, n, 1 if how == "one" else 3)

    for how, out in outs.items():
        want = []
        for xi in x:
            cuda_lib.rms_norm(xi, None, None, rows, n, q8_out=packed)
            torch.cuda.synchronize()
            call(how)
            want.append(out.clone())
        for i in range(24):
            cuda_lib.rms_norm(x[i % 4], None, None, rows, n, q8_out=packed)
            call(how)
            assert torch.equal(out, want[i % 4]), (how, i)


def test_norm_rows_that_are_not_finite_or_zero(cuda_lib):
    import torch
    x = torch.randn(4, 64, device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    out = torch.empty_like(x)
    packed = torch.empty(cuda_lib.q8_0_packed_bytes(4, 64), dtype=torch.uint8, device="cuda")
    cuda_lib.rms_norm(x, None, out, 4, 64, 1e-5, q8_out=packed)
    val = torch.empty(4, 64, device="cuda")
    cuda_lib.q8_0_dequant(packed, val, 4, 64)
    for got in (_np(out), _np(val)):
        assert np.isfinite(got[[0, 1, 3]]).all() and (got[1] == 0).all() and np.isnan(got[2]).all()


def test_norm_between_slices_of_one_buffer(cuda_lib):
    # x, the residual, the sum and the norm beside one another in wide rows
    import torch
    rows, n = 700, 264
    rng = np.random.default_rng(12)
    for dtype in ("f32", "bf16"):
        buf = _t(rng.standard_normal((rows, 4 * n + 8)).astype(np.float32), _dt(dtype))
        before = buf.clone()
        x, total, out, r = (buf[:, i:i + n] for i in (0, n, 2 * n, 3 * n + 8))
        y, h = ref.rms_norm(_np(x), _np(r), None, 1e-5)
        cuda_lib.rms_norm(x, None, out, rows, n, 1e-5, residual=r, sum_out=total)
        _within(_np(out), y, (64 * U + EPS[dtype]) * np.abs(y))
        _within(_np(total), h, EPS[dtype] * np.abs(h))
        for part in (slice(0, n), slice(3 * n, 4 * n + 8)):
            assert torch.equal(buf[:, part], before[:, part])


# ------------------------------------------------------------------ cache

def _pool(n_pages, page, n_kv, dim, seed=0):
    """A pool of garbage: every scale NaN, every code something."""
    import torch
    g = torch.Generator(device="cpu").manual_seed(seed)
    raw = torch.randint(0, 256, (n_pages, n_kv, ref.record_bytes(page, dim)), generator=g, dtype=torch.uint8)
    raw[:, :, 2 * page * dim:] = 0xFF
    return raw.to("cuda")


def _tables(rng, lens, page, n_pages, extra=1):
    width = max(1, max(-(-n // page) for n in lens) + extra)
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for s, n in enumerate(lens):
        m = -(-n // page)
        table[s, :m] = ids[at:at + m]
        at += m
    assert at <= n_pages
    return table


@pytest.mark.parametrize("page,n_kv,dim,dtype", [(16, 1, 64, "f32"), (64, 2, 128, "f32"), (48, 3, 96, "bf16"), (32, 2, 256, "f16"),
                                                 (128, 1, 192, "bf16"), (16, 2, 128, "f16")])
def test_append_and_read(cuda_lib, page, n_kv, dim, dtype):
    # several calls: prompts, single tokens, nothing, across block and page ends; codes and scales exactly
    import torch
    rng = np.random.default_rng(page + dim)
    steps = [[5, 0, 33, 1], [1, 1, 1, 1], [0, 17, 0, 15], [1, 1, 1, 1], [70, 2, 16, 0], [1, 1, 1, 1]]
    total = np.sum(steps, 0)
    raw = _pool(40, page, n_kv, dim)
    want = ref.Cache(raw.cpu().numpy().copy(), page, n_kv, dim)
    table = _tables(rng, total, page, 40)
    tt = _i32(table)
    lens = np.zeros(4, int)
    for i, new in enumerate(steps):
        lens = lens + new
        cu = np.concatenate([[0], np.cumsum(new)])
        amp = np.exp(rng.standard_normal((cu[-1], 1, 1)))
        k = _t((amp * rng.standard_normal((cu[-1], n_kv, dim))).astype(np.float32), _dt(dtype))
        # v inside a wider buffer, as a slice of a fused projection
        wide = _t((amp * rng.standard_normal((cu[-1], n_kv + 2, dim))).astype(np.float32), _dt(dtype))
        v = wide[:, 1:1 + n_kv]
        single = all(n == 1 for n in new)
        cuda_lib.kv_append(raw, tt, _i32(lens), k, v, n_kv, dim, page, cu_new=None if single else _i32(cu),
                           max_new=1 if single else int(max(new)))
        want.append(table, lens, cu, _np(k).astype(np.float32), _np(v).astype(np.float32))
        got = ref.Cache(raw.cpu().numpy(), page, n_kv, dim)
        assert np.array_equal(got.raw, want.raw), "step %d" % i  # garbage past the tokens included: nothing else is written
    start = np.array([3, 0, 17, 1])
    n = np.array([total[0] - 3, total[1], 5, 0])
    cu = np.concatenate([[0], np.cumsum(n)])
    ko = torch.full((cu[-1], n_kv, dim), 7.0, device="cuda", dtype=_dt(dtype))
    vo = torch.full((cu[-1] + 1, n_kv + 1, dim), 7.0, device="cuda", dtype=_dt(dtype))
    cuda_lib.kv_read(raw, tt, _i32(start), _i32(cu), ko, vo[:-1, :-1], n_kv, dim, page, int(n.max()))
    for s in range(4):
        kk, vv = want.read(table, s, start[s], n[s])
        for got, val in ((ko, kk), (vo[:-1, :-1], vv)):
            g = _np(got[cu[s]:cu[s + 1]])
            assert np.array_equal(g, _np(_t(val.astype(np.float32), _dt(dtype))))
    assert (vo[-1] == 7).all() and (vo[:, -1] == 7).all()


def test_append_values_that_are_not_finite_or_tiny(cuda_lib):
    import torch
    page, n_kv, dim = 32, 2, 64
    raw = _pool(4, page, n_kv, dim)
    want = ref.Cache(raw.cpu().numpy().copy(), page, n_kv, dim)
    table = np.array([[2, 0]], np.int32)
    k = torch.randn(40, n_kv, dim, device="cuda")
    v = torch.randn(40, n_kv, dim, device="cuda")
    k[3, 0, 5] = float("nan")
    v[20, 1, 0] = float("inf")
    v[0:16, 0] = 1e-40     # a scale below the normal numbers counts as 0
    k[32:, 1] = 0
    for lo, hi in ((0, 2), (2, 39), (39, 40)):
        cuda_lib.kv_append(raw, _i32(table), _i32([hi]), k[lo:hi], v[lo:hi], n_kv, dim, page, cu_new=_i32([0, hi - lo]), max_new=hi - lo)
        want.append(table, np.array([hi]), np.array([0, hi - lo]), k[lo:hi].cpu().numpy(), v[lo:hi].cpu().numpy())
    got = ref.Cache(raw.cpu().numpy(), page, n_kv, dim)
    for a, b in zip(got.read(table, 0, 0, 40), want.read(table, 0, 0, 40)):
        assert np.array_equal(a, b, equal_nan=True)
    a, b = want.read(table, 0, 0, 40)
    assert np.isnan(a[:16, 0]).all() and np.isfinite(a[16:]).all() and np.isfinite(a[:, 1]).all()
    assert np.isnan(b[16:32, 1]).all() and np.isfinite(b[:, 0]).all()


def test_append_again_changes_nothing(cuda_lib):
    import torch
    raw = _pool(6, 32, 1, 128)
    table = _i32([[1, 4, 2]])
    k, v = torch.randn(60, 1, 128, device="cuda"), torch.randn(60, 1, 128, device="cuda")
    cuda_lib.kv_append(raw, table, _i32([41]), k[:41], v[:41], 1, 128, 32, cu_new=_i32([0, 41]), max_new=41)
    args = (raw, table, _i32([60]), 3 * k[41:], v[41:], 1, 128, 32)
    cuda_lib.kv_append(*args, cu_new=_i32([0, 19]), max_new=19)
    once = raw.clone()
    cuda_lib.kv_append(*args, cu_new=_i32([0, 19]), max_new=19)
    assert torch.equal(raw, once)


def test_tokens_without_a_page(cuda_lib):
    # page numbers outside the pool and past the table: nothing is written, reads are NaN
    import torch
    page, n_kv, dim = 16, 1, 64
    raw = _pool(3, page, n_kv, dim)
    before = raw.clone()
    table = _i32([[-1, 3], [1 << 30, 1], [0, 2]])
    k = torch.randn(100, n_kv, dim, device="cuda")
    cu = [0, 32, 64, 100]
    cuda_lib.kv_append(raw, table, _i32([32, 32, 36]), k, k, n_kv, dim, page, cu_new=_i32(cu), max_new=36)
    want = ref.Cache(before.cpu().numpy().copy(), page, n_kv, dim)
    want.append(np.array([[-1, 3], [1 << 30, 1], [0, 2]]), np.array([32, 32, 36]), cu, k.cpu().numpy(), k.cpu().numpy())
    assert np.array_equal(raw.cpu().numpy().reshape(want.raw.shape), want.raw)
    ko, vo = torch.zeros(100, n_kv, dim, device="cuda"), torch.zeros(100, n_kv, dim, device="cuda")
    cuda_lib.kv_read(raw, table, None, _i32(cu), ko, vo, n_kv, dim, page, 36)
    nan = _np(ko).__ne__(_np(ko)).all((1, 2))
    assert nan[:48].all() and not nan[48:96].any() and nan[96:].all()
    # more new tokens than the sequence holds: nothing
    was = raw.clone()
    cuda_lib.kv_append(raw, table, _i32([5, 5, 5]), k, k, n_kv, dim, page, cu_new=_i32([0, 6, 6, 12]), max_new=6)
    assert torch.equal(raw, was)


def test_tokens_past_the_stated_bounds(cuda_lib):
    # a sequence with more new (or wanted) tokens than max_new (max_tokens): the first ones are, the others are not
    import torch
    page, n_kv, dim = 32, 2, 64
    raw = _pool(12, page, n_kv, dim)
    raw[:, :, 2 * page * dim:] = 0  # no NaN scales: the pool's bytes are compared
    want = ref.Cache(raw.cpu().numpy().copy(), page, n_kv, dim)
    table = np.array([[5, 1, 7], [2, 0, 3]], np.int32)
    k, v = torch.randn(90, n_kv, dim, device="cuda"), torch.randn(90, n_kv, dim, device="cuda")
    for most, lens, new in ((1, [5, 1], [5, 1]), (3, [5 + 12, 3], [12, 2]), (20, [17 + 55, 3 + 15], [55, 15])):
        cu = np.concatenate([[0], np.cumsum(new)])
        cuda_lib.kv_append(raw, _i32(table), _i32(lens), k[:cu[-1]], v[:cu[-1]], n_kv, dim, page, cu_new=_i32(cu), max_new=most)
        for s in range(2):  # the oracle is told of the first ones alone
            n, at = min(new[s], most), slice(cu[s], cu[s] + min(new[s], most))
            want.append(table[s:s + 1], [lens[s] - new[s] + n], [0, n], k[at].cpu().numpy(), v[at].cpu().numpy())
        assert np.array_equal(raw.cpu().numpy().reshape(want.raw.shape), want.raw), most
    cu, start = [0, 37, 46], [3, 1]
    for most in (1, 8, 16, 30):
        ko, vo = torch.full((46, n_kv, dim), 7.0, device="cuda"), torch.full((46, n_kv, dim), 7.0, device="cuda")
        cuda_lib.kv_read(raw, _i32(table), _i32(start), _i32(cu), ko, vo, n_kv, dim, page, most)
        for s in range(2):
            n = min(cu[s + 1] - cu[s], most)
            for got, val in zip((ko, vo), want.read(table, s, start[s], n)):
                assert np.array_equal(_np(got[cu[s]:cu[s] + n]), val, equal_nan=True)
                assert (got[cu[s] + n:cu[s + 1]] == 7).all(), most


# ------------------------------------------------------------------ attention

@pytest.fixture(params=["automatic", "decode", "tensor"])
def attn_kernel(request, cuda_lib):
    """The attention tests run with the automatic choice of the kernel and with either one wherever it can run."""
    old = cuda_lib.set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, ["automatic", "decode", "tensor"].index(request.param))
    yield
    cuda_lib.set_option(cuda_lib.QDQ_OPT_ATTN_KERNEL, old)
    assert cuda_lib.pipeline_timeouts() == 0


def _filled(rng, lens, page, n_kv, dim, n_pages=None, amp=1.0):
    """A pool whose sequences hold random tokens (garbage elsewhere), its table and the oracle's view of it."""
    n_pages = n_pages or sum(-(-max(n, 0) // page) for n in lens) + 3
    raw = _pool(n_pages, page, n_kv, dim).cpu().numpy()
    table = _tables(rng, [max(n, 0) for n in lens], page, n_pages)
    c = ref.Cache(raw, page, n_kv, dim)
    for s, n in enumerate(lens):
        for b in range(-(-max(n, 0) // ref.BLOCK)):
            pid, t0 = table[s, b * ref.BLOCK // page], b * ref.BLOCK % page
            for h in range(n_kv):
                for which in range(2):
                    c._codes(pid, h, which)[t0:t0 + ref.BLOCK] = rng.integers(-127, 128, (ref.BLOCK, dim))
                    c._scales(pid, h, which)[t0 // ref.BLOCK] = amp * np.exp(0.5 * rng.standard_normal()) / 60
    return _t(raw), table, c


def _values(c, table, s, n):
    """Fast read of the oracle's cache: (n, heads, dim) keys and values."""
    out = np.zeros((2, n, c.n_kv, c.dim))
    for b in range(-(-n // ref.BLOCK)):
        pid, t0 = table[s, b * ref.BLOCK // c.page], b * ref.BLOCK % c.page
        m = min(ref.BLOCK, n - b * ref.BLOCK)
        for h in range(c.n_kv):
            for which in range(2):
                code = c._codes(pid, h, which)[t0:t0 + m].astype(np.float32)
                with np.errstate(invalid="ignore"):
                    out[which, b * ref.BLOCK:b * ref.BLOCK + m, h] = code * c._scales(pid, h, which)[t0 // ref.BLOCK]
    return out[0], out[1]


def _attend(qdq, raw, table, lens, nq, q, heads, n_kv, dim, page, softcap=0.0, window=0, slopes=None, max_kv=None, scale=None,
            workspace=None, max_q=None, stream=None):
    import torch
    cu = np.concatenate([[0], np.cumsum(nq)])
    out = torch.full_like(q, 5.0)
    lse = torch.full((q.shape[0], heads), 5.0, device="cuda")
    max_q = max_q or int(max(nq))
    max_kv = max_kv if max_kv is not None else max(0, int(max(lens)))
    ws = workspace if workspace is not None else qdq.kv_attention_workspace(len(lens), max_q, max_kv, heads, n_kv, dim)
    single = max_q == 1 and all(n == 1 for n in nq)
    qdq.kv_attention(raw, _i32(table), _i32(lens), q, out, ws, heads, n_kv, dim, page, max_kv, cu_q=None if single else _i32(cu),
                     max_q=max_q, scale=scale, softcap=softcap, window=window, slopes=slopes, lse=lse, stream=stream)
    return out, lse


def _check_attention(c, table, lens, nq, q, out, lse, dtype, scale, softcap, window, slopes):
    cu = np.concatenate([[0], np.cumsum(nq)])
    qn, on, ln = _np(q), _np(out), _np(lse)
    for s, n in enumerate(lens):
        if nq[s] == 0:
            continue
        k, v = _values(c, table, s, n)
        pos = n - nq[s] + np.arange(nq[s])
        o, l, av, mag, z = ref.attention(qn[cu[s]:cu[s + 1]], k, v, pos, scale, softcap, window,
                                      None if slopes is None else _np(slopes))
        d = 2.0 ** -18 * mag + 2.0 ** -20 * (1 + softcap)
        tiny = 2.0 ** -25 if dtype == "f16" else 0
        _within(on[cu[s]:cu[s + 1]], o, ((2 * d + 2.0 ** -17 + (0 if dtype == "f32" else 2.0 ** -11))[..., None] * av + EPS[dtype] * np.abs(o) + tiny
                                             + 2.0 ** -39 * n * z[..., None]))
        with np.errstate(invalid="ignore"):
            _within(ln[cu[s]:cu[s + 1]], l, d + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(np.isinf(l), 0, l)))


ATTN = [
    # lens, queries, heads, kv heads, dim, page, dtype, softcap, window, bias
    ([1], [1], 1, 1, 64, 16, "f32", 0, 0, False),
    ([15, 16, 17, 33], [1] * 4, 6, 2, 128, 32, "f32", 0, 0, False),
    ([777], [1], 24, 8, 128, 64, "f32", 0, 0, False),
    ([0, 5, 0, 1000], [1] * 4, 8, 1, 128, 64, "bf16", 0, 0, False),
    ([4001], [1], 3, 1, 128, 128, "f32", 0, 0, True),
    ([300, 2], [3, 2], 7, 1, 96, 48, "f32", 30.0, 0, False),
    ([300, 129, 40], [1, 0, 40], 4, 4, 256, 32, "f16", 0, 37, True),
    ([50, 3], [5, 9], 10, 2, 192, 16, "bf16", 20.0, 16, True),
    ([700, 64], [65, 64], 6, 2, 64, 64, "f16", 50.0, 100, False),
    ([1500], [200], 12, 4, 128, 64, "f32", 0, 0, False),
    ([1500, 90, 257], [130, 90, 1], 8, 2, 128, 16, "bf16", 0, 0, False),
    ([513, 700], [129, 260], 16, 1, 64, 32, "f32", 30.0, 200, True),
    ([300, 90], [90, 70], 2, 1, 256, 64, "bf16", 0, 0, False),
    ([300, 90], [90, 70], 2, 1, 256, 64, "f32", 0, 50, False),
    ([1000, 80], [70, 80], 4, 2, 192, 48, "f32", 0, 0, True),
    ([1000, 80], [70, 80], 4, 2, 192, 16, "f16", 30.0, 0, False),
    ([400, 81], [100, 81], 3, 1, 96, 16, "bf16", 0, 0, False),
    ([64, 65, 127, 128], [64, 65, 127, 128], 4, 2, 64, 16, "f32", 0, 0, False),
    ([9000, 300], [80, 65], 2, 1, 128, 32, "bf16", 0, 0, False),
    ([9000], [65], 2, 1, 64, 32, "f32", 0, 8000, False),
    ([6000, 100, 2100], [1] * 3, 9, 3, 64, 16, "f16", 0, 1, False),
    ([6000, 100, 2100], [1] * 3, 32, 2, 128, 16, "bf16", 15.0, 1024, True),
]


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("lens,nq,heads,n_kv,dim,page,dtype,softcap,window,bias", ATTN)
def test_attention(cuda_lib, lens, nq, heads, n_kv, dim, page, dtype, softcap, window, bias):
    rng = np.random.default_rng(sum(lens) + heads + dim)
    raw, table, c = _filled(rng, lens, page, n_kv, dim)
    q = _t(1.5 * rng.standard_normal((sum(nq), heads, dim)).astype(np.float32), _dt(dtype))
    slopes = _t((2.0 ** -np.linspace(1, 8, heads)).astype(np.float32)) if bias else None
    out, lse = _attend(cuda_lib, raw, table, lens, nq, q, heads, n_kv, dim, page, softcap, window, slopes)
    _check_attention(c, table, lens, nq, q, out, lse, dtype, dim ** -0.5, softcap, window, slopes)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("dtype,nq", [("f32", 1), ("bf16", 1), ("f32", 150), ("bf16", 150)])
def test_attention_sharp_scores_and_uneven_scales(cuda_lib, dtype, nq):
    # large queries, scales over many orders of magnitude, blocks of zeros (scale 0)
    rng = np.random.default_rng(3)
    heads, n_kv, dim, page, n = 4, 2, 128, 32, 2000
    raw, table, c = _filled(rng, [n], page, n_kv, dim)
    for b in range(-(-n // 16)):
        pid, t0 = table[0, b * 16 // page], b * 16 % page
        for h in range(n_kv):
            c._scales(pid, h, 1)[t0 // 16] = 0.0 if b % 5 == 0 else 10.0 ** rng.uniform(-20, 3)
            c._scales(pid, h, 0)[t0 // 16] = 0.0 if b % 7 == 0 else 10.0 ** rng.uniform(-6, -1)
    raw = _t(c.raw)
    q = _t((10.0 ** rng.uniform(-3, 1, (nq, heads, 1)) * rng.standard_normal((nq, heads, dim))).astype(np.float32), _dt(dtype))
    out, lse = _attend(cuda_lib, raw, table, [n], [nq], q, heads, n_kv, dim, page)
    _check_attention(c, table, [n], [nq], q, out, lse, dtype, dim ** -0.5, 0, 0, None)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("heads,nq", [(8, 1), (2, 4)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_of_16_bit_calls_with_few_rows_keeps_both_parts(cuda_lib, dtype, heads, nq):
    # at most 8 rows per cache head: probabilities in two f16 parts, so no 2^-11 sum p|v| in the bound; values that
    # nearly cancel, where one part alone would show
    rng = np.random.default_rng(14)
    lens, n_kv, dim = [4, 36, 200], 1, 64
    raw, table, c = _filled(rng, lens, 32, n_kv, dim)
    for s, n in enumerate(lens):
        for b in range(-(-n // 16)):
            pid, t0 = table[s, b * 16 // 32], b * 16 % 32
            v = c._codes(pid, 0, 1)[t0:t0 + 16]
            v[1::2] = -v[::2]
            c._scales(pid, 0, 1)[t0 // 16] = 0.02
    raw = _t(c.raw)
    q = _t(0.02 * rng.standard_normal((3 * nq, heads, dim)).astype(np.float32), _dt(dtype))
    out, lse = _attend(cuda_lib, raw, table, lens, [nq] * 3, q, heads, n_kv, dim, 32)
    qn, on = _np(q), _np(out)
    for s, n in enumerate(lens):
        k, v = _values(c, table, s, n)
        o, _, av, mag, z = ref.attention(qn[s * nq:(s + 1) * nq], k, v, n - nq + np.arange(nq), 0.125)
        d = 2.0 ** -18 * mag + 2.0 ** -20
        _within(on[s * nq:(s + 1) * nq], o, (2 * d + 2.0 ** -17)[..., None] * av + EPS[dtype] * np.abs(o) + 2.0 ** -39 * 127 * n * z[..., None]
                + (2.0 ** -25 if dtype == "f16" else 0))


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nq", [1, 140])
def test_attention_rows_that_see_nothing(cuda_lib, nq):
    # more queries than tokens: the first rows stand before the sequence
    rng = np.random.default_rng(4)
    lens, queries = [0, max(0, nq - 9)], [nq, nq]
    raw, table, c = _filled(rng, lens, 32, 1, 64)
    q = _t(rng.standard_normal((2 * nq, 2, 64)).astype(np.float32))
    out, lse = _attend(cuda_lib, raw, table, lens, queries, q, 2, 1, 64, 32)
    _check_attention(c, table, lens, queries, q, out, lse, "f32", 0.125, 0, 0, None)
    assert (_np(out)[:nq] == 0).all() and np.isneginf(_np(lse)[:nq]).all()


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nq", [9, 150])
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 100, 1 << 20, 200, 199])
def test_attention_widest_windows_of_rows_before_the_sequence(cuda_lib, nq, window):
    # a window as long as there are numbers for hides nothing, also where the first queries stand before the sequence
    rng = np.random.default_rng(9)
    lens, queries = [3, 200], [nq, 1]
    raw, table, c = _filled(rng, lens, 32, 1, 64)
    q = _t(rng.standard_normal((nq + 1, 2, 64)).astype(np.float32))
    out, lse = _attend(cuda_lib, raw, table, lens, queries, q, 2, 1, 64, 32, window=window)
    _check_attention(c, table, lens, queries, q, out, lse, "f32", 0.125, 0, window, None)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nq", [4, 100])
def test_attention_nan_stays_in_its_rows(cuda_lib, nq):
    # a NaN block is seen by the rows at or after it (and by none past the window); a NaN or infinite
    # query makes its own rows NaN
    rng = np.random.default_rng(5)
    heads, n_kv, dim, page, n, window = 2, 1, 64, 16, 400, 20
    raw, table, c = _filled(rng, [n], page, n_kv, dim)
    blk = (n - nq // 2) // 16
    for which in range(2):
        c._scales(table[0, blk], 0, which)[0] = np.nan
    raw = _t(c.raw)
    q = rng.standard_normal((nq, heads, dim)).astype(np.float32)
    q[0, 1, 3] = np.inf
    q[nq - 1, 0, 0] = np.nan
    out, lse = _attend(cuda_lib, raw, table, [n], [nq], _t(q), heads, n_kv, dim, page, window=window)
    pos = n - nq + np.arange(nq)
    sees = (pos >= blk * 16) & (pos - window + 1 <= blk * 16 + 15)
    bad = np.stack([sees, sees], 1)
    bad[0, 1] = bad[nq - 1, 0] = True
    assert np.array_equal(np.isnan(_np(out)).any(-1), bad) and np.array_equal(np.isnan(_np(out)).all(-1), bad)
    assert np.array_equal(np.isnan(_np(lse)), bad)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nq", [1, 70])
def test_attention_lengths_and_pages_out_of_range(cuda_lib, nq):
    # lengths outside [0, max_kv_len], past the table, a page outside the pool: NaN for that sequence alone
    rng = np.random.default_rng(6)
    lens = [200, 200, 200, 200, 200, 200]
    raw, table, c = _filled(rng, lens, 16, 2, 64)
    given = [200, -1, 257, 250, 200, 200]
    table[4, 3] = c.raw.shape[0]
    table[5, 0] = -7
    q = _t(rng.standard_normal((6 * nq, 2, 64)).astype(np.float32))
    out, lse = _attend(cuda_lib, raw, table, given, [nq] * 6, q, 2, 2, 64, 16, max_kv=256)
    o = _np(out).reshape(6, -1)
    assert np.isfinite(o[0]).all() and np.isnan(o[1:]).all() and np.isnan(_np(lse).reshape(6, -1)[1:]).all()


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("nq,lens", [(1, [5000, 17, 3000]), (3, [900, 1, 5000]), (129, [600, 300, 129])])
def test_attention_repeats_bit_for_bit_on_one_workspace(cuda_lib, nq, lens):
    import torch
    rng = np.random.default_rng(7)
    raw, table, c = _filled(rng, lens, 64, 2, 128)
    q = _t(rng.standard_normal((3 * nq, 6, 128)).astype(np.float32))
    ws = cuda_lib.kv_attention_workspace(3, nq, 5000, 6, 2, 128)
    first = _attend(cuda_lib, raw, table, lens, [nq] * 3, q, 6, 2, 128, 64, max_kv=5000, workspace=ws)
    side = torch.cuda.Stream()
    for i in range(4):
        if i == 2:
            torch.cuda.synchronize()
        stream = side if i >= 2 else None  # the same workspace, later, on another stream
        again = _attend(cuda_lib, raw, table, lens, [nq] * 3, q, 6, 2, 128, 64, max_kv=5000, workspace=ws, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.usefixtures("attn_kernel")
def test_calls_of_other_shapes_share_a_workspace(cuda_lib):
    # whatever one call keeps in the workspace must not count as another's tickets
    import torch
    rng = np.random.default_rng(11)
    shapes = [  # (lengths, queries of each, heads, cache heads, dims, type, window)
        ([900, 1400], [200, 300], 6, 2, 64, "bf16", 0), ([700] * 40, [1] * 40, 8, 8, 64, "f32", 0),
        ([900, 1400], [200, 300], 4, 2, 256, "f32", 0), ([900, 1400], [200, 300], 4, 2, 256, "bf16", 100),
        ([5000], [1], 6, 2, 128, "f16", 0), ([64] * 500, [1] * 500, 2, 2, 64, "f32", 0)]
    size = max([cuda_lib.kv_attention_workspace_bytes(len(lens), max(nq), max(lens), h, kv, d) for lens, nq, h, kv, d, _, _ in shapes]
               + [cuda_lib.token_logprobs_workspace_bytes(r, n, 9) for r, n in ((1, 100000), (700, 300))])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    calls = []
    for lens, nq, heads, n_kv, dim, dtype, window in shapes:
        raw, table, _ = _filled(rng, lens, 32, n_kv, dim)
        q = _t(rng.standard_normal((sum(nq), heads, dim)).astype(np.float32), _dt(dtype))
        calls.append(lambda w, raw=raw, table=table, lens=lens, nq=nq, q=q, h=heads, kv=n_kv, d=dim, win=window:
                     [_np(t) for t in _attend(cuda_lib, raw, table, lens, nq, q, h, kv, d, 32, window=win, workspace=w)])
    for rows, n in ((1, 100000), (700, 300)):
        x = _t(rng.standard_normal((rows, n)).astype(np.float32))

        def scores(w, x=x, rows=rows, n=n):
            out = [torch.full(s, float("nan"), device="cuda") for s in ((rows,), (rows,), (rows, 9))]
            ids = torch.full((rows, 9), -1, dtype=torch.int32, device="cuda")
            w = cuda_lib.token_logprobs_workspace(rows, n, 9) if w is None else w
            cuda_lib.token_logprobs(x, _i32(np.zeros(rows)), out[0], out[1], rows, n, w, 9, ids, out[2])
            return [_np(t) for t in out + [ids]]
        calls.append(scores)
    alone = [c(None) for c in calls]
    for i in list(range(len(calls))) + list(rng.integers(0, len(calls), 24)):
        for a, b in zip(calls[i](ws), alone[i]):
            assert np.array_equal(a, b, equal_nan=True), i


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("n_seqs,nq,heads,n_kv,dim,max_kv", [
    (1, 1, 8, 8, 128, 161), (1, 1, 4, 2, 64, 40000), (24, 1, 8, 8, 64, 9000), (40, 3, 16, 8, 128, 700), (2, 40, 4, 2, 128, 3000),
    (2, 65, 2, 2, 64, 5000), (1, 300, 2, 1, 128, 2000), (40, 1, 8, 8, 64, 16384), (11, 3328, 4, 4, 64, 100)])
def test_attention_workspace_is_enough_for_any_window(cuda_lib, n_seqs, nq, heads, n_kv, dim, max_kv):
    # how a call is cut depends on the window; the workspace's size does not: nothing is written past it
    import torch
    page = 128
    lens = [max_kv - 7 * (i % 3) for i in range(n_seqs)]
    raw = cuda_lib.kv_pages(1, page, n_kv, dim)  # every page the same
    table = torch.zeros(n_seqs, -(-max_kv // page), dtype=torch.int32, device="cuda")
    size = cuda_lib.kv_attention_workspace_bytes(n_seqs, nq, max_kv, heads, n_kv, dim)
    buf = torch.zeros(size + 8192, dtype=torch.uint8, device="cuda")
    buf[size:] = 0x5A
    for dtype in ("f32", "bf16"):
        q = torch.randn(n_seqs * nq, heads, dim, device="cuda").to(_dt(dtype))
        out = torch.full_like(q, 5.0)
        for window in (0, 1, 17, 100, max_kv // 3, max_kv // 2, max_kv - 20, 2 * max_kv):
            cuda_lib.kv_attention(raw, table, _i32(lens), q, out, buf[:size], heads, n_kv, dim, page, max_kv,
                                  cu_q=_i32(np.arange(n_seqs + 1) * nq), max_q=nq, window=window)
            assert (out == 0).all() and (buf[size:] == 0x5A).all(), window


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_many_ragged_prompts(cuda_lib, dtype):
    # prompts whose tiles are dealt out in shares that cut them: empty sequences, single queries, some longer than
    # others, every one checked
    rng = np.random.default_rng(11)
    lens = [0, 700, 65, 1, 1300, 128, 0, 400, 260, 64]
    nq = [0, 150, 65, 1, 70, 128, 0, 3, 260, 64]
    raw, table, c = _filled(rng, lens, 32, 2, 64)
    q = _t(1.5 * rng.standard_normal((sum(nq), 4, 64)).astype(np.float32), _dt(dtype))
    for window in (0, 100):
        out, lse = _attend(cuda_lib, raw, table, lens, nq, q, 4, 2, 64, 32, window=window)
        _check_attention(c, table, lens, nq, q, out, lse, dtype, 0.125, 0, window, None)


@pytest.mark.parametrize("lens,nq,heads,n_kv,dim,dtype,window", [
    ([3000, 17, 0, 900, 1], [1] * 5, 6, 2, 128, "f32", 0),
    ([5000, 40], [1, 1], 4, 4, 64, "bf16", 0),
    ([700, 2100, 64], [5, 3, 9], 6, 3, 96, "f16", 0),
    ([1500, 10, 2600], [1, 0, 4], 8, 2, 256, "bf16", 0),
    ([130, 4000, 2000, 1999], [1] * 4, 12, 4, 192, "f32", 0),
    ([9000, 200], [1, 1], 2, 2, 64, "f32", 0),
    ([2500, 4100, 30], [2, 1, 1], 4, 2, 128, "f32", 3200),
    ([60] * 19 + [4000], [1] * 20, 7, 7, 64, "f16", 0)])
def test_attention_splits_follow_the_lengths(cuda_lib, lens, nq, heads, n_kv, dim, dtype, window):
    # few, uneven sequences with a bound far above their lengths; twice, for the tickets
    import torch
    rng = np.random.default_rng(sum(lens))
    raw, table, c = _filled(rng, lens, 32, n_kv, dim)
    q = _t((2 * rng.standard_normal((sum(nq), heads, dim))).astype(np.float32), _dt(dtype))
    ws = cuda_lib.kv_attention_workspace(len(lens), max(nq), 900000, heads, n_kv, dim)
    first = _attend(cuda_lib, raw, table, lens, nq, q, heads, n_kv, dim, 32, window=window, max_kv=900000, workspace=ws)
    _check_attention(c, table, lens, nq, q, first[0], first[1], dtype, dim ** -0.5, 0.0, window, None)
    again = _attend(cuda_lib, raw, table, lens, nq, q, heads, n_kv, dim, 32, window=window, max_kv=900000, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("n_kv,group,drafts,dim,dtype,bound", [
    (8, 3, 1, 128, "f32", 8000), (8, 1, 1, 64, "bf16", 3100), (4, 4, 4, 128, "f32", 6000), (2, 8, 1, 192, "f32", 6000),
    (4, 4, 4, 96, "f16", 4000), (4, 4, 4, 256, "bf16", 8192)])
def test_attention_workspace_holds_the_parts_of_idle_sequences(cuda_lib, n_kv, group, drafts, dim, dtype, bound):
    # as many tiles of rows as SMs, a CTA for each: what sequences without queries or with fewer leave goes to the
    # long ones, which are cut, and their parts need room
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = drafts * group
    R = 16 if dtype != "f32" and rows > 8 else 8  # rows of a tile
    n_seqs = sms // (n_kv * -(-rows // R))
    if n_seqs * n_kv * -(-rows // R) != sms:
        pytest.skip("no such number of sequences")
    rng = np.random.default_rng(n_kv + dim)
    lens = rng.integers(1, 150, n_seqs)
    nq = rng.integers(0, 2, n_seqs) if drafts == 1 else np.minimum(1, rng.integers(0, 4, n_seqs))
    long = rng.permutation(n_seqs)[:4]
    lens[long[:2]], nq[long[:2]] = [bound, bound - 333], [drafts, 1]
    lens[long[2:]], nq[long[2:]] = 2000, [0, drafts]
    raw, table, c = _filled(rng, lens, 64, n_kv, dim)
    q = _t(rng.standard_normal((nq.sum(), n_kv * group, dim)).astype(np.float32), _dt(dtype))
    size = cuda_lib.kv_attention_workspace_bytes(n_seqs, drafts, bound, n_kv * group, n_kv, dim)
    assert size - size // 8 // 256 * 256 >= sms * R * (dim + 2) * 4  # a part for each CTA; nothing is launched otherwise
    buf = torch.zeros(size + (8 << 20), dtype=torch.uint8, device="cuda")
    buf[size:] = 0x5A
    first = None
    for _ in range(2):
        out, lse = _attend(cuda_lib, raw, table, lens, nq, q, n_kv * group, n_kv, dim, 64, max_kv=bound, workspace=buf[:size],
                           max_q=drafts)
        assert (buf[size:] == 0x5A).all()
        first = first or (out, lse)
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    _check_attention(c, table, lens, nq, q, out, lse, dtype, dim ** -0.5, 0, 0, None)


def test_attention_splits_with_lengths_out_of_range(cuda_lib):
    import torch
    rng = np.random.default_rng(2)
    lens = [1000, 3000, 2000, 40]
    raw, table, c = _filled(rng, lens, 32, 2, 64)
    q = _t(rng.standard_normal((4, 4, 64)).astype(np.float32))
    told = [1000, 3001 + 32 * 40, -1, 40]  # the second past its table row, the third negative
    out, lse = _attend(cuda_lib, raw, table, told, [1] * 4, q, 4, 2, 64, 32, max_kv=900000)
    assert torch.isnan(out[[1, 2]]).all() and torch.isnan(lse[[1, 2]]).all()
    for s in (0, 3):
        _check_attention(c, table[s:s + 1], [lens[s]], [1], q[s:s + 1], out[s:s + 1], lse[s:s + 1], "f32", 0.125, 0.0, 0, None)


@pytest.mark.usefixtures("attn_kernel")
@pytest.mark.parametrize("lens,nq,max_q,dtype", [([300, 40], [2, 1], 1, "f32"), ([300, 40], [9, 5], 4, "f16"),
                                                 ([900, 400, 77], [200, 90, 30], 60, "bf16"), ([900, 400], [200, 150], 101, "f32")])
def test_attention_of_queries_past_max_q(cuda_lib, lens, nq, max_q, dtype):
    # a sequence's rows past max_q are not written; the others stand where all of them put them
    rng = np.random.default_rng(max_q)
    raw, table, c = _filled(rng, lens, 32, 2, 64)
    q = _t(rng.standard_normal((sum(nq), 6, 64)).astype(np.float32), _dt(dtype))
    out, lse = _attend(cuda_lib, raw, table, lens, nq, q, 6, 2, 64, 32, max_q=max_q)
    full, full_lse = _attend(cuda_lib, raw, table, lens, nq, q, 6, 2, 64, 32)
    _check_attention(c, table, lens, nq, q, full, full_lse, dtype, 0.125, 0, 0, None)
    cu = np.concatenate([[0], np.cumsum(nq)])
    for s in range(len(lens)):
        n = min(nq[s], max_q)
        for got, whole in ((out, full), (lse, full_lse)):
            assert (got[cu[s] + n:cu[s + 1]] == 5).all()
            got[cu[s] + n:cu[s + 1]] = whole[cu[s] + n:cu[s + 1]]  # for the comparison below
    _check_attention(c, table, lens, nq, q, out, lse, dtype, 0.125, 0, 0, None)


@pytest.mark.usefixtures("attn_kernel")
def test_attention_strided_rows(cuda_lib):
    # q and out inside wider buffers; other elements stay
    import torch
    rng = np.random.default_rng(8)
    raw, table, c = _filled(rng, [130, 70], 32, 2, 64)
    wide = _t(rng.standard_normal((2, 8, 64)).astype(np.float32))
    q = wide[:, 2:6]
    out = torch.full((2, 9, 64), 3.0, device="cuda")
    ws = cuda_lib.kv_attention_workspace(2, 1, 130, 4, 2, 64)
    cuda_lib.kv_attention(raw, _i32(table), _i32([130, 70]), q, out[:, 1:5], ws, 4, 2, 64, 32, 130)
    lse = torch.empty(2, 4, device="cuda")
    plain = torch.empty(2, 4, 64, device="cuda")
    cuda_lib.kv_attention(raw, _i32(table), _i32([130, 70]), q.contiguous(), plain, ws, 4, 2, 64, 32, 130, lse=lse)
    assert torch.equal(out[:, 1:5], plain) and (out[:, 0] == 3).all() and (out[:, 5:] == 3).all()
    _check_attention(c, table, [130, 70], [1, 1], q.contiguous(), plain, lse, "f32", 0.125, 0, 0, None)


def test_attention_between_slices_of_one_buffer(cuda_lib):
    # the queries and the output beside one another in wide rows
    import torch
    rng = np.random.default_rng(13)
    lens = [130, 70, 5]
    raw, table, c = _filled(rng, lens, 32, 2, 64)
    wide = _t(rng.standard_normal((3, 11, 64)).astype(np.float32))
    before = wide.clone()
    q, out = wide[:, 1:5], wide[:, 6:10]
    plain = torch.empty(3, 4, 64, device="cuda")
    ws = cuda_lib.kv_attention_workspace(3, 1, 130, 4, 2, 64)
    cuda_lib.kv_attention(raw, _i32(table), _i32(lens), q.contiguous(), plain, ws, 4, 2, 64, 32, 130)
    cuda_lib.kv_attention(raw, _i32(table), _i32(lens), q, out, ws, 4, 2, 64, 32, 130)
    assert torch.equal(out, plain)
    assert torch.equal(wide[:, :6], before[:, :6]) and torch.equal(wide[:, 10], before[:, 10])


@pytest.mark.usefixtures("attn_kernel")
def test_cache_offsets_past_32_bits(cuda_lib):
    # pages beyond 4 GB: append, read and attention reach the same tokens
    import torch
    page, n_kv, dim = 128, 8, 128
    rec = cuda_lib.kv_page_bytes(page, n_kv, dim)
    n_pages = (5 << 30) // rec
    raw = torch.empty(n_pages, rec, dtype=torch.uint8, device="cuda")
    table = _i32([[n_pages - 1, n_pages - 7], [n_pages - 2, 0]])
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.randn(400, n_kv, dim, device="cuda", generator=g)
    v = torch.randn(400, n_kv, dim, device="cuda", generator=g)
    cu = _i32([0, 200, 400])
    small = torch.empty(4, rec, dtype=torch.uint8, device="cuda")
    low = _i32([[3, 1], [2, 0]])
    q = torch.randn(2, 8, dim, device="cuda", generator=g)
    got = []
    for pool, tab in ((raw, table), (small, low)):
        cuda_lib.kv_append(pool, tab, _i32([200, 200]), k, v, n_kv, dim, page, cu_new=cu, max_new=200)
        ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        cuda_lib.kv_read(pool, tab, None, cu, ko, vo, n_kv, dim, page, 200)
        ws = cuda_lib.kv_attention_workspace(2, 1, 200, 8, n_kv, dim)
        cuda_lib.kv_attention(pool, tab, _i32([200, 200]), q, out, ws, 8, n_kv, dim, page, 200)
        got.append((ko, vo, out))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0] - k).abs().max() <= k.abs().max() / 127


# ------------------------------------------------------------------ log probabilities

def _logprobs(qdq, x, tokens, k, entropy=True):
    import torch
    rows, n = x.shape
    lp, ent = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    ti, tl = torch.full((rows, k), -5, dtype=torch.int32, device="cuda"), torch.full((rows, k), 9.0, device="cuda")
    ws = qdq.token_logprobs_workspace(rows, n, k)
    for _ in range(2):  # the second call finds the workspace as the first left it
        qdq.token_logprobs(x, _i32(tokens), lp, ent, rows, n, ws, k=k, top_index=ti, top_logprob=tl)
    return [_np(t) for t in (lp, ent, ti, tl)]


def _check_logprobs(x, tokens, k, got):
    lp, ent, ti, tl = ref.logprobs(x, tokens, k)
    n = x.shape[1]
    mag = np.array([np.abs(r[np.isfinite(r)]).max() if np.isfinite(r).any() else 0 for r in x])
    t = (n / 256 + 64) * U + 2.0 ** -21 * (mag + 1)
    assert np.array_equal(got[2], ti)
    with np.errstate(invalid="ignore"):
        _within(got[0], lp, t)
        _within(got[1], ent, t * (4 + 2 * ent))
        _within(got[3], tl, t[:, None])


@pytest.mark.parametrize("rows,n,k,dtype", [
    (1, 1, 1, "f32"), (2, 2, 0, "f32"), (3, 5, 5, "bf16"), (4, 64, 64, "f16"), (2, 1000, 7, "f32"), (3, 4095, 33, "f32"),
    (2, 4097, 20, "bf16"), (1, 128256, 20, "f32"), (1, 128256, 64, "bf16"), (5, 50001, 1, "f16"), (40, 8200, 5, "f32"),
    (1300, 777, 3, "bf16"), (9, 200003, 13, "f32")])
def test_logprobs(cuda_lib, rows, n, k, dtype):
    rng = np.random.default_rng(rows + n)
    x = _t((2.5 * rng.standard_normal((rows, n))).astype(np.float32), _dt(dtype))  # 16-bit types: many ties
    tokens = rng.integers(0, n, rows)
    tokens[-1] = n - 1
    _check_logprobs(_np(x), tokens, k, _logprobs(cuda_lib, x, tokens, k))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (0, 1), (2, 8)])
def test_logprobs_alignment(cuda_lib, dtype, offset, pad):
    rng = np.random.default_rng(offset + pad)
    rows, n = 6, 4099
    buf = _t((3 * rng.standard_normal(rows * (n + pad) + offset)).astype(np.float32), _dt(dtype))
    x = buf[offset:].as_strided((rows, n), (n + pad, 1))
    tokens = rng.integers(0, n, rows)
    _check_logprobs(_np(x), tokens, 9, _logprobs(cuda_lib, x, tokens, 9))


@pytest.mark.parametrize("n,k", [(300, 64), (5000, 20), (20000, 64), (128256, 40)])
def test_logprobs_orders_that_defeat_the_bound(cuda_lib, n, k):
    # constant rows, rising, falling, the best in one thread's share, masked (-inf) but for fewer than k
    rows = np.zeros((7, n), np.float32)
    rows[1] = np.arange(n) / n
    rows[2] = -np.arange(n) / n
    rows[3, :: max(1, n // 100)] = 5
    rows[4] = -np.inf
    rows[4, n // 2:n // 2 + 3] = [1, 2, 1]
    rows[5] = np.where(np.arange(n) % 1024 < 4, np.arange(n) / 1000, -3)
    rows[6] = -1e30
    rows[6, 7] = -0.0
    rows[6, 9] = 0.0
    tokens = np.array([0, n - 1, 0, 1, n // 2 + 1, 4, 9])
    _check_logprobs(rows, tokens, k, _logprobs(cuda_lib, _t(rows), tokens, k))


def test_logprobs_not_finite_and_tokens_out_of_range(cuda_lib):
    n, k = 9000, 6
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, n)).astype(np.float32)
    x[1, [50, 8000]] = np.nan
    x[2, 77] = np.inf
    x[3] = -np.inf
    tokens = np.array([5, 5, 5, 5, -1, n])
    got = _logprobs(cuda_lib, _t(x), tokens, k)
    _check_logprobs(x, tokens, k, got)
    assert np.isnan(got[0]).tolist() == [False, True, True, True, True, True]
    assert np.isnan(got[1]).tolist() == [False, True, True, True, False, False]


def test_logprobs_rows_past_32_bits(cuda_lib):
    import torch
    n, stride = 5000, (1 << 31) + 3
    buf = torch.empty(2 * stride + n, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, n), (stride, 1))
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, n)).astype(np.float32)
    x.copy_(_t(v))
    tokens = np.array([0, 1, n - 1])
    _check_logprobs(_np(x), tokens, 4, _logprobs(cuda_lib, x, tokens, 4))


# ------------------------------------------------------------------ together

def test_empty_tensors(cuda_lib):
    # no rows, no sequences, no queries: nothing to do, and nothing to refuse
    import torch

    def f(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    none, table, pages = f(0, 128), f(2, 3, dtype=torch.int32), cuda_lib.kv_pages(4, 16, 2, 64)
    cuda_lib.rms_norm(none, None, f(0, 128), 0, 128, residual=f(0, 128), sum_out=f(0, 128))
    cuda_lib.rms_norm(none, f(128), None, 0, 128, q8_out=f(0, dtype=torch.uint8))
    before = pages.clone()
    for tab, lens, most in ((table, _i32([0, 0]), 0), (table[:0], _i32([]), 1)):
        cu = _i32([0] * (len(tab) + 1))
        cuda_lib.kv_append(pages, tab, lens, none, none, 2, 64, 16, cu_new=cu, max_new=most)
        cuda_lib.kv_read(pages, tab, None, cu, f(0, 128), f(0, 128), 2, 64, 16, most)
        ws = cuda_lib.kv_attention_workspace(len(tab), most, 48, 2, 2, 64)
        cuda_lib.kv_attention(pages, tab, lens, none, f(0, 128), ws, 2, 2, 64, 16, 48, cu_q=cu, max_q=most, lse=f(0, 2))
    cuda_lib.token_logprobs(f(0, 500), _i32([]), f(0), f(0), 0, 500, cuda_lib.token_logprobs_workspace(0, 500, 3), 3,
                            f(0, 3, dtype=torch.int32), f(0, 3))
    torch.cuda.synchronize()
    assert torch.equal(pages, before)


def test_operators_on_a_stream_of_their_own_in_a_graph(cuda_lib):
    # the decode chain captured into a CUDA graph on a side stream gives what the calls give
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    n, n_kv, heads, dim, page = 3, 2, 6, 64, 32
    width = (heads + 2 * n_kv) * dim
    x = torch.randn(n, width, device="cuda", generator=g)
    out, qkv = torch.empty(n, heads, dim, device="cuda"), torch.empty(n, width, device="cuda")
    table, lens = _i32([[0, 1], [2, 3], [4, 5]]), _i32([40, 33, 1])
    ws = cuda_lib.kv_attention_workspace(n, 1, 64, heads, n_kv, dim)
    k0 = torch.randn(39 + 32, n_kv, dim, device="cuda", generator=g)

    def chain(pages):
        cuda_lib.rms_norm(x, None, qkv, n, width)
        k = qkv[:, heads * dim:(heads + n_kv) * dim]
        v = qkv[:, (heads + n_kv) * dim:]
        cuda_lib.kv_append(pages, table, lens, k, v, n_kv, dim, page)
        cuda_lib.kv_attention(pages, table, lens, qkv[:, :heads * dim], out, ws, heads, n_kv, dim, page, 64)

    def fresh():
        p = cuda_lib.kv_pages(6, page, n_kv, dim)
        cuda_lib.kv_append(p, table, _i32([39, 32, 0]), k0, k0, n_kv, dim, page, cu_new=_i32([0, 39, 71, 71]), max_new=39)
        return p

    a, b = fresh(), fresh()
    chain(a)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        chain(b)
    graph.replay()
    graph.replay()  # appending the same tokens twice changes nothing
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(a, b)
