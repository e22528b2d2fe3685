"""The decode example's prompt pass, call by call, against float64 forms.

Every call of the library is recorded with copies of its tensors before and after it.  What a call is
given has to be, bit for bit, what an earlier one made; what it makes is checked from what it was given:
embedding rows and the residual's sums exactly (one f32 addition), norms within 65 u |y| (u = 2^-24), matrix
products within 4e-3 sum |w||x|, the SwiGLU of two such products g + dg, u + du within |du| |silu(g)| + 1.1 |dg| (|u| + |du|)
+ 8 u |mid| (|silu'| < 1.1), the cache's bytes as its definition's, attention within (2 d + 2^-17) sum p|v|
+ u |o| + 2^-39 127 n z with d = 2^-18 a + 2^-20, log probabilities within (n / 256 + 64) u + 2^-21 (max |x| + 1).
"""
import numpy as np
import pytest

from oracle import decode_oracle as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LENS = (70, 1, 17, 33)


class Recorder:
    """The library; calls that launch something are kept as (name, arguments before, arguments after)."""

    def __init__(self, qdq):
        self.qdq, self.calls = qdq, []

    def __getattr__(self, name):
        f = getattr(self.qdq, name)
        if not callable(f) or "workspace" in name or name.endswith("_bytes") or name in ("kv_pages", "upload_q4k"):
            return f

        def call(*args, **kw):
            import torch

            def copies():
                return [a.clone() if torch.is_tensor(a) else a for a in args], \
                    {k: a.clone() if torch.is_tensor(a) else a for k, a in kw.items()}

            before = copies()
            f(*args, **kw)
            self.calls.append((name, before, copies()))
        return call


def _np(t):
    return t.double().cpu().numpy()


def _near(got, want, bound):
    assert np.all(np.abs(_np(got) - want) <= bound), np.max(np.abs(_np(got) - want) / np.maximum(bound, 1e-300))


def test_prompt_call_by_call(cuda_lib, monkeypatch):
    import torch

    import synth
    from examples import decode
    z = decode.Sizes(n_embd=256, n_ff=512, n_heads=4, n_kv=2, head_dim=64, n_vocab=896, n_layers=2, page_tokens=32)
    weights = decode.random_weights(z, 8)
    dec = decode.Decoder(z, weights, len(LENS), 96)
    recorder = Recorder(cuda_lib)
    monkeypatch.setattr(decode, "qdq", recorder)
    rng = np.random.default_rng(9)
    prompts = [synth.token_ids(rng, n, z.n_vocab) for n in LENS]
    returned = dec.prompt(prompts)
    calls = iter(recorder.calls)
    M, cu = sum(LENS), np.cumsum([0, *LENS])

    def following(name):
        got, before, after = next(calls)
        assert got == name
        return before, after

    def dense(kind, packed, n_out, n_in):
        w = torch.empty(n_out, n_in, device="cuda")
        getattr(cuda_lib, kind + "_dequant")(packed, w, n_out, n_in)
        return w

    def product(weight, x, n_out, kind="q4k"):
        (a, _), (b, _) = following(kind + "_gemm_batch")
        n_in = x.shape[1]
        assert torch.equal(a[0], weight) and torch.equal(a[1], x) and a[4:7] == [n_out, n_in, M]
        w = _np(dense(kind, weight, n_out, n_in))
        _near(b[2], _np(x) @ w.T, 4e-3 * (np.abs(_np(x)) @ np.abs(w).T))
        return b[2]

    def norm(x, residual, gain, packed=False):
        (a, kw), (b, after) = following("rms_norm")
        assert torch.equal(a[0], x) and torch.equal(a[1], gain) and a[3:6] == [M, z.n_embd, z.eps]
        h = x
        if residual is not None:
            assert torch.equal(kw["residual"], residual)
            h = residual + x
            if not packed:
                assert torch.equal(after["sum_out"], h)
        want = _np(h) / np.sqrt((_np(h) ** 2).mean(1, keepdims=True) + z.eps) * _np(gain)
        _near(b[2], want, 65 * U * np.abs(want))
        if packed:  # half a step of d = f16(m / 127), its rounding and the norm's, as in the norm's own test
            assert torch.equal(after["q8_out"], dec.states)
            m = np.abs(want.reshape(M, -1, 32)).max(-1, keepdims=True)
            step = (m / 127 * (0.5 + 127 * 2.0 ** -11) * (1 + 2.0 ** -10) + 128 * 2.0 ** -25) * np.ones((1, 1, 32))
            _near(dense("q8_0", dec.states, M, z.n_embd), want, step.reshape(M, -1) + 65 * U * np.abs(want))
        return h, b[2]

    embed, layers, gain, head = weights
    (a, _), (b, _) = following("q6k_get_rows")
    ids = np.concatenate(prompts)
    assert a[1].tolist() == ids.tolist()
    h, fresh = b[2], None
    assert torch.equal(h, dense("q6k", embed, z.n_vocab, z.n_embd)[torch.from_numpy(ids).long().cuda()])
    pool = [ref.Cache(np.zeros(c.shape, np.uint8), z.page_tokens, z.n_kv, z.head_dim) for c in dec.caches]
    table = dec.table.cpu().numpy()
    for i, w in enumerate(layers):
        h, n = norm(h, None, w["n1"]) if fresh is None else norm(fresh, h, w["n1"])
        q, k, v = product(w["q"], n, z.n_q), product(w["k"], n, z.n_k), product(w["v"], n, z.n_k)
        (a, kw), (b, _) = following("kv_append")
        assert torch.equal(a[3], k) and torch.equal(a[4], v) and a[2].tolist() == list(LENS)
        assert kw["cu_new"].tolist() == cu.tolist() and kw["max_new"] == max(LENS)
        kf, vf = (x.cpu().numpy().reshape(M, z.n_kv, z.head_dim) for x in (k, v))
        pool[i].append(table, np.array(LENS), cu, kf, vf)
        assert np.array_equal(b[0].cpu().numpy().reshape(pool[i].raw.shape), pool[i].raw)
        assert torch.equal(b[0], dec.caches[i])
        (a, kw), (b, _) = following("kv_attention")
        assert torch.equal(a[0], dec.caches[i]) and torch.equal(a[3], q) and a[2].tolist() == list(LENS)
        assert kw["cu_q"].tolist() == cu.tolist()
        for s, m in enumerate(LENS):
            at = slice(cu[s], cu[s + 1])
            kk, vv = pool[i].read(table, s, 0, m)
            o, _, av, mag, zz = ref.attention(_np(q[at]).reshape(m, z.n_heads, -1), kk, vv, np.arange(m), z.head_dim ** -0.5,
                                              slopes=_np(dec.slopes))
            d = 2.0 ** -18 * mag + 2.0 ** -20
            _near(b[4][at].reshape(m, z.n_heads, -1), o,
                  (2 * d + 2.0 ** -17)[..., None] * av + U * np.abs(o) + 2.0 ** -39 * 127 * m * zz[..., None])
        h, n = norm(product(w["o"], b[4], z.n_embd), h, w["n2"])
        (a, _), (b, _) = following("q4k_swiglu_batch")
        assert torch.equal(a[0], w["g"]) and torch.equal(a[1], w["u"]) and torch.equal(a[2], n)
        x, mid = _np(n), b[3]
        gw, uw = (_np(dense("q4k", w[m], z.n_ff, z.n_embd)) for m in "gu")
        g, u, dg, du = x @ gw.T, x @ uw.T, 4e-3 * (np.abs(x) @ np.abs(gw).T), 4e-3 * (np.abs(x) @ np.abs(uw).T)
        silu = g / (1 + np.exp(-g))
        _near(mid, silu * u, du * np.abs(silu) + 1.1 * dg * (np.abs(u) + du) + 8 * U * np.abs(silu * u))
        fresh = product(w["d"], mid, z.n_embd)
    _, n = norm(fresh, h, gain, packed=True)
    logits = product(head, n, z.n_vocab, "q8_0")
    (a, _), (b, _) = following("token_logprobs")
    assert torch.equal(a[0], logits) and next(calls, None) is None
    x = _np(logits)
    t = (z.n_vocab / 256 + 64) * U + 2.0 ** -21 * (np.abs(x).max() + 1)
    lse = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1)) + x.max(1)
    for s, p in enumerate(prompts):
        rows = np.arange(cu[s], cu[s + 1] - 1)
        assert len(returned[s]) == len(p) - 1
        _near(returned[s], x[rows, p[1:]] - lse[rows], t)
        best = int(np.argmax(x[cu[s + 1] - 1]))
        assert int(dec.ids[s]) == best
    assert dec.kv_len.tolist() == list(LENS)
