"""The decode example: its steps from a graph and without one agree, and a step's stages are right.

Stages are checked from the step's own buffers against float64 forms, with the bounds of the operators'
own tests (u = 2^-24): the norm 65 u |y|, the logits 1e-5 sum |w||x|, log probabilities
t = (n / 256 + 64) u + 2^-21 (max |x| + 1), attention (2 d + 2^-17) sum p|v| + u |o| + 2^-39 127 n z
with d = 2^-18 a + 2^-20, a = scale sum |q||k| + |bias|, and a cached value half a code of its block.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _np(t):
    return t.double().cpu().numpy()


@pytest.fixture(scope="module")
def model():
    from examples import decode
    z = decode.Sizes(n_embd=256, n_ff=512, n_heads=4, n_kv=2, head_dim=64, n_vocab=896, n_layers=2, page_tokens=32)
    return decode, z, decode.random_weights(z, 3)


def _started(model, lens=(70, 1, 17), max_len=96):
    import synth
    decode, z, w = model
    dec = decode.Decoder(z, w, len(lens), max_len)
    rng = np.random.default_rng(5)
    lp = dec.prompt([synth.token_ids(rng, n, z.n_vocab) for n in lens])
    assert [len(x) for x in lp] == [n - 1 for n in lens]
    assert all(bool((x <= 0).all()) for x in lp)
    return dec


def test_graph_and_plain_steps_agree(model):
    import ggml_quantized_dequant_gb300 as qdq
    a, b = _started(model), _started(model)
    ids, lps = a.generate(9)
    ids2, lps2 = b.generate(9, graph=False)
    assert (ids == ids2).all() and (lps == lps2).all()
    assert a.kv_len.tolist() == [79, 10, 26]
    assert qdq.pipeline_timeouts() == 0
    with pytest.raises(ValueError):
        a.generate(96)


def test_a_step_against_float64(model):
    import torch

    import ggml_quantized_dequant_gb300 as qdq
    decode, z, _ = model
    dec = _started(model)
    dec.generate(5, graph=False)
    h, n = _np(dec.h), _np(dec.n)
    want = h / np.sqrt((h * h).mean(1, keepdims=True) + z.eps) * _np(dec.gain)
    assert np.all(np.abs(n - want) <= 65 * U * np.abs(want))

    W = torch.empty(z.n_vocab, z.n_embd, device="cuda")
    qdq.q8_0_dequant(dec.head, W, z.n_vocab, z.n_embd)
    W, x = _np(W), _np(dec.logits)
    assert np.all(np.abs(x - n @ W.T) <= 1e-5 * (np.abs(n) @ np.abs(W).T))

    t = (z.n_vocab / 256 + 64) * U + 2.0 ** -21 * (np.abs(x).max() + 1)
    lse = np.log(np.exp(x - x.max(1, keepdims=True)).sum(1)) + x.max(1)
    order = np.argsort(-x, 1, kind="stable")[:, :dec.top]
    assert (dec.top_id.cpu().numpy() == order).all()
    assert np.all(np.abs(_np(dec.top_lp) - (np.take_along_axis(x, order, 1) - lse[:, None])) <= t)
    assert np.all(np.abs(_np(dec.given_lp) - (x[:, 0] - lse)) <= t)
    assert (dec.ids.cpu().numpy() == order[:, 0]).all()

    lens = dec.kv_len.tolist()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    k, v = (torch.empty(sum(lens), z.n_k, device="cuda") for _ in range(2))
    qdq.kv_read(dec.caches[-1], dec.table, None, cu, k, v, z.n_kv, z.head_dim, z.page_tokens, max(lens))
    k, v, q, got = _np(k), _np(v), _np(dec.q), _np(dec.a)
    for s, m in enumerate(lens):
        ks, vs = (y[sum(lens[:s]):sum(lens[:s + 1])].reshape(m, z.n_kv, z.head_dim) for y in (k, v))
        block = ks[(m - 1) // 16 * 16:]  # the last token's block: a code is at most its largest value / 127
        new = _np(dec.k)[s].reshape(z.n_kv, z.head_dim)
        top = np.maximum(np.abs(block).max((0, 2)), np.abs(new).max(1))[:, None]
        assert np.all(np.abs(ks[-1] - new) <= top / 127 * 0.5001)
        for head in range(z.n_heads):
            kv = head // (z.n_heads // z.n_kv)
            qh = q[s].reshape(z.n_heads, z.head_dim)[head]
            bias = float(dec.slopes[head]) * (m - 1 - np.arange(m))
            sc = z.head_dim ** -0.5
            e = sc * ks[:, kv] @ qh - bias
            p = np.exp(e - e.max())
            p /= p.sum()
            o = p @ vs[:, kv]
            d = 2.0 ** -18 * (sc * np.abs(ks[:, kv]) @ np.abs(qh) + bias).max() + 2.0 ** -20
            z_most = (p[:, None] * np.abs(vs[:, kv])).max()
            bound = (2 * d + 2.0 ** -17) * (p @ np.abs(vs[:, kv])) + U * np.abs(o) + 2.0 ** -39 * 127 * m * z_most
            assert np.all(np.abs(got[s].reshape(z.n_heads, z.head_dim)[head] - o) <= bound)


def test_recall_and_refusals(model):
    import torch

    import ggml_quantized_dequant_gb300 as qdq
    decode, z, w = model
    dec = _started(model)
    dec.generate(2, graph=False)
    got = _np(dec.recall())
    S = torch.empty(dec.n_states, z.n_embd, device="cuda")
    qdq.q8_0_dequant(dec.states, S, dec.n_states, z.n_embd)
    S, n = _np(S), _np(dec.n)
    assert np.all(np.abs(got - n @ S.T) <= 1e-5 * (np.abs(n) @ np.abs(S).T))
    with pytest.raises(ValueError):
        decode.Decoder(z, w, 9, 64)
    with pytest.raises(ValueError):
        dec.prompt([[1, 2]])
