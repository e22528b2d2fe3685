"""Cases that time the operators around the quantised projections of a decode step.

Four operators, each in a plain form of elementary torch operations and as calls of this
repository's library:

* ``attend``: attention of query tokens over a paged key/value cache held in 8 bits, one f32
  scale for each block of 16 tokens and head (optional tanh cap of the scores, distance bias
  and sliding window);
* ``append``: new keys and values quantised into that cache, then read back as the values the
  cache stands for;
* ``norm``: root-mean-square norm with the residual's addition, to the input's type or to a
  packed Q8_0 matrix;
* ``logprobs``: log probabilities of given tokens with the entropy and the top alternatives.

Cache layout: a page holds ``page`` tokens; in it each key/value head has one record of
``align128(2 * page * dim + 8 * page / 16)`` bytes: key codes (page x dim int8), value codes
(page x dim int8), key scales (page / 16 f32), value scales (page / 16 f32).  Value = code * scale.
Query token i of a sequence with n queries and kv_len cached tokens stands at position
kv_len - n + i and sees the keys at positions up to its own.
"""
import math

import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------------ cases

def _attend(seqs, queries, lo, hi, heads, kv_heads, dim, page, dtype, softcap=0.0, window=0, bias=False):
    return {"op": "attend", "seqs": seqs, "queries": queries, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "softcap": softcap, "window": window, "bias": bias}


def _append(seqs, old_lo, old_hi, new_lo, new_hi, kv_heads, dim, page, dtype):
    return {"op": "append", "seqs": seqs, "old_lo": old_lo, "old_hi": old_hi, "new_lo": new_lo,
            "new_hi": new_hi, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}


def _norm(rows, n, dtype, residual, q8):
    return {"op": "norm", "rows": rows, "n": n, "dtype": dtype, "residual": residual, "q8": q8}


def _logprobs(rows, n, k, dtype):
    return {"op": "logprobs", "rows": rows, "n": n, "k": k, "dtype": dtype}


def listed():
    return [
        # one user's decode step early in a conversation: 3072-wide activations as 24 heads of 128, 1024-wide K and V
        {"name": "attend one token"} | _attend(1, 1, 777, 777, 24, 8, 128, 64, "f32"),
        # a serving batch's decode step, sequences of every length up to 8K
        {"name": "attend batch"} | _attend(48, 1, 1, 8191, 24, 8, 128, 64, "f32"),
        # one long document, one token at a time
        {"name": "attend long"} | _attend(1, 1, 131071, 131071, 32, 8, 128, 128, "bf16"),
        # drafted tokens verified together: few queries per sequence, capped scores, a window, small heads
        {"name": "attend drafts"} | _attend(16, 5, 200, 6001, 16, 2, 64, 32, "f16", softcap=30.0, window=1500),
        # a prompt's chunk over what is cached of it
        {"name": "attend prompt"} | _attend(2, 512, 3500, 4600, 24, 8, 128, 64, "bf16"),
        # the cache's side of a decode step: one token for each sequence
        {"name": "append tokens"} | _append(48, 0, 8190, 1, 1, 8, 128, 64, "f32"),
        # the cache's side of a prompt batch
        {"name": "append prompts"} | _append(6, 0, 500, 900, 3001, 8, 128, 64, "bf16"),
        # between two projections of one decode step
        {"name": "norm one row"} | _norm(1, 3072, "f32", True, False),
        # a prompt's norm, wide rows
        {"name": "norm prompt"} | _norm(4096, 8192, "bf16", True, False),
        # a prompt's norm kept as a Q8_0 matrix
        {"name": "norm to Q8_0"} | _norm(1500, 3072, "f32", True, True),
        # the last token's answer: its log probability and twenty alternatives
        {"name": "logprobs one row"} | _logprobs(1, 128256, 20, "f32"),
        # a prompt scored token by token
        {"name": "logprobs prompt"} | _logprobs(300, 128256, 5, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "norm", "logprobs"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    if op == "attend":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        queries = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
        seqs = _log(rng, 1, 64) if queries <= 8 else rng.randint(1, 3)
        hi = _log(rng, max(queries, 17), max(queries + 1, min(100000, (40 << 20) // (seqs * kv_heads * dim))) if queries <= 8
                  else 4500)
        lo = max(queries, 1) if seqs > 1 else hi
        return _attend(seqs, queries, min(lo, hi), hi, heads, kv_heads, dim, page, dtype,
                       softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, _log(rng, 16, 4096)]),
                       bias=rng.random() < 0.3)
    if op == "append":
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        page = rng.choice([16, 32, 64, 128])
        if rng.random() < 0.5:
            seqs, new_lo, new_hi = _log(rng, 1, 128), 1, rng.choice([1, 1, 4])
        else:
            seqs, new_lo, new_hi = rng.randint(1, 8), 1, _log(rng, 17, 1000)
        return _append(seqs, 0, _log(rng, 1, 2000), new_lo, new_hi, kv_heads, dim, page, dtype)
    if op == "norm":
        rows = _log(rng, 1, 4096)
        n = 32 * _log(rng, 4, 256)
        q8 = rng.random() < 0.4
        return _norm(rows, n if q8 else n + rng.choice([0, 0, 1, 8, 20]), dtype, rng.random() < 0.7, q8)
    n = _log(rng, 1000, 160000)
    return _logprobs(max(1, _log(rng, 1, max(1, min(2000, (36 << 20) // n)))), n, rng.choice([0, 1, 5, 20, 64]), dtype)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], spread evenly and out of order, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _kv_lens(c):
    return _spread(c["seqs"], c["lo"], c["hi"])


def _record(page, dim):
    return (2 * page * dim + 8 * (page // BLOCK) + 127) // 128 * 128


# ------------------------------------------------------------------------------ inputs

def _cache(g, lens, page, kv_heads, dim):
    """A pool of pages in random order and each sequence's page numbers (-1 past its end); the last page is spare."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 2
    rec = _record(page, dim)
    pages = torch.zeros(n_pages, kv_heads, rec, dtype=torch.uint8, device="cuda")
    codes = torch.empty(n_pages, kv_heads, 2 * page * dim, device="cuda").normal_(0, 32.0, generator=g)
    pages[:, :, : 2 * page * dim] = codes.round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    del codes
    nb = page // BLOCK
    scales = (torch.randn(n_pages, kv_heads, 2 * nb, device="cuda", generator=g) * 0.25).exp() / 32
    pages[:, :, 2 * page * dim: 2 * page * dim + 8 * nb] = scales.contiguous().view(torch.uint8)
    order = torch.randperm(n_pages - 1, device="cuda", generator=g).to(torch.int32)
    width = max(1, max(need))
    at = [[0] * width for _ in lens]
    first = 0
    for i, m in enumerate(need):
        at[i] = list(range(first, first + m)) + [-1] * (width - m)
        first += m
    at = torch.tensor(at, device="cuda")
    table = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32))
    return pages, table.contiguous()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed + 1) + 17)
    t = DTYPES[c["dtype"]]
    st = {"c": c}

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if c["op"] == "attend":
        lens = _kv_lens(c)
        st["pages"], st["table"] = _cache(g, lens, c["page"], c["kv_heads"], c["dim"])
        st["kv_len"] = _ints(lens)
        st["cu_q"] = _ints([i * c["queries"] for i in range(c["seqs"] + 1)])
        rows = c["seqs"] * c["queries"]
        st["q"] = (randn(rows, c["heads"], c["dim"]) * 1.5).to(t)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["heads"]) for h in range(c["heads"])],
                                    device="cuda") if c["bias"] else None
        st["out"] = torch.empty(rows, c["heads"], c["dim"], dtype=t, device="cuda")
        st["lse"] = torch.empty(rows, c["heads"], device="cuda")
    elif c["op"] == "append":
        old = _spread(c["seqs"], c["old_lo"], c["old_hi"])
        new = _spread(c["seqs"], c["new_lo"], c["new_hi"])[::-1]
        lens = [a + b for a, b in zip(old, new)]
        st["pages"], st["table"] = _cache(g, lens, c["page"], c["kv_heads"], c["dim"])
        st["kv_len"] = _ints(lens)
        cu = [0]
        for b in new:
            cu.append(cu[-1] + b)
        st["cu_new"] = _ints(cu)
        st["k"] = randn(cu[-1], c["kv_heads"], c["dim"]).to(t)
        st["v"] = randn(cu[-1], c["kv_heads"], c["dim"]).to(t)
        start = [a // BLOCK * BLOCK for a in old]  # what is read back: from the first block that changes
        cr = [0]
        for a, b in zip(start, lens):
            cr.append(cr[-1] + b - a)
        st["start"], st["cu_read"] = _ints(start), _ints(cr)
        st["max_new"], st["max_read"] = max(new), max(b - a for a, b in zip(start, lens))
        st["k_out"] = torch.empty(cr[-1], c["kv_heads"], c["dim"], dtype=t, device="cuda")
        st["v_out"] = torch.empty(cr[-1], c["kv_heads"], c["dim"], dtype=t, device="cuda")
    elif c["op"] == "norm":
        st["x"] = (randn(c["rows"], c["n"]) * (randn(c["rows"], 1) * 0.5).exp()).to(t)
        st["residual"] = (randn(c["rows"], c["n"]) * 2).to(t) if c["residual"] else None
        st["weight"] = 1 + 0.2 * randn(c["n"])
        st["sum"] = torch.empty(c["rows"], c["n"], dtype=t, device="cuda") if c["residual"] else None
        if c["q8"]:
            st["packed"] = torch.empty(c["rows"] * (c["n"] // 32) * 34, dtype=torch.uint8, device="cuda")
        else:
            st["out"] = torch.empty(c["rows"], c["n"], dtype=t, device="cuda")
    else:
        st["logits"] = (randn(c["rows"], c["n"]) * 2.5).to(t)
        best = st["logits"].float().argmax(1)
        other = torch.randint(0, c["n"], (c["rows"],), device="cuda", generator=g)
        st["tokens"] = torch.where(torch.rand(c["rows"], device="cuda", generator=g) < 0.5, best, other).to(torch.int32)
        st["logprob"] = torch.empty(c["rows"], device="cuda")
        st["entropy"] = torch.empty(c["rows"], device="cuda")
        st["top_index"] = torch.empty(c["rows"], c["k"], dtype=torch.int32, device="cuda")
        st["top_logprob"] = torch.empty(c["rows"], c["k"], device="cuda")
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    op = state["c"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "norm": _own_norm, "logprobs": _own_logprobs}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "norm": _plain_norm, "logprobs": _plain_logprobs}[op](state)


def _own_attend(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    ws = st.get("workspace")
    if ws is None:  # kept by the caller from step to step, zeroed once
        ws = st["workspace"] = qdq.kv_attention_workspace(c["seqs"], c["queries"], c["hi"],
                                                          c["heads"], c["kv_heads"], c["dim"])
    qdq.kv_attention(st["pages"], st["table"], st["kv_len"], st["q"], st["out"], ws, n_heads=c["heads"],
                     n_kv=c["kv_heads"], head_dim=c["dim"], page_tokens=c["page"], max_kv_len=c["hi"],
                     cu_q=st["cu_q"] if c["queries"] > 1 else None, max_q=c["queries"], softcap=c["softcap"],
                     window=c["window"], slopes=st["slopes"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_append(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    qdq.kv_append(st["pages"], st["table"], st["kv_len"], st["k"], st["v"], n_kv=c["kv_heads"], head_dim=c["dim"],
                  page_tokens=c["page"], cu_new=st["cu_new"] if st["max_new"] > 1 else None, max_new=st["max_new"])
    qdq.kv_read(st["pages"], st["table"], st["start"], st["cu_read"], st["k_out"], st["v_out"], n_kv=c["kv_heads"],
                head_dim=c["dim"], page_tokens=c["page"], max_tokens=st["max_read"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_norm(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    if not c["q8"]:
        qdq.rms_norm(st["x"], st["weight"], st["out"], c["rows"], c["n"], 1e-5, residual=st["residual"], sum_out=st["sum"])
        return {"out": st["out"], "sum": st["sum"]}
    qdq.rms_norm(st["x"], st["weight"], None, c["rows"], c["n"], 1e-5, residual=st["residual"], sum_out=st["sum"],
                 q8_out=st["packed"])
    return {"out": _packed_values(st), "sum": st["sum"]}


def _own_logprobs(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    ws = st.get("workspace")
    if ws is None:
        ws = st["workspace"] = qdq.token_logprobs_workspace(c["rows"], c["n"], c["k"])
    qdq.token_logprobs(st["logits"], st["tokens"], st["logprob"], st["entropy"], c["rows"], c["n"], ws, k=c["k"],
                       top_index=st["top_index"], top_logprob=st["top_logprob"])
    return {"logprob": st["logprob"], "entropy": st["entropy"], "top_index": st["top_index"],
            "top_logprob": st["top_logprob"]}


def _packed_values(st):
    """The values of a packed Q8_0 matrix: int8 codes, then one f16 scale for each 32 of them."""
    c = st["c"]
    m = c["rows"] * c["n"]
    codes = st["packed"][:m].view(torch.int8).view(c["rows"], c["n"] // 32, 32)
    return (codes * st["packed"][m:].view(torch.float16).view(c["rows"], c["n"] // 32, 1)).view(c["rows"], c["n"])


# ------------------------------------------------------------------------------ plain forms

def _planes(pages, page, dim):
    """Views of the pool: codes (pages, heads, 2, page, dim) and scales (pages, heads, 2, page / 16)."""
    n, h, rec = pages.shape
    nb = page // BLOCK
    codes = pages.view(torch.int8).as_strided((n, h, 2, page, dim), (h * rec, rec, page * dim, dim, 1))
    scales = pages.view(torch.float32).as_strided((n, h, 2, nb), (h * rec // 4, rec // 4, nb, 1), page * dim // 2)
    return codes, scales


def _plain_attend(st):
    c = st["c"]
    S, n, H, Hk, D, T = c["seqs"], c["queries"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // Hk
    codes, scales = _planes(st["pages"], T, D)
    table = st["table"].long()
    kv = codes[table].float() * scales[table].repeat_interleave(BLOCK, -1).unsqueeze(-1)  # S, P, Hk, 2, T, D
    kv = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, S, Hk, -1, D)
    L = kv.shape[3]
    q = st["q"].float().view(S, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * n, D)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    s = s.view(S, Hk, G, n, L)
    pos = (st["kv_len"].long() - n)[:, None] + torch.arange(n, device="cuda")  # S, n
    far = pos[:, :, None] - torch.arange(L, device="cuda")                     # S, n, L
    if c["bias"]:
        s = s - st["slopes"].view(Hk, G, 1, 1) * far[:, None, None].float()
    seen = far >= 0
    if c["window"]:
        seen = seen & (far < c["window"])
    s = torch.where(seen[:, None, None], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, Hk, G * n, L), kv[1]).view(S, Hk, G, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.log(total) + top).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(S * n, H, D).to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(S * n, H)}


def _plain_append(st):
    c = st["c"]
    D, T = c["dim"], c["page"]
    codes, scales = _planes(st["pages"], T, D)
    table, kv_len, cu = st["table"].long(), st["kv_len"].long(), st["cu_new"].long()
    old = kv_len - (cu[1:] - cu[:-1])
    nb = -(-st["max_new"] // BLOCK) + 1
    first = old // BLOCK * BLOCK
    pos = first[:, None, None] + torch.arange(nb * BLOCK, device="cuda").view(1, nb, BLOCK)  # S, nb, 16
    was = pos < old[:, None, None]
    new = (pos >= old[:, None, None]) & (pos < kv_len[:, None, None])
    used = new.any(-1)                                                            # S, nb
    spare = st["pages"].shape[0] - 1
    page = torch.where(used, table.gather(1, (pos[:, :, 0] // T).clamp(max=table.shape[1] - 1)), torch.full_like(used, spare, dtype=torch.long))
    at = pos[:, :, 0] % T                                                         # first token of the block in its page
    row = (cu[:-1, None, None] + pos - old[:, None, None]).clamp(0, st["k"].shape[0] - 1)
    x = torch.stack([st["k"][row], st["v"][row]], 0).float().permute(1, 2, 4, 0, 3, 5)  # S, nb, heads, 2, 16, D
    new, was = new[:, :, None, None, :, None], was[:, :, None, None, :, None]
    x = torch.where(new, x, torch.zeros_like(x))
    slot = at[:, :, None] + torch.arange(BLOCK, device="cuda")
    there = codes[page[:, :, None], :, :, slot].permute(0, 1, 3, 4, 2, 5).float()  # S, nb, heads, 2, 16, D
    s_old = scales[page, :, :, at // BLOCK]                                       # S, nb, heads, 2
    s_old = torch.where(was.any(-2).squeeze(-1), s_old, torch.zeros_like(s_old))
    s_new = x.abs().amax((-1, -2))
    s_new = s_new / torch.full_like(s_new, 127.0)
    s_new = torch.where(s_new < torch.finfo(torch.float32).tiny, torch.zeros_like(s_new), s_new)
    s = torch.maximum(s_old, s_new)
    one = torch.ones_like(s)
    some = s > 0
    inv = torch.where(some, one / torch.where(some, s, one), torch.zeros_like(s))[..., None, None]
    again = torch.where(some, s_old / torch.where(some, s, one), torch.zeros_like(s))[..., None, None]
    q = torch.where(was, torch.round(there * again), torch.where(new, torch.round(x * inv).clamp(-127, 127), there))
    codes[page[:, :, None], :, :, slot] = q.permute(0, 1, 4, 2, 3, 5).to(torch.int8)
    scales[page, :, :, at // BLOCK] = s
    # what was written, as values
    cr = st["cu_read"].long()
    flat = torch.arange(st["k_out"].shape[0], device="cuda")
    seq = torch.searchsorted(cr[1:], flat, right=True)
    p = st["start"].long()[seq] + flat - cr[seq]
    pg = table[seq, p // T]
    values = codes[pg, :, :, p % T].float() * scales[pg, :, :, p % T // BLOCK].unsqueeze(-1)  # total, heads, 2, D
    values = values.to(st["k"].dtype)
    return {"k": values[:, :, 0], "v": values[:, :, 1]}


def _plain_norm(st):
    c = st["c"]
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5) * st["weight"]
    total = h.to(st["x"].dtype) if st["residual"] is not None else None
    if not c["q8"]:
        return {"out": y.to(st["x"].dtype), "sum": total}
    y = y.view(c["rows"], c["n"] // 32, 32)
    d = y.abs().amax(-1, keepdim=True)
    d = (d / torch.full_like(d, 127.0)).to(torch.float16)
    df = d.float()
    codes = torch.where(df > 0, torch.round(y / torch.where(df > 0, df, torch.ones_like(df))).clamp(-127, 127), torch.zeros_like(y))
    m = c["rows"] * c["n"]
    st["packed"][:m] = codes.to(torch.int8).view(-1).view(torch.uint8)
    st["packed"][m:] = d.reshape(-1).view(torch.uint8)
    return {"out": _packed_values(st), "sum": total}


def _plain_logprobs(st):
    c = st["c"]
    x = st["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total) + top
    mean = (torch.where(e > 0, e * (x - top), torch.zeros_like(e))).sum(1) / total[:, 0]
    logprob = (x.gather(1, st["tokens"].long()[:, None]) - lse)[:, 0]
    best, index = torch.sort(x, dim=1, descending=True, stable=True)
    k = c["k"]
    return {"logprob": logprob, "entropy": torch.log(total[:, 0]) - mean, "top_index": index[:, :k].to(torch.int32),
            "top_logprob": best[:, :k] - lse}


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "norm": _exact_norm, "logprobs": _exact_logprobs}[case["op"]](st)


def _stored(st, seq, pos):
    """The keys and values of a sequence's positions, as code times scale in 64 bits: two (len, heads, dim) tensors."""
    c = st["c"]
    T, D = c["page"], c["dim"]
    rec = st["pages"][st["table"][seq].long()[pos // T]]  # len, heads, record
    out = []
    for which in range(2):
        at = which * T * D + (pos % T)[:, None] * D + torch.arange(D, device="cuda")
        code = rec.gather(2, at[:, None].expand(-1, c["kv_heads"], -1)).view(torch.int8).double()
        at = 2 * T * D + 4 * (which * (T // BLOCK) + pos % T // BLOCK)[:, None] + torch.arange(4, device="cuda")
        scale = rec.gather(2, at[:, None].expand(-1, c["kv_heads"], -1)).contiguous().view(torch.float32).double()
        out.append((code, scale))
    return out


def _exact_attend(st):
    c = st["c"]
    n, H, Hk, D = c["queries"], c["heads"], c["kv_heads"], c["dim"]
    out, lses = [], []
    for i, length in enumerate(_kv_lens(c)):
        (kc, ks), (vc, vs) = _stored(st, i, torch.arange(length, device="cuda"))
        k, v = kc * ks, vc * vs
        q = st["q"][i * n:(i + 1) * n].double()
        where = torch.arange(length, device="cuda")
        at = length - n + torch.arange(n, device="cuda")
        far = at[:, None] - where
        hidden = far < 0
        if c["window"] > 0:
            hidden |= far >= c["window"]
        o, ls = [], []
        for h in range(H):
            s = q[:, h] @ k[:, h * Hk // H].T / math.sqrt(D)
            if c["softcap"] > 0:
                s = torch.tanh(s / c["softcap"]) * c["softcap"]
            if c["bias"]:
                s = s - st["slopes"][h].double() * far
            s = s.masked_fill(hidden, -math.inf)
            ls.append(torch.logsumexp(s, 1))
            o.append(torch.nan_to_num(torch.softmax(s, 1), nan=0.0) @ v[:, h * Hk // H])
        out.append(torch.stack(o, 1))
        lses.append(torch.stack(ls, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lses)}


def _exact_append(st):
    cu, lens = st["cu_new"].tolist(), st["kv_len"].tolist()
    got = [[], []]
    for i, length in enumerate(lens):
        old = length - (cu[i + 1] - cu[i])
        start = old // BLOCK * BLOCK
        pair = _stored(st, i, torch.arange(start, max(old, start), device="cuda")) if old > start else [(None, None)] * 2
        for which, name in enumerate(("k", "v")):
            x = st[name][cu[i]:cu[i + 1]].double()
            pad = -(length - start) % BLOCK
            old_code, old_scale = pair[which]
            full = torch.zeros(length - start + pad, *x.shape[1:], dtype=torch.float64, device="cuda")
            full[old - start:length - start] = x
            b = full.view(-1, BLOCK, *x.shape[1:]).abs().amax((1, 3)) / 127  # blocks, heads
            if old > start:
                b[0] = torch.maximum(b[0], old_scale[0, :, 0])
            s = b.repeat_interleave(BLOCK, 0)[..., None]
            code = torch.where(s > 0, torch.round(full / torch.where(s > 0, s, 1.0)), 0.0)
            if old > start:
                code[:old - start] = torch.round(old_code * old_scale / s[:old - start])
            got[which].append((code * s)[:length - start])
    return {"k": torch.cat(got[0]), "v": torch.cat(got[1])}


def _exact_norm(st):
    c = st["c"]
    h = st["x"].double()
    if c["residual"]:
        h += st["residual"].double()
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["n"] + 1e-5) * st["weight"].double()
    if c["q8"]:
        y = y.view(c["rows"], -1, 32)
        d = (y.abs().amax(2, keepdim=True) / 127).to(torch.float16).double()
        y = (torch.round(y / d).clamp(-127, 127) * d).nan_to_num(nan=0.0).view(c["rows"], c["n"])
    return {"out": y, "sum": h if c["residual"] else None}


def _exact_logprobs(st):
    c = st["c"]
    got = {"logprob": [], "entropy": [], "top_index": [], "top_logprob": []}
    for i in range(0, c["rows"], 64):
        lp = torch.log_softmax(st["logits"][i:i + 64].double(), 1)
        got["logprob"].append(lp[torch.arange(lp.shape[0], device="cuda"), st["tokens"][i:i + 64].long()])
        got["entropy"].append(-torch.special.xlogy(lp.exp(), lp.exp()).sum(1))
        o = torch.argsort(-st["logits"][i:i + 64].double(), dim=1, stable=True)[:, :c["k"]]
        got["top_index"].append(o.to(torch.int32))
        got["top_logprob"].append(lp.gather(1, o))
    return {k: torch.cat(v) for k, v in got.items()}


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    e = SIZE[c["dtype"]]
    if c["op"] == "attend":
        n, w = c["queries"], c["window"]
        tokens = pairs = 0
        for length in _kv_lens(c):
            tokens += min(length, w + n - 1) if w else length
            first = length - n + 1  # the first query's keys
            pairs += sum(min(first + i, w) if w else first + i for i in range(n))
        rows = c["seqs"] * n
        return {"bytes": tokens * c["kv_heads"] * (2 * c["dim"] + 8 / BLOCK) + rows * c["heads"] * (2 * c["dim"] * e + 4),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "append":
        old = _spread(c["seqs"], c["old_lo"], c["old_hi"])
        new = _spread(c["seqs"], c["new_lo"], c["new_hi"])[::-1]
        width = 2 * c["kv_heads"] * c["dim"]
        back = sum(a % BLOCK + b for a, b in zip(old, new))
        # new tokens in, their codes out, the codes read back, the values out
        return {"bytes": width * (sum(new) * (e + 1) + back * (1 + e)), "flops": 4 * width * sum(new)}
    if c["op"] == "norm":
        m = c["rows"] * c["n"]
        out = 34 / 32 + 34 / 32 + 2 if c["q8"] else e  # the packed matrix written and read, its values written
        return {"bytes": m * (e + (2 * e if c["residual"] else 0) + out) + 4 * c["n"], "flops": 5 * m}
    m = c["rows"] * c["n"]
    return {"bytes": m * e + c["rows"] * (12 + 8 * c["k"]), "flops": 5 * m}
