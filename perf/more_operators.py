"""Cases that time the operators of drafted tokens: several tokens of a sequence guessed ahead, run in one
step, verified, and the accepted ones kept.

Four operators, each in a plain form of elementary torch operations and as calls of this repository's library:

* ``rotate``: queries and keys normed for each head and turned by their positions, keys and values
  quantised into the paged 8-bit cache, then read back as the values the cache stands for;
* ``tree``: attention of a sequence's tree of drafted tokens over the cache: a token sees what was cached
  before the tree, its ancestors and itself;
* ``verify``: drafted tokens accepted or rejected by the target's probabilities with given random numbers, and
  the token that follows;
* ``keep``: the cached tokens of an accepted path moved to the places that follow the old ones, read back.

Cache layout: a page holds ``page`` tokens; in it each key/value head has one record of
``align128(2 * page * dim + 8 * page / 16)`` bytes: key codes (page x dim int8), value codes
(page x dim int8), key scales (page / 16 f32), value scales (page / 16 f32).  Value = code * scale.

A tree of n nodes is n int32 parents: a node's parent is an earlier node, or -1.  Node i is the i-th of the
sequence's last n cached tokens; its position is kv_len - n + depth(i).
"""
import math
import random

import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------ cases

def _rotate(seqs, old_lo, old_hi, new_lo, new_hi, heads, kv_heads, dim, page, dtype, turned, pairs="halves", norm=True, tree=False):
    return {"op": "rotate", "seqs": seqs, "old_lo": old_lo, "old_hi": old_hi, "new_lo": new_lo, "new_hi": new_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "turned": turned, "pairs": pairs,
            "norm": norm, "tree": tree}


def _tree(seqs, nodes_lo, nodes_hi, lo, hi, heads, kv_heads, dim, page, dtype, softcap=0.0, window=0, bias=False):
    return {"op": "tree", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "softcap": softcap, "window": window, "bias": bias}


def _verify(seqs, nodes_lo, nodes_hi, n, dtype, drafts, tree, temperature=1.0):
    return {"op": "verify", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "n": n, "dtype": dtype,
            "drafts": drafts, "tree": tree, "temperature": temperature}


def _keep(seqs, nodes_lo, nodes_hi, old_lo, old_hi, kv_heads, dim, page):
    return {"op": "keep", "seqs": seqs, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "old_lo": old_lo, "old_hi": old_hi,
            "kv_heads": kv_heads, "dim": dim, "page": page}


def listed():
    return [
        # one user's decode step: one token's queries and keys
        {"name": "rotate one token"} | _rotate(1, 776, 776, 1, 1, 24, 8, 128, 64, "f32", 128),
        # a serving batch whose sequences each bring a small tree of drafts; half of each head turned
        {"name": "rotate drafts"} | _rotate(48, 1, 8100, 5, 26, 32, 8, 128, 64, "bf16", 64, "adjacent", True, True),
        # a prompt batch
        {"name": "rotate prompts"} | _rotate(6, 0, 500, 900, 3001, 24, 8, 128, 64, "bf16", 128),
        # one user's tree of drafts early in a conversation
        {"name": "tree one"} | _tree(1, 13, 13, 777, 777, 24, 8, 128, 64, "f32"),
        # a serving batch, trees and sequences of every size
        {"name": "tree batch"} | _tree(16, 7, 64, 300, 8191, 24, 8, 128, 64, "bf16"),
        # a long document with a tree of drafts
        {"name": "tree long"} | _tree(1, 26, 26, 131071, 131071, 32, 8, 128, 128, "bf16"),
        # small heads, capped scores, a distance bias and a window
        {"name": "tree window"} | _tree(9, 3, 31, 200, 6001, 16, 2, 64, 32, "f16", 30.0, 1500, True),
        # one user's chain of drafts with their probabilities
        {"name": "verify one chain"} | _verify(1, 6, 6, 128256, "f32", "probabilities", False),
        # a serving batch's chains
        {"name": "verify chains"} | _verify(48, 2, 8, 128256, "bf16", "probabilities", False, 0.8),
        # trees of the likeliest tokens of a draft, which has no probabilities to give
        {"name": "verify trees"} | _verify(16, 9, 40, 128256, "f32", "given", True),
        # one user's accepted path
        {"name": "keep one path"} | _keep(1, 13, 13, 777, 777, 8, 128, 64),
        # a serving batch's accepted paths
        {"name": "keep paths"} | _keep(48, 5, 60, 1, 8100, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "tree", "tree", "verify", "verify", "keep"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotate":
        if rng.random() < 0.6:
            seqs, new_lo, new_hi = _log(rng, 1, 128), 1, rng.choice([1, 1, rng.randint(2, 64)])
        else:
            seqs, new_lo, new_hi = rng.randint(1, 6), 1, _log(rng, 65, 1500)
        seqs = max(1, min(seqs, (40 << 20) // (new_hi * (heads + 2 * kv_heads) * dim)))
        return _rotate(seqs, 0, _log(rng, 1, 2000), new_lo, new_hi, heads, kv_heads, dim, page, dtype,
                       rng.choice([dim, dim, dim // 2, 32]), rng.choice(["halves", "adjacent"]), rng.random() < 0.6,
                       1 < new_hi <= 64 and rng.random() < 0.7)
    if op == "tree":
        nodes = rng.randint(2, 64)
        seqs = _log(rng, 1, 32)
        hi = _log(rng, nodes + 1, max(nodes + 2, min(100000, (32 << 20) // (seqs * kv_heads * dim),
                                                     (12 << 30) // (seqs * nodes * heads * dim))))
        return _tree(seqs, rng.choice([1, nodes]), nodes, nodes if seqs > 1 else hi, hi, heads, kv_heads, dim, page, dtype,
                     rng.choice([0.0, 0.0, 30.0, 50.0]), rng.choice([0, 0, _log(rng, 5, 4096)]), rng.random() < 0.3)
    if op == "verify":
        n = _log(rng, 1000, 160000)
        nodes = rng.choice([1, rng.randint(2, 8), rng.randint(9, 64)])
        seqs = _log(rng, 1, max(1, min(128, (40 << 20) // (n * nodes))))
        return _verify(seqs, rng.choice([1, nodes]), nodes, n, dtype, rng.choice(["probabilities", "probabilities", "given"]),
                       rng.random() < 0.5, rng.choice([1.0, 1.0, 0.7, 1.3, 0.0]))
    nodes = rng.randint(2, 64)
    return _keep(_log(rng, 1, 128), rng.choice([1, nodes]), nodes, 0, _log(rng, 1, 3000), kv_heads, dim, page)


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], spread evenly and out of order, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _news(c):
    """New tokens (nodes) of each sequence."""
    if c["op"] == "rotate":
        return _spread(c["seqs"], c["new_lo"], c["new_hi"])[::-1]
    return _spread(c["seqs"], c["nodes_lo"], c["nodes_hi"])[::-1]


def _lens(c):
    """Cached tokens of each sequence, the new ones included."""
    if c["op"] == "tree":
        return [max(a, b) for a, b in zip(_spread(c["seqs"], c["lo"], c["hi"]), _news(c))]
    return [a + b for a, b in zip(_spread(c["seqs"], c["old_lo"], c["old_hi"]), _news(c))]


def _more(c):
    """Nodes of each sequence that are kept besides the root: up to 8."""
    return [min(n - 1, m) for n, m in zip(_news(c), _spread(c["seqs"], 0, 8))]


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


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


def _parents(rng, n, tree):
    """Parents of n nodes: a chain, or a tree that goes on from its last node more often than it branches."""
    return [i - 1 if i == 0 or not tree or rng.random() < 0.4 else rng.randrange(i) for i in range(n)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed + 1) + 17)
    rng = random.Random(seed)
    st = {"c": c}
    news = _news(c)
    cu = _starts(news)
    st["cu"], st["most"] = _ints(cu), max(news)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if c["op"] == "verify":
        return _prepare_verify(st, g, rng, news)
    lens = _lens(c)
    st["pages"], st["table"] = _cache(g, lens, c["page"], c["kv_heads"], c["dim"])
    st["kv_len"] = _ints(lens)
    D = c["dim"]
    if c["op"] == "tree":
        t = DTYPES[c["dtype"]]
        st["parent"] = _ints([p for n in news for p in _parents(rng, n, True)])
        st["q"] = (randn(cu[-1], c["heads"], D) * 1.5).to(t)
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["heads"]) for h in range(c["heads"])],
                                    device="cuda") if c["bias"] else None
        st["out"] = torch.empty(cu[-1], c["heads"], D, dtype=t, device="cuda")
        st["lse"] = torch.empty(cu[-1], c["heads"], device="cuda")
        return st
    old = [a - b for a, b in zip(lens, news)]
    if c["op"] == "rotate":
        t = DTYPES[c["dtype"]]
        st["q"] = (randn(cu[-1], c["heads"], D) * 1.5).to(t)
        st["k"] = (randn(cu[-1], c["kv_heads"], D) * 1.5).to(t)
        st["v"] = randn(cu[-1], c["kv_heads"], D).to(t)
        st["q_weight"] = 1 + 0.2 * randn(D) if c["norm"] else None
        st["k_weight"] = 1 + 0.2 * randn(D) if c["norm"] else None
        i = torch.arange(c["turned"] // 2, device="cuda", dtype=torch.float64)
        st["freqs"] = (500000.0 ** (-2 * i / c["turned"])).float()
        st["parent"] = _ints([p for n in news for p in _parents(rng, n, True)]) if c["tree"] else None
        st["q_out"] = torch.empty(cu[-1], c["heads"], D, dtype=t, device="cuda")
        after = lens
    else:
        paths = []
        for n, more in zip(news, _more(c)):  # the root and some later nodes
            kept = sorted(rng.sample(range(1, n), more))
            paths.append([0] + kept)
        st["accepted"] = _ints([len(p) - 1 for p in paths])
        st["path"] = _ints([p + [-1] * (st["most"] - len(p)) for p in paths])
        after = [a + len(p) for a, p in zip(old, paths)]
    start = [a // BLOCK * BLOCK for a in old]  # what is read back: from the first block that changes
    cr = _starts([b - a for a, b in zip(start, after)])
    st["start"], st["cu_read"], st["max_read"] = _ints(start), _ints(cr), max(b - a for a, b in zip(start, after))
    back = torch.float32 if c["op"] == "keep" else torch.bfloat16
    st["k_out"] = torch.empty(cr[-1], c["kv_heads"], D, dtype=back, device="cuda")
    st["v_out"] = torch.empty(cr[-1], c["kv_heads"], D, dtype=back, device="cuda")
    return st


def _prepare_verify(st, g, rng, news):
    c = st["c"]
    rows, V = sum(news), c["n"]
    logits = torch.randn(rows, V, device="cuda", generator=g) * 2.5
    few = torch.randint(0, V, (rows, 16), device="cuda", generator=g)  # a few tokens have most of the probability
    logits.scatter_(1, few, math.log(V) + 3 + 2 * torch.randn(rows, 16, device="cuda", generator=g))
    drafted = logits + torch.randn(rows, V, device="cuda", generator=g) * 0.8
    st["logits"] = logits.to(DTYPES[c["dtype"]])
    del logits
    parents = [_parents(rng, n, c["tree"]) for n in news]
    up, rank = [], []  # the row of a node's parent, and how many of that one's children come before the node
    for at, p in zip(_starts(news), parents):
        up += [at + max(x, 0) for x in p]
        rank += [sum(y == x for y in p[1:i]) if i else 0 for i, x in enumerate(p)]
    up, rank = torch.tensor(up, device="cuda"), torch.tensor(rank, device="cuda")
    st["parent"] = _ints([x for p in parents for x in p]) if c["tree"] else None
    st["draft_probs"] = None
    if c["drafts"] == "probabilities":
        probs = torch.softmax(drafted / (c["temperature"] or 1.0), 1)
        st["tokens"] = torch.cat([torch.multinomial(probs[u], 1, generator=g)[:, 0] for u in up.split(64)]).to(torch.int32)
        st["draft_probs"] = probs
    else:
        best = torch.topk(drafted, min(V, 64), dim=1).indices
        st["tokens"] = best[up, rank].to(torch.int32)
    st["uniform"] = torch.rand(rows, device="cuda", generator=g)
    st["accepted"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    st["path"] = torch.empty(c["seqs"], st["most"], dtype=torch.int32, device="cuda")
    st["next"] = torch.empty(c["seqs"], dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------------------ one pass

def run(state):
    op = state["c"]["op"]
    if own:
        return {"rotate": _own_rotate, "tree": _own_tree, "verify": _own_verify, "keep": _own_keep}[op](state)
    return {"rotate": _plain_rotate, "tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}[op](state)


def _own_rotate(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    qdq.kv_append_rope(st["pages"], st["table"], st["kv_len"], st["q"], st["q_out"], st["k"], st["v"], n_heads=c["heads"],
                       n_kv=c["kv_heads"], head_dim=c["dim"], page_tokens=c["page"], freqs=st["freqs"],
                       interleaved=c["pairs"] == "adjacent", q_weight=st["q_weight"], k_weight=st["k_weight"], eps=EPS,
                       cu_new=st["cu"] if st["most"] > 1 else None, max_new=st["most"], parent=st["parent"])
    return {"q": st["q_out"], **_own_read(st)}


def _own_read(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    qdq.kv_read(st["pages"], st["table"], st["start"], st["cu_read"], st["k_out"], st["v_out"], n_kv=c["kv_heads"],
                head_dim=c["dim"], page_tokens=c["page"], max_tokens=st["max_read"])
    return {"k": st["k_out"], "v": st["v_out"]}


def _own_tree(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    ws = st.get("workspace")
    if ws is None:  # kept by the caller from step to step, zeroed once
        ws = st["workspace"] = qdq.kv_attention_workspace(c["seqs"], st["most"], c["hi"], c["heads"], c["kv_heads"], c["dim"])
    qdq.kv_tree_attention(st["pages"], st["table"], st["kv_len"], st["q"], st["out"], ws, n_heads=c["heads"],
                          n_kv=c["kv_heads"], head_dim=c["dim"], page_tokens=c["page"], max_kv_len=c["hi"], cu_q=st["cu"],
                          max_q=st["most"], parent=st["parent"], softcap=c["softcap"], window=c["window"],
                          slopes=st["slopes"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _own_verify(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    ws = st.get("workspace")
    if ws is None:
        ws = st["workspace"] = qdq.verify_drafts_workspace(c["seqs"], st["most"], c["n"])
    qdq.verify_drafts(st["logits"], st["tokens"], st["uniform"], st["accepted"], st["path"], st["next"], n=c["n"], workspace=ws,
                      cu=st["cu"], max_rows=st["most"], parent=st["parent"], draft_probs=st["draft_probs"],
                      temperature=c["temperature"])
    return {"accepted": st["accepted"], "path": st["path"], "next": st["next"]}


def _own_keep(st):
    import ggml_quantized_dequant_gb300 as qdq
    c = st["c"]
    qdq.kv_keep(st["pages"], st["table"], st["kv_len"], st["cu"], st["path"], st["accepted"], n_kv=c["kv_heads"],
                head_dim=c["dim"], page_tokens=c["page"])
    return _own_read(st)


# ------------------------------------------------------------------------------ plain forms

def _planes(pages, page, dim):
    """Views of the pool: codes (pages, heads, 2, page, dim) and scales (pages, heads, 2, page / 16)."""
    n, h, rec = pages.shape
    nb = page // BLOCK
    codes = pages.view(torch.int8).as_strided((n, h, 2, page, dim), (h * rec, rec, page * dim, dim, 1))
    scales = pages.view(torch.float32).as_strided((n, h, 2, nb), (h * rec // 4, rec // 4, nb, 1), page * dim // 2)
    return codes, scales


def _padded(st, values, fill):
    """Row values as (sequences, most), ``fill`` past a sequence's rows."""
    cu = st["cu"].long()
    i = torch.arange(st["most"], device="cuda")
    at = cu[:-1, None] + i
    return torch.where(i < (cu[1:] - cu[:-1])[:, None], values[at.clamp(max=values.shape[0] - 1)], fill)


def _ancestors(st):
    """(sequences, most, most): whether node j is node i or one of its ancestors."""
    p = _padded(st, st["parent"].long(), -1)
    step = (p[:, :, None] == torch.arange(st["most"], device="cuda")).double()
    step = step + torch.eye(st["most"], device="cuda", dtype=torch.float64)
    return torch.matrix_power(step, 64) > 0  # a node is at most 63 steps from its root


def _read_back(st):
    c = st["c"]
    codes, scales = _planes(st["pages"], c["page"], c["dim"])
    cr = st["cu_read"].long()
    flat = torch.arange(st["k_out"].shape[0], device="cuda")
    seq = torch.searchsorted(cr[1:], flat, right=True)
    p = st["start"].long()[seq] + flat - cr[seq]
    pg = st["table"].long()[seq, p // c["page"]]
    values = codes[pg, :, :, p % c["page"]].float() * scales[pg, :, :, p % c["page"] // BLOCK].unsqueeze(-1)
    values = values.to(st["k_out"].dtype)
    return {"k": values[:, :, 0], "v": values[:, :, 1]}


def _normed_and_turned(c, x, weight, cos, sin):
    """x (rows, heads, dim) in f32; cos and sin (rows, 1, turned / 2)."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    r = c["turned"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["pairs"] == "adjacent" else (x[..., : r // 2], x[..., r // 2: r])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if c["pairs"] == "adjacent" else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rotate(st):
    c = st["c"]
    cu, kv_len = st["cu"].long(), st["kv_len"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(st["most"], device="cuda")
    depth = _ancestors(st).sum(-1) - 1 if c["tree"] else i.expand(c["seqs"], -1)
    pos = ((kv_len - new)[:, None] + depth)[i < new[:, None]]  # of each row
    angle = (pos.double()[:, None] * st["freqs"].double())[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _normed_and_turned(c, st["q"].float(), st["q_weight"], cos, sin)
    k = _normed_and_turned(c, st["k"].float(), st["k_weight"], cos, sin)
    _plain_append(st, k, st["v"].float())
    return {"q": q.to(st["q"].dtype), **_read_back(st)}


def _plain_append(st, k, v):
    c = st["c"]
    D, T = c["dim"], c["page"]
    codes, scales = _planes(st["pages"], T, D)
    table, kv_len, cu = st["table"].long(), st["kv_len"].long(), st["cu"].long()
    old = kv_len - (cu[1:] - cu[:-1])
    nb = -(-st["most"] // BLOCK) + 1
    first = old // BLOCK * BLOCK
    pos = first[:, None, None] + torch.arange(nb * BLOCK, device="cuda").view(1, nb, BLOCK)  # S, nb, 16
    was = pos < old[:, None, None]
    new = (pos >= old[:, None, None]) & (pos < kv_len[:, None, None])
    used = new.any(-1)                                                            # S, nb
    spare = st["pages"].shape[0] - 1
    page = torch.where(used, table.gather(1, (pos[:, :, 0] // T).clamp(max=table.shape[1] - 1)),
                       torch.full_like(used, spare, dtype=torch.long))
    at = pos[:, :, 0] % T                                                         # first token of the block in its page
    row = (cu[:-1, None, None] + pos - old[:, None, None]).clamp(0, k.shape[0] - 1)
    x = torch.stack([k[row], v[row]], 0).permute(1, 2, 4, 0, 3, 5)                # S, nb, heads, 2, 16, D
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


def _plain_tree(st):
    c = st["c"]
    S, n, H, Hk, D, T = c["seqs"], st["most"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    G = H // Hk
    codes, scales = _planes(st["pages"], T, D)
    table, kv_len, cu = st["table"].long(), st["kv_len"].long(), st["cu"].long()
    kv = codes[table].float() * scales[table].repeat_interleave(BLOCK, -1).unsqueeze(-1)  # S, P, Hk, 2, T, D
    kv = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, S, Hk, -1, D)
    L = kv.shape[3]
    i = torch.arange(n, device="cuda")
    mine = i < (cu[1:] - cu[:-1])[:, None]                                       # S, n
    row = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][row].float().view(S, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * n, D)
    s = torch.matmul(q, kv[0].transpose(-1, -2)) * (1.0 / math.sqrt(D))
    if c["softcap"]:
        s = c["softcap"] * torch.tanh(s / c["softcap"])
    s = s.view(S, Hk, G, n, L)
    base = (kv_len - (cu[1:] - cu[:-1]))[:, None]                                # S, 1
    up = _ancestors(st)
    depth = up.sum(-1) - 1                                                       # S, n
    j = torch.arange(L, device="cuda").expand(S, L)
    node = (j - base).clamp(0, n - 1)
    drafted = (j >= base) & (j < kv_len[:, None])
    pos_j = torch.where(drafted, base + depth.gather(1, node), j)
    seen = (j < base)[:, None] | (drafted[:, None] & up.gather(2, node[:, None].expand(-1, n, -1)))
    far = (base + depth)[:, :, None] - pos_j[:, None]                            # S, n, L
    if c["window"]:
        seen = seen & (far < c["window"])
    if c["bias"]:
        s = s - st["slopes"].view(Hk, G, 1, 1) * far[:, None, None].float()
    s = torch.where(seen[:, None, None], s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)  # a node sees itself
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, Hk, G * n, L), kv[1]).view(S, Hk, G, n, D) / total
    lse = (torch.log(total) + top).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(S, n, H, D)[mine].to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(S, n, H)[mine]}


def _plain_verify(st):
    """In 64 bits: a draw lies next to the border of two tokens as often as sums are off."""
    c = st["c"]
    S, n, V = c["seqs"], st["most"], c["n"]
    cu = st["cu"].long()
    i = torch.arange(n, device="cuda")
    row = (cu[:-1, None] + i).clamp(max=st["tokens"].shape[0] - 1)
    parent = _padded(st, st["parent"].long(), -1) if c["tree"] else (i - 1).expand(S, n)
    there = i < (cu[1:] - cu[:-1])[:, None]
    token, u = st["tokens"].long()[row], st["uniform"].double()[row]
    every = torch.arange(S, device="cuda")

    def target(r):  # the target's probabilities after the tokens of these rows
        x = st["logits"][r].double()
        if c["temperature"] == 0:  # all on the largest, the first of equals
            best = torch.where(x == x.amax(1, keepdim=True), torch.arange(V, device="cuda"), V).amin(1)
            return torch.zeros_like(x).scatter_(1, best[:, None], 1.0)
        x = x / c["temperature"]
        e = torch.exp(x - x.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)

    at = torch.zeros_like(every)
    path = torch.full((S, n), -1, device="cuda")
    path[:, 0] = 0
    count = torch.zeros_like(every)
    w = target(row[:, 0])  # what is left of the probabilities at each sequence's present node
    for k in range(1, n):
        asked = there[:, k] & (parent[:, k] == at)
        x = token[:, k]
        if c["drafts"] == "given":
            q = torch.zeros_like(w).scatter_(1, x[:, None], 1.0)
        else:
            q = st["draft_probs"][row[every, at]].double()
        px, qx = w[every, x], q[every, x]
        if c["temperature"] == 0:
            yes = asked & (px > 0)
            rest = w
        else:
            yes = asked & (u[:, k] * qx < px)
            rest = w * (1 - q) if c["drafts"] == "given" else (w - q).clamp(min=0)
            left = rest.sum(1, keepdim=True)
            rest = torch.where(left > 0, rest / torch.where(left > 0, left, 1.0), w)
        w = torch.where(yes[:, None], target(row[:, k]), torch.where(asked[:, None], rest, w))
        count = count + yes
        path[every, torch.where(yes, count, 0)] = torch.where(yes, k, 0)
        at = torch.where(yes, k, at)
    run_up = torch.cumsum(w, 1)
    last = torch.where(w > 0, torch.arange(V, device="cuda"), 0).amax(1)
    found = (run_up <= u[:, :1] * run_up[:, -1:]).sum(1)
    return {"accepted": count.to(torch.int32), "path": path.to(torch.int32), "next": torch.minimum(found, last).to(torch.int32)}


def _plain_keep(st):
    c = st["c"]
    T, D = c["page"], c["dim"]
    codes, scales = _planes(st["pages"], T, D)
    table, cu = st["table"].long(), st["cu"].long()
    old = st["kv_len"].long() - (cu[1:] - cu[:-1])
    end = old + st["accepted"].long() + 1
    nb = -(-st["path"].shape[1] // BLOCK) + 1
    to = (old // BLOCK * BLOCK)[:, None, None] + torch.arange(nb * BLOCK, device="cuda").view(1, nb, BLOCK)  # S, nb, 16
    kept = to < end[:, None, None]
    moved = kept & (to >= old[:, None, None])
    step = (to - old[:, None, None]).clamp(0, st["path"].shape[1] - 1).flatten(1)
    src = torch.where(moved, old[:, None, None] + st["path"].long().gather(1, step).view_as(to), to)
    used = kept.any(-1)
    spare = st["pages"].shape[0] - 1
    width = table.shape[1] - 1

    def place(p):
        return table.gather(1, (p // T).clamp(max=width).flatten(1)).view_as(p)

    src = torch.where(kept, src, 0)
    pg = place(src)
    code = codes[pg, :, :, src % T]                    # S, nb, 16, heads, 2, D
    s_src = scales[pg, :, :, src % T // BLOCK]         # S, nb, 16, heads, 2
    s_src = torch.where(kept[..., None, None], s_src, torch.zeros_like(s_src))
    s = s_src.amax(2)
    ratio = torch.where(s[:, :, None] > 0, s_src / torch.where(s[:, :, None] > 0, s[:, :, None], torch.ones_like(s_src)), 0.0)
    code = torch.round(code.float() * ratio.unsqueeze(-1)).to(torch.int8)
    to_page = torch.where(used, place(to[:, :, 0]), spare)
    slot = to % T
    there = codes[to_page[:, :, None], :, :, slot]
    codes[to_page[:, :, None], :, :, slot] = torch.where(kept[..., None, None, None], code, there)
    scales[to_page, :, :, to[:, :, 0] % T // BLOCK] = s
    return _read_back(st)


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"rotate": _exact_rotate, "tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](st)


def _stored(st, seq, pos):
    """The keys and values of a sequence's positions in 64 bits: two (codes, scales) of (len, heads, dim) and (len, heads, 1)."""
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


def _lines(parents):
    """Each node's way down from its root, itself at the end."""
    lines = []
    for i, p in enumerate(parents):
        lines.append((lines[p] if p >= 0 else []) + [i])
    return lines


def _rows_of(st):
    cu = st["cu"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _exact_rotate(st):
    c = st["c"]
    lens = st["kv_len"].tolist()
    qs, got = [], [[], []]
    r = c["turned"]

    def turn(x, weight, pos):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + EPS) * weight.double()
        z = torch.polar(torch.ones(len(pos), r // 2, dtype=torch.float64, device="cuda"),
                        torch.outer(pos.double(), st["freqs"].double()))[:, None]
        if c["pairs"] == "adjacent":
            y = torch.view_as_real(torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous()) * z).flatten(-2)
        else:
            y = torch.complex(x[..., : r // 2], x[..., r // 2: r]) * z
            y = torch.cat([y.real, y.imag], -1)
        return torch.cat([y, x[..., r:]], -1)

    for s, (a, b) in enumerate(_rows_of(st)):
        old = lens[s] - (b - a)
        depth = [len(x) - 1 for x in _lines(st["parent"][a:b].tolist())] if c["tree"] else list(range(b - a))
        pos = old + torch.tensor(depth, device="cuda")
        qs.append(turn(st["q"][a:b], st["q_weight"], pos))
        fresh = [turn(st["k"][a:b], st["k_weight"], pos), st["v"][a:b].double()]
        start = old // BLOCK * BLOCK
        pair = _stored(st, s, torch.arange(start, old, device="cuda")) if old > start else None
        for which, x in enumerate(fresh):
            pad = -(lens[s] - start) % BLOCK
            full = torch.zeros(lens[s] - start + pad, *x.shape[1:], dtype=torch.float64, device="cuda")
            full[old - start:lens[s] - start] = x
            top = full.view(-1, BLOCK, *x.shape[1:]).abs().amax((1, 3)) / 127
            if pair:
                top[0] = torch.maximum(top[0], pair[which][1][0, :, 0])
            step = top.repeat_interleave(BLOCK, 0)[..., None]
            code = torch.where(step > 0, torch.round(full / torch.where(step > 0, step, 1.0)), 0.0)
            if pair:
                code[:old - start] = torch.round(pair[which][0] * pair[which][1] / step[:old - start])
            got[which].append((code * step)[:lens[s] - start])
    return {"q": torch.cat(qs), "k": torch.cat(got[0]), "v": torch.cat(got[1])}


def _exact_tree(st):
    c = st["c"]
    H, Hk, D = c["heads"], c["kv_heads"], c["dim"]
    out, lses = [], []
    for s, (a, b) in enumerate(_rows_of(st)):
        length = int(st["kv_len"][s])
        base = length - (b - a)
        (kc, ks), (vc, vs) = _stored(st, s, torch.arange(length, device="cuda"))
        k, v = kc * ks, vc * vs
        q = st["q"][a:b].double()
        lines = _lines(st["parent"][a:b].tolist())
        where = torch.arange(length, dtype=torch.float64, device="cuda")
        hidden = torch.ones(b - a, length, dtype=torch.bool, device="cuda")
        hidden[:, :base] = False
        for i, line in enumerate(lines):
            hidden[i, [base + x for x in line]] = False
            where[base + i] = base + len(line) - 1
        far = where[base:, None] - where
        if c["window"] > 0:
            hidden |= far >= c["window"]
        o, ls = [], []
        for h in range(H):
            x = q[:, h] @ k[:, h * Hk // H].T / math.sqrt(D)
            if c["softcap"] > 0:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if c["bias"]:
                x = x - st["slopes"][h].double() * far
            x = x.masked_fill(hidden, -math.inf)
            ls.append(torch.logsumexp(x, 1))
            o.append(torch.softmax(x, 1) @ v[:, h * Hk // H])
        out.append(torch.stack(o, 1))
        lses.append(torch.stack(ls, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lses)}


def _exact_verify(st):
    c = st["c"]
    n = st["most"]
    accepted, paths, nexts = [], [], []
    for a, b in _rows_of(st):
        parents = st["parent"][a:b].tolist() if c["tree"] else list(range(-1, b - a - 1))
        tokens, u = st["tokens"][a:b].tolist(), st["uniform"][a:b].double().tolist()
        path, present = [0], 0
        while True:
            x = st["logits"][a + present].double()
            if c["temperature"] == 0:
                best = int((x == x.max()).nonzero()[0])
                taken = [i for i in range(1, b - a) if parents[i] == present and tokens[i] == best]
                if not taken:
                    nexts.append(best)
                    break
                present = taken[0]
                path.append(present)
                continue
            p = torch.softmax(x / c["temperature"], 0)
            went = None
            for i in range(1, b - a):
                if parents[i] != present:
                    continue
                if c["drafts"] == "given":
                    q = torch.zeros_like(p)
                    q[tokens[i]] = 1
                else:
                    q = st["draft_probs"][a + present].double()
                if u[i] * float(q[tokens[i]]) < float(p[tokens[i]]):
                    went = i
                    break
                rest = torch.relu(p - q) if c["drafts"] != "given" else p.masked_fill(q > 0, 0.0)
                if float(rest.sum()) > 0:
                    p = rest / rest.sum()
            if went is None:
                border = torch.cumsum(p, 0)
                at = int(torch.searchsorted(border, border[-1:] * u[0], right=True))
                nexts.append(min(at, int(p.nonzero()[-1])))
                break
            present = went
            path.append(went)
        accepted.append(len(path) - 1)
        paths.append(path + [-1] * (n - len(path)))
    return {"accepted": _ints(accepted), "path": _ints(paths), "next": _ints(nexts)}


def _exact_keep(st):
    got = [[], []]
    lens = st["kv_len"].tolist()
    for s, (a, b) in enumerate(_rows_of(st)):
        old = lens[s] - (b - a)
        start = old // BLOCK * BLOCK
        line = st["path"][s].tolist()[: int(st["accepted"][s]) + 1]
        src = list(range(start, old)) + [old + x for x in line]
        pair = _stored(st, s, torch.tensor(src, device="cuda"))
        for which, (code, scale) in enumerate(pair):
            parts = []
            for x, y in zip(code.split(BLOCK), scale.split(BLOCK)):
                top = y.amax(0, keepdim=True)
                parts.append(torch.round(x * (y / top)) * top)
            got[which].append(torch.cat(parts))
    return {"k": torch.cat(got[0]), "v": torch.cat(got[1])}


# ------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    news = _news(c)
    if c["op"] == "verify":
        # a row of logits for each accepted draft and one more; at these distributions about half of the drafts on a
        # line are accepted.  One row of draft probabilities where a draft is rejected.
        seen = sum(min(n, 2) for n in news)
        rejected = sum(n > 1 for n in news) if c["drafts"] == "probabilities" and c["temperature"] else 0
        return {"bytes": c["n"] * (seen * SIZE[c["dtype"]] + 4 * rejected) + 16 * sum(news), "flops": c["n"] * (4 * seen + 4 * rejected)}
    lens = _lens(c)
    width = 2 * c["kv_heads"] * c["dim"]
    if c["op"] == "tree":
        e = SIZE[c["dtype"]]
        w = c["window"]
        tokens = sum(min(a, w + n) if w else a for a, n in zip(lens, news))
        pairs = sum(n * (min(a, w) if w else a) for a, n in zip(lens, news))
        rows = sum(news)
        return {"bytes": tokens * c["kv_heads"] * (2 * c["dim"] + 8 / BLOCK) + rows * (c["heads"] * (2 * c["dim"] * e + 4) + 4),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    old = [a - b for a, b in zip(lens, news)]
    if c["op"] == "rotate":
        e = SIZE[c["dtype"]]
        back = sum(a % BLOCK + b for a, b in zip(old, news))
        # queries in and out, new keys and values in, their codes out, the codes read back, the values out
        return {"bytes": sum(news) * (2 * e * c["heads"] * c["dim"] + width * (e + 1)) + width * back * (1 + 2),
                "flops": sum(news) * 10 * (c["heads"] + c["kv_heads"]) * c["dim"]}
    kept = sum(1 + m for m in _more(c))
    back = kept + sum(a % BLOCK for a in old)
    return {"bytes": width * (2 * kept + back * (1 + 4)), "flops": width * kept}
