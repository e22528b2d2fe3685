"""A decoder on one GPU: prompts scored in one batch, then tokens one by one from a CUDA graph.

Every operation on the device is an entry point of the library (tensors, copies and graphs come from
torch).  Per layer, with h the residual stream:

    n = norm(h);  q, k, v = Wq n, Wk n, Wv n;  k, v -> paged 8-bit cache;  o = Wo attention(q, cache)
    h = h + o;    n = norm(h);                 h = h + Wd (silu(Wg n) * Wu n)

and at the end the Q8_0 output projection of norm(h) and its log probabilities.  Positions enter as the
attention's distance bias.  Prompts of different lengths lie behind one another in one batch of rows
(tensor-core GEMMs and prompt attention); a step of single tokens runs the GEMVs.  Weights are random.

    python -m examples.decode --layers 4 --prompts 700 64 1 300 --new 32
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import numpy as np
import torch

import ggml_quantized_dequant_gb300 as qdq
import synth


@dataclass
class Sizes:
    n_embd: int = synth.N_EMBD
    n_ff: int = synth.N_FF
    n_heads: int = 24
    n_kv: int = 8
    head_dim: int = 128
    n_vocab: int = synth.N_VOCAB
    n_layers: int = 4
    page_tokens: int = 64
    eps: float = 1e-5

    @property
    def n_q(self):
        return self.n_heads * self.head_dim

    @property
    def n_k(self):
        return self.n_kv * self.head_dim


def random_weights(z: Sizes, seed: int = 0):
    """Packed weights on the device: (embedding, layers, output norm, output projection)."""
    rng = np.random.default_rng(seed)

    def q4k(n_out, n_in):
        d = 1 / (257 * n_in ** 0.5)  # sc q - 7.5 m of uniform bytes has mean 0 and deviation 257
        return qdq.upload_q4k(synth.q4k_blocks(rng, n_out, n_in, (0.9 * d, 1.1 * d), (6.75 * d, 8.25 * d)), n_out, n_in)

    def gain():
        return torch.from_numpy(rng.uniform(0.5, 1.5, z.n_embd).astype(np.float32)).cuda()

    embed = qdq.upload_q6k(synth.q6k_blocks(rng, z.n_vocab, z.n_embd, (2e-4, 1e-3)), z.n_vocab, z.n_embd)
    layers = [dict(n1=gain(), q=q4k(z.n_q, z.n_embd), k=q4k(z.n_k, z.n_embd), v=q4k(z.n_k, z.n_embd),
                   o=q4k(z.n_embd, z.n_q), n2=gain(), g=q4k(z.n_ff, z.n_embd), u=q4k(z.n_ff, z.n_embd),
                   d=q4k(z.n_embd, z.n_ff)) for _ in range(z.n_layers)]
    d = 1 / (73 * z.n_embd ** 0.5)
    head = qdq.upload_q8_0(synth.q8_0_blocks(rng, z.n_vocab, z.n_embd, (d, 3 * d)), z.n_vocab, z.n_embd)
    return embed, layers, gain(), head


class Decoder:
    """Up to 8 sequences of at most ``max_len`` tokens."""

    def __init__(self, z: Sizes, weights, n_seqs: int, max_len: int, top: int = 5, seed: int = 0):
        if not 1 <= n_seqs <= 8:
            raise ValueError("1 to 8 sequences")
        self.z, self.n_seqs, self.max_len, self.top = z, n_seqs, max_len, top
        self.embed, self.layers, self.gain, self.head = weights
        per_seq = -(-max_len // z.page_tokens)
        self.caches = [qdq.kv_pages(n_seqs * per_seq, z.page_tokens, z.n_kv, z.head_dim) for _ in self.layers]
        order = np.random.default_rng(seed).permutation(n_seqs * per_seq)  # pages lie anywhere
        self.table = torch.from_numpy(order.reshape(n_seqs, per_seq).astype(np.int32)).cuda()
        self.kv_len = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / z.n_heads) for i in range(z.n_heads)], device="cuda")
        # a step's buffers, at fixed addresses for the graph
        f = lambda *shape: torch.zeros(shape, dtype=torch.float32, device="cuda")
        i = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")
        b = n_seqs
        self.ids, self.h, self.n = i(b), f(b, z.n_embd), f(b, z.n_embd)
        self.q, self.k, self.v, self.a = f(b, z.n_q), f(b, z.n_k), f(b, z.n_k), f(b, z.n_q)
        self.o, self.mid, self.logits = f(b, z.n_embd), f(b, z.n_ff), f(b, z.n_vocab)
        self.entropy, self.top_id, self.top_lp = f(b), i(b, top), f(b, top)
        self.given, self.given_lp = i(b), f(b)
        self.attn_ws = qdq.kv_attention_workspace(b, 1, max_len, z.n_heads, z.n_kv, z.head_dim)
        self.lp_ws = qdq.token_logprobs_workspace(b, z.n_vocab, top)
        self.states = None  # the prompts' last hidden states, a packed Q8_0 matrix
        self.graph = None

    def prompt(self, prompts):
        """Run the prompts through the model; the log probability of each of their tokens but the first ones.

        Leaves the caches filled and each sequence's first new token in ``ids``."""
        z, M = self.z, sum(map(len, prompts))
        if len(prompts) != self.n_seqs or min(map(len, prompts)) < 1 or max(map(len, prompts)) > self.max_len:
            raise ValueError("one prompt of 1 to max_len tokens per sequence")
        lens, most = [len(p) for p in prompts], max(map(len, prompts))
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        ids = np.concatenate(prompts).astype(np.int32)
        cu, self.kv_len[:] = i32(np.cumsum([0] + lens)), i32(lens)
        f = lambda n: torch.empty(M, n, dtype=torch.float32, device="cuda")
        h, n, y = f(z.n_embd), f(z.n_embd), f(z.n_embd)
        q, k, v, a, mid = f(z.n_q), f(z.n_k), f(z.n_k), f(z.n_q), f(z.n_ff)
        ws = torch.empty(max(qdq.gemm_batch_workspace_bytes(M, z.n_embd, z.n_ff), qdq.gemm_batch_workspace_bytes(M, z.n_embd, z.n_q),
                             qdq.gemm_batch_workspace_bytes(M, z.n_vocab, z.n_embd),
                             qdq.q4k_swiglu_batch_workspace_bytes(M, z.n_ff, z.n_embd)), dtype=torch.uint8, device="cuda")
        attn_ws = qdq.kv_attention_workspace(self.n_seqs, most, most, z.n_heads, z.n_kv, z.head_dim)
        qdq.q6k_get_rows(self.embed, i32(ids), h, M, z.n_vocab, z.n_embd)
        fresh = None  # the last layer's output, which the next norm adds to h
        for w, cache in zip(self.layers, self.caches):
            if fresh is None:
                qdq.rms_norm(h, w["n1"], n, M, z.n_embd, z.eps)
            else:
                qdq.rms_norm(fresh, w["n1"], n, M, z.n_embd, z.eps, residual=h, sum_out=h)
            for m, out, width in ((w["q"], q, z.n_q), (w["k"], k, z.n_k), (w["v"], v, z.n_k)):
                qdq.q4k_gemm_batch(m, n, out, ws, width, z.n_embd, M)
            qdq.kv_append(cache, self.table, self.kv_len, k, v, z.n_kv, z.head_dim, z.page_tokens, cu_new=cu, max_new=most)
            qdq.kv_attention(cache, self.table, self.kv_len, q, a, attn_ws, z.n_heads, z.n_kv, z.head_dim, z.page_tokens, most,
                             cu_q=cu, max_q=most, slopes=self.slopes)
            qdq.q4k_gemm_batch(w["o"], a, y, ws, z.n_embd, z.n_q, M)
            qdq.rms_norm(y, w["n2"], n, M, z.n_embd, z.eps, residual=h, sum_out=h)
            qdq.q4k_swiglu_batch(w["g"], w["u"], n, mid, ws, z.n_ff, z.n_embd, M)
            qdq.q4k_gemm_batch(w["d"], mid, y, ws, z.n_embd, z.n_ff, M)
            fresh = y
        self.states = torch.empty(qdq.q8_0_packed_bytes(M, z.n_embd), dtype=torch.uint8, device="cuda")
        self.n_states = M
        qdq.rms_norm(fresh, self.gain, n, M, z.n_embd, z.eps, residual=h, q8_out=self.states)
        logits = f(z.n_vocab)
        qdq.q8_0_gemm_batch(self.head, n, logits, ws, z.n_vocab, z.n_embd, M)
        # row r is asked for the token after it; a sequence's last row only for its best ones
        after = i32(np.concatenate([np.append(p[1:], 0) for p in prompts]))
        lp, entropy = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        top_id = torch.empty(M, self.top, dtype=torch.int32, device="cuda")
        top_lp = torch.empty(M, self.top, device="cuda")
        qdq.token_logprobs(logits, after, lp, entropy, M, z.n_vocab, qdq.token_logprobs_workspace(M, z.n_vocab, self.top),
                           self.top, top_id, top_lp)
        last = cu[1:].long() - 1
        self.ids.copy_(top_id[last, 0])
        return [x[:-1] for x in torch.split(lp, lens)]

    def launch_step(self):
        """The kernels of one step: ``ids`` in, the next ones out; the cache has one token more."""
        z, b = self.z, self.n_seqs
        self.kv_len += 1
        qdq.q6k_get_rows(self.embed, self.ids, self.h, b, z.n_vocab, z.n_embd)
        for w, cache in zip(self.layers, self.caches):
            qdq.rms_norm(self.h, w["n1"], self.n, b, z.n_embd, z.eps)
            qdq.q4k_qkv(w["q"], w["k"], w["v"], self.n, self.q, self.k, self.v, z.n_q, z.n_k, z.n_embd, b)
            qdq.kv_append(cache, self.table, self.kv_len, self.k, self.v, z.n_kv, z.head_dim, z.page_tokens)
            qdq.kv_attention(cache, self.table, self.kv_len, self.q, self.a, self.attn_ws, z.n_heads, z.n_kv, z.head_dim,
                             z.page_tokens, self.max_len, slopes=self.slopes)
            qdq.q4k_gemv(w["o"], self.a, self.o, z.n_embd, z.n_q, b)
            qdq.rms_norm(self.o, w["n2"], self.n, b, z.n_embd, z.eps, residual=self.h, sum_out=self.h)
            qdq.q4k_ffn_residual(w["g"], w["u"], w["d"], self.n, self.h, self.h, self.mid, z.n_embd, z.n_ff, b)
        qdq.rms_norm(self.h, self.gain, self.n, b, z.n_embd, z.eps)
        qdq.q8_0_gemv(self.head, self.n, self.logits, z.n_vocab, z.n_embd, b)
        qdq.token_logprobs(self.logits, self.given, self.given_lp, self.entropy, b, z.n_vocab, self.lp_ws, self.top, self.top_id,
                           self.top_lp)
        self.ids.copy_(self.top_id[:, 0])

    def capture(self):
        """Record one step; replaying it runs the step."""
        ids, kv_len = self.ids.clone(), self.kv_len.clone()
        room = torch.clamp(kv_len, max=self.max_len - 1)
        self.kv_len.copy_(room)
        # one step outside the capture sets up what the library keeps per device; what it changed is put back
        saved = [c.clone() for c in self.caches]
        self.launch_step()
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.launch_step()
        for c, s in zip(self.caches, saved):
            c.copy_(s)
        self.ids.copy_(ids)
        self.kv_len.copy_(kv_len)

    def generate(self, n_new: int, graph: bool = True):
        """The next ``n_new`` tokens of each sequence (best ones first in ``top_id``) and their log probabilities."""
        if int(self.kv_len.max()) + n_new > self.max_len:
            raise ValueError("no room in the cache")
        if graph and self.graph is None:
            self.capture()
        ids = torch.empty(n_new, self.n_seqs, dtype=torch.int32, device="cuda")
        lps = torch.empty(n_new, self.n_seqs, device="cuda")
        for t in range(n_new):
            self.graph.replay() if graph else self.launch_step()
            ids[t], lps[t] = self.ids, self.top_lp[:, 0]
        return ids.t().contiguous(), lps.t().contiguous()

    def recall(self):
        """Products of each sequence's present hidden state with all of the prompts' states."""
        out = torch.empty(self.n_seqs, self.n_states, device="cuda")
        qdq.q8_0_gemv(self.states, self.n, out, self.n_states, self.z.n_embd, self.n_seqs)
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 1, 300], help="their lengths")
    ap.add_argument("--new", type=int, default=32)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    z = Sizes(n_layers=args.layers)
    dec = Decoder(z, random_weights(z, args.seed), len(args.prompts), max(args.prompts) + args.new)
    rng = np.random.default_rng(args.seed)
    lp = dec.prompt([synth.token_ids(rng, n, z.n_vocab) for n in args.prompts])
    for s, x in enumerate(lp):
        print(f"prompt {s}: {len(x) + 1} tokens" + (f", mean log probability {float(x.mean()):.3f}" if len(x) else ""))
    dec.capture()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    ids, lps = dec.generate(args.new)
    stop.record()
    torch.cuda.synchronize()
    for s in range(dec.n_seqs):
        print(f"sequence {s}: {ids[s, :8].tolist()} ..., mean log probability {float(lps[s].mean()):.3f}")
    print(f"{start.elapsed_time(stop) / args.new * 1e3:.1f} us per step of {dec.n_seqs} tokens, {z.n_layers} layers")


if __name__ == "__main__":
    main()
