"""A decode loop over the library's calls: QKV projection, rotary positions
with cache append, attention over the paged cache, output projection, LM head
and sampling, for a batch of sequences with prompts of different lengths.

    python examples/decode_step.py [--steps 8] [--kv e4m3|mxfp4]

One layer of a 1024-wide model (16 query heads, 8 key/value heads of 128) with
random Q8G64 weights and a small vocabulary; norms and the residual, which are
not this library's, are left out.  Each call enqueues on the current stream and
nothing is copied to the host inside the loop.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from weight_only_block_amd import qgemv as Q  # noqa: E402
from weight_only_block_amd import synth  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB, PAGE = 1024, 16, 8, 128, 2000, 16
WIDTH = (Q_HEADS + 2 * KV_HEADS) * DIM


class Block:
    """Weights, cache and buffers of the layer for up to `seqs` sequences of
    at most `length` tokens."""

    def __init__(self, seqs: int, length: int, kv: str = "bf16", seed: int = 0):
        rng = synth.rng_for(41, seed)
        self.seqs, self.length = seqs, length
        # each matrix in two layouts: one row takes the plain calls, 2..16 the matrix cores'
        self.qkv = self._matrix(rng, WIDTH, HIDDEN)
        self.o = self._matrix(rng, HIDDEN, Q_HEADS * DIM)
        self.head = self._matrix(rng, VOCAB, HIDDEN)
        self.embed = torch.from_numpy(rng.standard_normal((VOCAB, HIDDEN)).astype(np.float32)).bfloat16().cuda()
        pages_each = -(-length // PAGE)
        shape = (seqs * pages_each, KV_HEADS, PAGE, DIM)
        if kv == "bf16":
            self.cache = Q.KVCache(*[torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
        elif kv == "mxfp4":
            shapes = [shape[:3] + (DIM // 2,)] * 2 + [shape[:3] + (DIM // 32,)] * 2      # codes, exponent bytes
            self.cache = Q.KVCache(*[torch.zeros(s, dtype=torch.uint8, device="cuda") for s in shapes])
        else:
            # keys and values of these weights are of the order of 10: 448 codes cover some 40
            scales = [torch.full((KV_HEADS,), 0.1, device="cuda") for _ in range(2)]
            self.cache = Q.KVCache(*[torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)],
                                   *scales)
        self.rope = Q.Rope(DIM, base=1000000.0)
        # sequence b owns pages in a mixed order
        order = torch.from_numpy(rng.permutation(seqs * pages_each).astype(np.int32)).cuda()
        self.table = order.view(seqs, pages_each)
        self.len = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        size = max(Q.paged_attention_workspace_size(self.cache, seqs * n, Q_HEADS, seqs, n, length) for n in (1, length))
        self.workspace = torch.zeros(size, dtype=torch.uint8, device="cuda")
        self.sample_space = torch.zeros(Q.sample_workspace_size(seqs, VOCAB), dtype=torch.uint8, device="cuda")

    @staticmethod
    def _matrix(rng, n, k):
        q, s = synth.q8g64_weights(rng, n, k)
        s = (s.view(np.float16) * np.float16(2.0 ** -6)).view(np.uint16)
        dev = lambda a: torch.from_numpy(a).cuda()
        return {"n": n, "k": k, "plain": dev(Q.qpack_q8g64(q, s)), "mma": dev(Q.qpack_q8g64_mma(q, s)), "q": q, "s": s}

    @staticmethod
    def project(w, x):
        """x [rows][K] bf16 through a matrix, up to 16 rows a call."""
        y = torch.empty(x.shape[0], w["n"], dtype=torch.float32, device="cuda")
        for at in range(0, x.shape[0], 16):
            part = x[at:at + 16]
            if part.shape[0] == 1:
                Q.qgemv_q8g64(w["plain"], part, y[at:at + 16], w["n"], w["k"])
            else:
                Q.qgemv_q8g64_mma(w["mma"], part, y[at:at + 16], w["n"], w["k"])
        return y

    def forward(self, tokens, counts):
        """New tokens (ids, sequence after sequence; counts[b] of them for
        sequence b) -> logits after each sequence's last one."""
        starts = torch.zeros(self.seqs + 1, dtype=torch.int32, device="cuda")
        n = torch.tensor(counts, dtype=torch.int32, device="cuda")
        starts[1:] = torch.cumsum(n, 0)
        total, most = sum(counts), max(counts)
        owner = torch.repeat_interleave(torch.arange(self.seqs, device="cuda"), n.long(), output_size=total)
        pos = self.len[owner] + (torch.arange(total, device="cuda") - starts[owner]).int()
        slots = self.table[owner, (pos // PAGE).long()].long() * PAGE + pos % PAGE
        x = self.embed[tokens.long()]
        qkv = self.project(self.qkv, x).view(total, -1, DIM)
        q = torch.empty(total, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        Q.rope_append(self.cache, self.rope, qkv[:, :Q_HEADS], qkv[:, Q_HEADS:Q_HEADS + KV_HEADS],
                      qkv[:, Q_HEADS + KV_HEADS:], pos.int(), slots, q)
        self.len += n
        out = torch.empty_like(q)
        Q.paged_attention(self.cache, q, out, starts, self.len, self.table, self.workspace, most, self.length)
        y = self.project(self.o, out.view(total, -1)[starts[1:].long() - 1].contiguous())
        self.last = {"q": q, "out": out, "starts": starts, "len": self.len.clone()}
        return self.project(self.head, y.bfloat16())

    def cached(self, seq: int, dtype=torch.bfloat16):
        """Keys and values of one sequence as the cache holds them, [tokens][heads][dim]:
        for another worker, or a cache of another type."""
        i = torch.arange(int(self.len[seq]), device="cuda")
        slots = self.table[seq, i // PAGE].long() * PAGE + i % PAGE
        k, v = [torch.empty(len(i), KV_HEADS, DIM, dtype=dtype, device="cuda") for _ in range(2)]
        Q.kv_read(self.cache, slots, k, v)
        return k, v

    def sample(self, logits, u, **settings):
        idx = torch.empty(self.seqs, dtype=torch.int32, device="cuda")
        Q.sample_f32(logits, u, idx, self.sample_space, **settings)
        return idx


def generate(block, prompts, steps, seed=0, watch=None):
    """Token ids that follow the prompts: [steps][seqs], on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    settings = {"temperature": torch.full((block.seqs,), 0.8, device="cuda"),
                "top_k": torch.full((block.seqs,), 50, dtype=torch.int32, device="cuda"),
                "top_p": torch.full((block.seqs,), 0.95, device="cuda"),
                "min_p": torch.full((block.seqs,), 0.01, device="cuda")}
    tokens, counts, out = torch.cat(prompts), [len(p) for p in prompts], []
    for _ in range(steps):
        logits = block.forward(tokens, counts)
        u = torch.rand(block.seqs, generator=g, device="cuda")
        tokens = block.sample(logits, u, **settings)
        counts = [1] * block.seqs
        if watch:
            watch(block, logits, u, tokens, settings)
        out.append(tokens)
    return torch.stack(out)


def main():
    args = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    args.add_argument("--steps", type=int, default=8)
    args.add_argument("--kv", choices=("bf16", "e4m3", "mxfp4"), default="bf16")
    opts = args.parse_args()
    lengths = [37, 5, 120, 64]
    block = Block(len(lengths), max(lengths) + opts.steps, opts.kv)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).int().cuda() for n in lengths]
    for row in generate(block, prompts, opts.steps).t().tolist():
        print(" ".join("%4d" % t for t in row))


if __name__ == "__main__":
    main()
