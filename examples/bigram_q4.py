"""A next-token model from end to end on the library's dense-table operators.

A bigram model (the next token's logits are W · E[token]) is trained on tokens
of a random Markov chain: lookups by ``spmv_embed``, the gradient of the table by
``spmv_embed_grad``. W is then converted to 4 bits by ``spmv_q4_quantize`` and
tokens are decoded one at a time, the lookup and the 4-bit product
``spmv_q4_run`` captured in one CUDA graph per step; the table is served from 4
bits too (``spmv_embed_q4``).

    python examples/bigram_q4.py [--vocab 2000] [--dim 256] [--steps 200]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spmv_sparse_storage_gb300 as sp  # noqa: E402


def chain(vocab, gen, follow=4):
    """A Markov chain in which each token has a few likely successors."""
    after = torch.randint(0, vocab, (vocab, follow), device="cuda", generator=gen)
    weight = torch.rand(vocab, follow, device="cuda", generator=gen) ** 2 + 0.05
    return after, weight / weight.sum(1, keepdim=True)


def sample(after, weight, n, gen):
    """n (token, next token) pairs."""
    t = torch.randint(0, after.shape[0], (n,), device="cuda", generator=gen)
    pick = torch.multinomial(weight[t], 1, generator=gen)
    return t, after[t].gather(1, pick)[:, 0]


class Q4:
    """A matrix converted to 4 bits: codes, scales and zero points."""

    def __init__(self, w, group=64):
        rows, cols = w.shape
        self.group = group
        self.codes = torch.empty(rows, (cols + 1) // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(rows, -(-cols // group), dtype=torch.bfloat16, device="cuda")
        self.zeros = torch.empty_like(self.scales, dtype=torch.uint8)
        sp.spmv_q4_quantize(w, self.codes, self.scales, group, zeros=self.zeros)

    def product(self, x, y):
        sp.spmv_q4_run(self.codes, self.scales, self.group, x, y, zeros=self.zeros)

    def rows(self, tokens, out, scale):
        sp.spmv_embed_q4(self.codes, self.scales, self.group, tokens, out, scale=scale,
                         zeros=self.zeros)


def train(vocab, dim, steps, batch, gen, lr=2.0):
    """(E, W, chain, first loss, last loss): plain gradient descent on the cross entropy."""
    law = chain(vocab, gen)
    scale = math.sqrt(dim)
    E = torch.randn(vocab, dim, device="cuda", generator=gen) * (0.3 / scale)
    W = torch.randn(vocab, dim, device="cuda", generator=gen) * (0.3 / scale)
    dE, x = torch.empty_like(E), torch.empty(batch, dim, device="cuda")
    losses = []
    for _ in range(steps):
        token, target = sample(*law, batch, gen)
        sp.spmv_embed(E, token, x, scale=scale)
        logits = x @ W.t()
        losses.append(torch.nn.functional.cross_entropy(logits, target))
        g = torch.softmax(logits, 1)
        g[torch.arange(batch, device="cuda"), target] -= 1.0
        g /= batch
        dx = g @ W
        W -= (lr * scale) * (g.t() @ x)
        sp.spmv_embed_grad(dx, token, dE, scale=scale)
        E -= (lr / scale) * dE
    losses = torch.stack(losses).tolist()
    return E, W, law, losses[0], sum(losses[-5:]) / len(losses[-5:])


def decode(E4, W4, dim, first, n):
    """n tokens after ``first``, greedily, one 4-bit lookup and product a token."""
    scale = math.sqrt(dim)
    vocab = W4.codes.shape[0]
    token = torch.tensor([first], device="cuda")
    x = torch.empty(1, dim, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(1, vocab, device="cuda")

    def step():
        E4.rows(token, x, scale)
        W4.product(x, logits)
        token.copy_(logits.argmax(1))

    step()  # outside the capture first
    token.fill_(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out = []
    for _ in range(n):
        graph.replay()
        out.append(token.clone())
    return torch.cat(out).tolist()


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--vocab", type=int, default=2000)
    p.add_argument("--dim", type=int, default=256)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--batch", type=int, default=8192)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(a.seed)
    E, W, law, first, last = train(a.vocab, a.dim, a.steps, a.batch, gen)
    E4, W4 = Q4(E), Q4(W)
    # the 4-bit model's loss on new pairs, against the trained one's
    token, target = sample(*law, a.batch, gen)
    scale = math.sqrt(a.dim)
    x = torch.empty(a.batch, a.dim, device="cuda")
    sp.spmv_embed(E, token, x, scale=scale)
    dense = float(torch.nn.functional.cross_entropy(x @ W.t(), target))
    x4, y4 = x.bfloat16(), torch.empty(a.batch, a.vocab, device="cuda")
    E4.rows(token, x4, scale)
    W4.product(x4, y4)
    quant = float(torch.nn.functional.cross_entropy(y4, target))
    text = decode(E4, W4, a.dim, 0, 32)
    likely = sum(int(b in law[0][t].tolist()) for t, b in zip([0] + text[:-1], text))
    print(f"loss {first:.3f} -> {last:.3f}; on new pairs {dense:.3f}, in 4 bits {quant:.3f}; "
          f"{likely} of {len(text)} decoded tokens follow the chain")
    return {"first": first, "last": last, "dense": dense, "quant": quant, "likely": likely,
            "decoded": len(text)}


if __name__ == "__main__":
    main()
