"""Several continuations of one prompt, drawn side by side.

A one-layer model with random weights stands in for a language model; what is shown is the
decode loop around it:

1. the prompt's keys and values go into a paged cache (``PagedBatch.build_tables`` says where);
2. the first token of every continuation is drawn from the prompt's one row of logits, with one
   given random number each (``Sampler.sample_given``);
3. each step, the continuations' tables grow, their new keys and values are stored, attention
   reads the shared part of the prompt once for all of them (``PagedBatch.attention``), and the
   next tokens are drawn.

Run: python examples/parallel_sampling.py [--continuations 32] [--prompt 1000] [--steps 24]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from device_token_sampling_gb300 import PagedBatch, Sampler  # noqa: E402

Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB, BLOCK = 16, 4, 64, 32000, 16


class Model:
    """Embedding, one attention layer with a residual, and a head."""

    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        d = Q_HEADS * HEAD_DIM

        def weights(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()

        self.embed = weights(VOCAB, d, scale=1.0)
        self.qkv = weights(d, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM, scale=d ** -0.5)
        self.out = weights(d, d, scale=d ** -0.5)
        self.head = weights(d, VOCAB, scale=2.5 * d ** -0.5)

    def project(self, tokens):
        """Embeddings and the heads' q, k, v of ``tokens``."""
        x = self.embed[tokens]
        q, k, v = (x @ self.qkv).split((Q_HEADS * HEAD_DIM, KV_HEADS * HEAD_DIM,
                                        KV_HEADS * HEAD_DIM), dim=-1)
        return (x, q.unflatten(-1, (Q_HEADS, HEAD_DIM)), k.unflatten(-1, (KV_HEADS, HEAD_DIM)),
                v.unflatten(-1, (KV_HEADS, HEAD_DIM)))

    def logits(self, x, attended):
        h = x + attended.flatten(1) @ self.out
        h = h / h.float().square().mean(-1, keepdim=True).sqrt()
        return h.bfloat16() @ self.head


def generate(n: int, prompt_len: int, steps: int, seed: int = 0, watch=None):
    """Tokens [n, steps] of ``n`` continuations of a random prompt.  ``watch``, if given, is
    called with a dict of each step's tensors."""
    dev = "cuda"
    model = Model(seed)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    prompt = torch.randint(0, VOCAB, (prompt_len,), generator=g, device=dev)
    uniforms = torch.rand((steps, n), generator=g, device=dev)

    def i32(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    columns = -(-(prompt_len + steps) // BLOCK)
    shared = prompt_len // BLOCK              # whole blocks of the prompt are shared
    tail = prompt_len - shared * BLOCK        # the rest each continuation holds itself
    n_blocks = columns + n * (columns - shared)
    cache = torch.zeros((2, n_blocks, BLOCK, KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=dev)
    keys, values = cache[0], cache[1]
    slots_of = cache.flatten(1, 2)
    free = torch.randperm(n_blocks, generator=g, device=dev).int()

    sampler = Sampler(max_batch=n, max_vocab=VOCAB)
    ones, zeros = np.ones(n, np.float32), np.zeros(n, np.float32)
    sampler.reset_params(0.9 * ones, np.full(n, 200), 0.95 * ones, 0.01 * ones, zeros, zeros, ones,
                         np.zeros(n, np.uint64))
    paged = PagedBatch(n, BLOCK, columns, Q_HEADS, KV_HEADS, HEAD_DIM)
    first = PagedBatch(1, BLOCK, columns, Q_HEADS, KV_HEADS, HEAD_DIM)

    # the prompt, one request
    table = torch.empty((1, columns), dtype=torch.int32, device=dev)
    held, cursor, _, slots, _, status = first.build_tables(
        table, i32([prompt_len]), i32([prompt_len]), free, i32([0]), capacity=prompt_len)
    x, q, k, v = model.project(prompt)
    slots_of[0].index_copy_(0, slots, k)
    slots_of[1].index_copy_(0, slots, v)
    attended, _ = first.attention(q[-1:], keys, values, table, i32([prompt_len]))
    logits = model.logits(x[-1:], attended)
    # one row, n draws
    tokens, _ = sampler.sample_given(logits, uniforms[:1])
    tokens = tokens[0]
    if watch:
        watch(dict(step=0, logits=logits, uniforms=uniforms[:1], tokens=tokens, status=status))

    # the continuations: a table of their own behind the shared blocks
    prefix = table[0, :shared].contiguous()
    table = torch.empty((n, columns), dtype=torch.int32, device=dev)
    lens = torch.full((n,), prompt_len, dtype=torch.int32, device=dev)
    held, cursor, _, slots, _, _ = paged.build_tables(
        table, lens, torch.full_like(lens, tail), free, cursor, prefix_blocks=prefix,
        capacity=n * tail)
    if tail:
        slots_of[0].index_copy_(0, slots, k[-tail:].repeat(n, 1, 1))
        slots_of[1].index_copy_(0, slots, v[-tail:].repeat(n, 1, 1))
    one = torch.ones_like(lens)
    drawn = [tokens]
    for step in range(1, steps):
        lens = lens + 1
        held, cursor, _, slots, _, status = paged.build_tables(
            table, lens, one, free, cursor, held=held, prefix_blocks=prefix)
        x, q, k, v = model.project(tokens)
        slots_of[0].index_copy_(0, slots, k)
        slots_of[1].index_copy_(0, slots, v)
        attended, lse = paged.attention(q, keys, values, table, lens, prefix, shared * BLOCK,
                                        max_seq_len=prompt_len + step)
        logits = model.logits(x, attended)
        tokens, _ = sampler.sample_given(logits, uniforms[step])
        drawn.append(tokens)
        if watch:
            watch(dict(step=step, q=q, keys=keys, values=values, table=table, lens=lens,
                       prefix=prefix, attended=attended, lse=lse, logits=logits,
                       uniforms=uniforms[step], tokens=tokens, status=status))
    paged.check_errors()
    sampler.check_device_errors()
    return torch.stack(drawn, 1)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--continuations", type=int, default=32)
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--steps", type=int, default=24)
    a = p.parse_args()
    for row in generate(a.continuations, a.prompt, a.steps).tolist():
        print(*row)


if __name__ == "__main__":
    main()
