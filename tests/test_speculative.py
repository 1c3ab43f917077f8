"""Speculative decoding over a paged cache with branches: fork, copies, tables, attention of the
drafted chunk, verification, release and compaction together.  A plain record of every request's
own keys and values stands beside the cache."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from pagedlib import chunk_reference
from test_verify import check

HQ, HKV, D, V = 8, 2, 64, 700


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Loop:
    """The serving state of ``rows`` requests, and the record that it is held against."""

    def __init__(self, lens, bs, K, n_blocks, seed):
        from device_token_sampling_gb300 import PagedBatch, Sampler
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.bs, self.K, self.n = len(lens), bs, K, n_blocks
        self.cols = -(-(max(lens) + 400) // bs)
        self.paged = PagedBatch(self.B, bs, self.cols, HQ, HKV, D)
        self.sampler = Sampler(max_batch=self.B, max_vocab=V)
        self.cache = torch.zeros((2, n_blocks, bs, HKV, D), dtype=torch.bfloat16, device="cuda")
        self.wq = torch.randn((D * HQ, V), generator=self.g, device="cuda") * 0.2
        self.table = torch.full((self.B, self.cols), -1, dtype=torch.int32, device="cuda")
        self.held = i32([0] * self.B)
        self.free, self.cursor = i32(self.rng.permutation(n_blocks)), i32([0])
        self.lens = i32([0] * self.B)
        self.record = [torch.zeros((2, 0, HKV, D), dtype=torch.bfloat16, device="cuda")
                       for _ in lens]
        self.grow(np.asarray(lens))

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").bfloat16()

    def grow(self, n):
        """n[b] new tokens a request: blocks, slots, keys and values.  Returns the starts."""
        self.lens = self.lens + i32(n)
        T = int(n.sum())
        self.held, self.cursor, starts, slots, positions, status = self.paged.build_tables(
            self.table, self.lens, i32(n), self.free, self.cursor, held=self.held, capacity=T)
        assert (status == 0).all()
        new = self.randn(2, T, HKV, D)
        self.cache.flatten(1, 2).index_copy_(1, slots, new)
        at = np.concatenate([[0], np.cumsum(n)])
        for b in range(self.B):
            self.record[b] = torch.cat([self.record[b], new[:, at[b]:at[b + 1]]], 1)
        return starts

    def branch(self, parents):
        """The rows of the next step continue ``parents``."""
        new = torch.empty_like(self.table)
        self.held, self.lens, self.cursor, src, dst, status = self.paged.fork(
            self.table, self.held, self.lens, i32(parents), self.free, self.cursor, new)
        assert (status == 0).all()
        self.paged.copy_blocks([self.cache[0], self.cache[1]], src, dst)
        self.table = new
        self.record = [self.record[p] for p in parents]

    def step(self):
        """Draft, attend, verify, keep what was accepted."""
        n = self.rng.integers(0, self.K + 1, self.B)
        starts = self.grow(n + 1)
        T = int(n.sum()) + self.B
        q = self.randn(T, HQ, D)
        out, lse = self.paged.chunk_attention(q, starts, self.cache[0], self.cache[1],
                                              self.table, self.lens)
        want, wlse, b_out, b_lse = chunk_reference(q, starts, self.cache[0], self.cache[1],
                                                   self.table, self.lens, self.bs, D ** -0.5)
        assert bool(((out.double() - want).abs() <= b_out).all())
        assert bool(((lse.double() - wlse).abs() <= b_lse).all())
        z = out.float().flatten(1) @ self.wq * 8
        p = z.softmax(-1)
        draft = torch.zeros((self.B, self.K, V), device="cuda")
        at = starts.tolist()
        for b in range(self.B):
            draft[b, :n[b]] = (z[at[b]:at[b] + n[b]]
                               + torch.randn((n[b], V), generator=self.g, device="cuda") * 0.5
                               ).softmax(-1)
        draft[:, :, 0] += 1e-6
        x = torch.multinomial(draft.flatten(0, 1), 1, generator=self.g).view(self.B, self.K).int()
        u = torch.rand((self.B, self.K + 1), generator=self.g, device="cuda")
        tokens, accepted = self.sampler.verify(p, x, u, draft_probs=draft, draft_lens=i32(n),
                                               starts=starts)
        for b in range(self.B):
            check(tokens[b].cpu().numpy(), int(accepted[b]), p[at[b]:at[b + 1]].cpu().numpy(),
                  x[b].cpu().numpy(), u[b].cpu().numpy(), draft[b].cpu().numpy(), int(n[b]))
        self.lens = self.lens - i32(n) + accepted
        for b in range(self.B):
            self.record[b] = self.record[b][:, :int(self.lens[b])]
        self.held, self.free, self.cursor = self.paged.release(self.table, self.held, self.lens,
                                                               self.n)
        return int(accepted.sum()), int(n.sum())

    def pack(self):
        self.held, self.free, self.cursor, src, dst, count, _ = self.paged.compact(
            self.table, self.held, self.lens, self.n)
        self.paged.copy_blocks([self.cache[0], self.cache[1]], src, dst, count=count)
        n = int(self.cursor)
        assert int(self.table.max()) < n and torch.equal(
            torch.unique(self.table[self.table >= 0]).int(),
            torch.arange(n, device="cuda").int())

    def hold_against_the_record(self):
        """Every request's cached tokens are its own; no free block is anybody's."""
        self.paged.check_errors()
        self.sampler.check_device_errors()
        free = set(self.free[int(self.cursor):].tolist())
        for b in range(self.B):
            m = int(self.lens[b])
            assert m == self.record[b].shape[1]
            assert int(self.held[b]) == -(-m // self.bs)
            ids = self.table[b, :int(self.held[b])]
            assert not free & set(ids.tolist())
            assert (self.table[b, int(self.held[b]):] == -1).all()
            assert torch.equal(self.cache[:, ids.long()].flatten(1, 2)[:, :m], self.record[b])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,bs,K", [
    ([1, 40, 7, 130, 64], 16, 4), ([300], 64, 7), ([5] * 40, 8, 1), ([33, 900], 4, 5)])
def test_loop(lens, bs, K):
    B = len(lens)
    need = sum(-(-(m + 80) // bs) for m in lens) * 2 + 2 * B
    loop = Loop(lens, bs, K, need, seed=B * bs)
    accepted = drafted = 0
    for step in range(9):
        if step % 3 == 1:           # some rows end, others go on twice and more
            loop.branch(np.sort(loop.rng.integers(0, B, B)) if step == 1
                        else loop.rng.integers(0, B, B))
        a, n = loop.step()
        accepted, drafted = accepted + a, drafted + n
        loop.hold_against_the_record()
        if step % 4 == 2:
            loop.pack()
            loop.hold_against_the_record()
    assert 0 < accepted < drafted


@pytest.mark.gpu
def test_captured_step():
    """Tables, attention, verification, release and the move to the low ids as one graph, on
    buffers of their own, replayed over several steps, against the same calls one by one."""
    from device_token_sampling_gb300 import PagedBatch, Sampler
    B, bs, K, n, cols = 6, 16, 3, 400, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    T = B * (K + 1)
    steps = [dict(new=torch.randn((2, T, HKV, D), generator=g, device="cuda").bfloat16(),
                  q=torch.randn((T, HQ, D), generator=g, device="cuda").bfloat16(),
                  x=torch.randint(0, 9, (B, K), generator=g, device="cuda").int(),
                  u=torch.rand((B, K + 1), generator=g, device="cuda")) for _ in range(5)]
    wq = torch.randn((D * HQ, V), generator=g, device="cuda") * 0.1
    prompt = torch.randn((2, n, bs, HKV, D), generator=g, device="cuda").bfloat16()
    results = []
    for captured in (False, True):
        with PagedBatch(B, bs, cols, HQ, HKV, D) as p, Sampler(max_batch=B, max_vocab=V) as s:
            cache, live = prompt.clone(), {k: v.clone() for k, v in steps[0].items()}
            table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
            lens = i32([3, 16, 100, 31, 64, 250])
            held, cursor, *_ = p.build_tables(table, lens, lens * 0, torch.arange(n).int().cuda()
                                              .flip(0).contiguous(), i32([0]))
            free = torch.arange(n).int().cuda().flip(0).contiguous()

            def step():
                lens.add_(K + 1)
                h, c, starts, slots, _, status = p.build_tables(
                    table, lens, torch.full_like(lens, K + 1), free, cursor, held=held, capacity=T)
                cache.flatten(1, 2).index_copy_(1, slots, live["new"])
                out, _ = p.chunk_attention(live["q"], starts, cache[0], cache[1], table, lens)
                probs = (out.float().flatten(1) @ wq).softmax(-1)
                probs[:, :9] *= 20
                probs /= probs.sum(-1, keepdim=True)
                tokens, accepted = s.verify(probs, live["x"], live["u"], starts=starts)
                lens.sub_(K - accepted)
                r = p.release(table, h, lens, n)
                m = p.compact(table, r[0], lens, n)
                p.copy_blocks([cache[0], cache[1]], m[3], m[4], count=m[5])
                held.copy_(m[0])
                free.copy_(m[1])
                cursor.copy_(m[2])
                return tokens, accepted, status, out

            state = [x.clone() for x in (cache, table, lens, held, free, cursor)]
            graph = None
            if captured:
                step()                                # (what is set up by a first call)
                for x, was in zip((cache, table, lens, held, free, cursor), state):
                    x.copy_(was)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    got = step()
            seen = []
            for x in steps:
                for k in live:
                    live[k].copy_(x[k])
                if captured:
                    graph.replay()
                else:
                    got = step()
                assert (got[2] == 0).all()
                seen += [t.clone() for t in got + (table, lens, held, free, cursor)]
            p.check_errors()
            s.check_device_errors()
            results.append(seen + [cache])
    assert sum(int(x.sum()) for x in results[0][1::9][:5]) > 0
    for a, b in zip(*results):
        assert torch.equal(a, b)
