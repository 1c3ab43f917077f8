"""PagedBatch.fork, release, compact and copy_blocks against plain references."""
from __future__ import annotations

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def fork_reference(table, held, seq, parents, free, cursor, bs, cols):
    """One row at a time; returns (table, held, seq, cursor, src, dst, status)."""
    R, B = len(parents), len(seq)
    out = np.full((R, cols), -1)
    o_held, o_seq, status = np.zeros(R, int), np.zeros(R, int), np.zeros(R, int)
    src, dst = np.full(R, -1), np.full(R, -1)
    at = cursor if 0 <= cursor <= len(free) else len(free)
    got = 0
    seen = set()
    for r, p in enumerate(parents):
        if p == -1:
            continue
        if not 0 <= p < B:
            status[r] = 2
            continue
        first = p not in seen
        seen.add(p)
        blocks = -(-seq[p] // bs)
        if seq[p] < 0 or held[p] < 0 or held[p] > cols or blocks > held[p]:
            status[r] = 2
            continue
        if first:
            n = held[p]
            out[r, :n] = table[p, :n]
        else:
            n = blocks
            if seq[p] % bs:
                if at + got >= len(free):
                    status[r] = 1
                    continue
                src[r], dst[r] = table[p, n - 1], free[at + got]
                got += 1
            out[r, :n] = table[p, :n]
            if dst[r] >= 0:
                out[r, n - 1] = dst[r]
        o_held[r], o_seq[r] = n, seq[p]
    return out, o_held, o_seq, cursor + got if got else cursor, src, dst, status


def reclaim_reference(table, held, seq, n_blocks, prefix, bs, cols):
    """(table, held, free, cursor) of release, and of compact (table, src, dst, prefix)."""
    B = len(seq)
    kept = [min(-(-max(s, 0) // bs), min(max(h, 0), cols)) for s, h in zip(seq, held)]
    used = set(int(x) for x in prefix if 0 <= x < n_blocks)
    for r in range(B):
        used |= {int(x) for x in table[r, :kept[r]] if 0 <= x < n_blocks}
    order = sorted(used)
    free = order + [x for x in range(n_blocks) if x not in used]
    n = len(order)
    out = np.array(table)
    for r in range(B):
        out[r, kept[r]:cols] = -1
    src = [x for x in order if x >= n]
    dst = [x for x in range(n) if x not in used]
    now = {x: x for x in order if x < n} | dict(zip(src, dst))
    new = np.full((B, cols), -1)
    for r in range(B):
        new[r, :kept[r]] = [now.get(int(x), -1) for x in table[r, :kept[r]]]
    pad = [-1] * (n_blocks // 2 - len(src))
    return (out, kept, free, n, new, src + pad, dst + pad, len(src),
            [now.get(int(x), -1) for x in prefix])


def paged(B, bs, cols):
    from device_token_sampling_gb300 import PagedBatch
    return PagedBatch(max_batch=B, block_size=bs, max_blocks=cols)


@gpu
@pytest.mark.parametrize("B,R,bs,cols,extra", [
    (1, 1, 16, 4, 0), (1, 9, 16, 4, 3), (5, 3, 1, 40, 0), (7, 600, 8, 300, 5),
    (40, 17, 64, 257, 1), (3, 1500, 16, 20, 0), (1024, 1024, 4, 33, 2)])
def test_fork(B, R, bs, cols, extra):
    g = np.random.default_rng([B, R, bs])
    for case in range(3):
        seq = g.integers(0, cols * bs + 1, B)
        held = np.minimum(-(-seq // bs) + g.integers(0, 3, B), cols)
        table = g.integers(0, 10000, (B, cols + extra))
        parents = g.integers(-1, B, R)
        free = g.permutation(20000)[:R if case else max(0, R // 3)]
        cursor = [0, len(free) // 2, min(3, len(free))][case]
        if case == 2:                                  # some that are refused
            seq[g.random(B) < 0.2] *= -1
            held[g.random(B) < 0.2] = cols + 5
            parents[g.random(R) < 0.2] = B + 2
            parents[g.random(R) < 0.1] = -2
        want = fork_reference(table, held, seq, parents, free, cursor, bs, cols)
        out = torch.full((R, cols + extra), -7, dtype=torch.int32, device="cuda")
        with paged(max(B, R), bs, cols) as p:
            got = p.fork(dev(table), dev(held), dev(seq), dev(parents), dev(free), dev([cursor]),
                         out)
            p.check_errors()
        assert (out[:, cols:] == -7).all()
        np.testing.assert_array_equal(out[:, :cols].cpu(), want[0])
        for x, w, name in zip(got, want[1:], ("held", "seq", "cursor", "src", "dst", "status")):
            np.testing.assert_array_equal(x.cpu().numpy(), np.atleast_1d(w), err_msg=name)


@gpu
@pytest.mark.parametrize("cursor", [-1, 4, 2 ** 31 - 1])
def test_fork_without_a_free_list(cursor):
    """A cursor past the list leaves nothing: the children that need a block are refused."""
    table, held, seq = np.arange(8).reshape(2, 4), [2, 2], [5, 8]
    with paged(5, 4, 4) as p:
        out = torch.empty((5, 4), dtype=torch.int32, device="cuda")
        got = p.fork(dev(table), dev(held), dev(seq), dev([0, 0, 1, 1, 0]), dev([9, 9, 9]),
                     dev([cursor]), out)
    assert got[5].tolist() == [0, 1, 0, 0, 1] and got[2].item() == cursor
    assert out[2].tolist() == out[3].tolist() == [4, 5, -1, -1]


@gpu
@pytest.mark.parametrize("B,bs,cols,n_blocks,n_prefix", [
    (1, 16, 1, 1, 0), (1, 16, 4, 40, 0), (3, 1, 70, 33, 5), (29, 8, 300, 4000, 7),
    (300, 64, 33, 31, 0), (700, 16, 64, 100000, 8), (64, 16, 2000, 1 << 20, 600)])
@pytest.mark.parametrize("compact", [False, True])
def test_release_and_compact(B, bs, cols, n_blocks, n_prefix, compact):
    g = np.random.default_rng([B, bs, cols])
    for case in range(2):
        held = g.integers(0, cols + 1, B)
        seq = np.where(g.random(B) < 0.3, 0, g.integers(0, cols * bs + 2 * bs, B))
        top = n_blocks if case == 0 else max(1, n_blocks // 3)
        table = g.integers(0, top, (B, cols + 3))
        prefix = g.integers(0, n_blocks, n_prefix)
        want = reclaim_reference(table, held, seq, n_blocks, prefix, bs, cols)
        t = dev(table)
        pre = dev(prefix) if n_prefix else None
        with paged(B, bs, cols) as p:
            if not compact:
                h, free, cursor = p.release(t, dev(held), dev(seq), n_blocks, prefix_blocks=pre)
                p.check_errors()
                np.testing.assert_array_equal(t.cpu()[:, :cols], want[0][:, :cols])
                np.testing.assert_array_equal(t.cpu()[:, cols:], table[:, cols:])
                np.testing.assert_array_equal(free.cpu(), want[2])
            else:
                new = torch.full((B, cols + 1), -7, dtype=torch.int32, device="cuda")
                h, free, cursor, src, dst, count, prefix_now = p.compact(
                    t, dev(held), dev(seq), n_blocks, prefix_blocks=pre, out_table=new)
                p.check_errors()
                np.testing.assert_array_equal(t.cpu(), table)
                assert (new[:, cols:] == -7).all()
                np.testing.assert_array_equal(new.cpu()[:, :cols], want[4])
                np.testing.assert_array_equal(free.cpu(), np.arange(n_blocks))
                np.testing.assert_array_equal(src.cpu(), want[5])
                np.testing.assert_array_equal(dst.cpu(), want[6])
                assert count.item() == want[7]
                np.testing.assert_array_equal(prefix_now.cpu(), want[8])
                again = p.compact(t, dev(held), dev(seq), n_blocks, prefix_blocks=pre)
                np.testing.assert_array_equal(t.cpu()[:, :cols], want[4])   # in place
                assert again[5].item() == want[7]
        np.testing.assert_array_equal(h.cpu(), want[1])
        assert cursor.item() == want[3]


@gpu
def test_largest_batch():
    """As many rows as a handle takes, all of one parent, then of as many."""
    B, bs, cols = 16384, 16, 3
    g = np.random.default_rng(0)
    seq = g.integers(0, cols * bs + 1, B)
    held = -(-seq // bs)
    table = g.integers(0, 50000, (B, cols))
    free = np.arange(50000, 50000 + B)
    with paged(B, bs, cols) as p:
        for parents in (np.full(B, 16383), g.integers(0, B, B), np.full(B, -1)):
            want = fork_reference(table, held, seq, parents, free, 0, bs, cols)
            out = torch.empty((B, cols), dtype=torch.int32, device="cuda")
            got = p.fork(dev(table), dev(held), dev(seq), dev(parents), dev(free), dev([0]), out)
            p.check_errors()
            np.testing.assert_array_equal(out.cpu(), want[0])
            for x, w in zip(got, want[1:]):
                np.testing.assert_array_equal(x.cpu().numpy(), np.atleast_1d(w))


@gpu
@pytest.mark.parametrize("compact", [False, True])
def test_largest_cache(compact):
    """As many blocks as a cache may have, few of them in use, at both ends."""
    n, bs, cols = 1 << 24, 1, 5
    table = np.array([[n - 1, 0, n // 2, 7, 9], [3, n - 2, n - 1, 5, 5]])
    held, seq = np.array([3, 5]), np.array([4, 3])
    want = reclaim_reference(table, held, seq, 64, [], bs, cols)[1]
    used = sorted({n - 1, 0, n // 2, 3, n - 2})
    with paged(2, bs, cols) as p:
        t = dev(table)
        if not compact:
            h, free, cursor = p.release(t, dev(held), dev(seq), n)
            p.check_errors()
            assert h.tolist() == want and cursor.item() == 5 and free[:5].tolist() == used
            rest = torch.arange(n, device="cuda")
            rest = rest[~torch.isin(rest, torch.tensor(used, device="cuda"))]
            assert torch.equal(free[5:].long(), rest)
        else:
            h, free, cursor, src, dst, count, _ = p.compact(t, dev(held), dev(seq), n)
            p.check_errors()
            assert cursor.item() == 5 and count.item() == 3
            assert src[:4].tolist() == [n // 2, n - 2, n - 1, -1] and dst[:3].tolist() == [1, 2, 4]
            assert t.tolist() == [[4, 0, 1, -1, -1], [3, 2, 4, -1, -1]]
            assert torch.equal(free, torch.arange(n, device="cuda").int())


@gpu
@pytest.mark.parametrize("count,copied", [(-3, 0), (0, 0), (1, 1), (2, 2), (99, 2)])
def test_copies_counted_on_the_device(count, copied):
    cache = torch.arange(6 * 8, device="cuda").view(6, 8).float()
    want = cache.clone()
    want[torch.tensor([4, 5][:copied], dtype=torch.long)] = cache[:copied]
    with paged(1, 16, 1) as p:
        p.copy_blocks([cache], dev([0, 1]), dev([4, 5]), count=dev([count]))
        p.check_errors()
    assert torch.equal(cache, want)


@gpu
def test_ids_outside_the_cache_are_reported():
    from device_token_sampling_gb300 import VtError
    table = np.array([[0, -1, 99], [5, 2 ** 30, 3]])
    with paged(2, 4, 3) as p:
        for compact in (False, True):
            t = dev(table)
            f = p.compact if compact else p.release
            out = f(t, dev([3, 3]), dev([12, 5]), 8)
            assert out[2].item() == 2                  # 0 and 5
            with pytest.raises(VtError, match="outside the cache"):
                p.check_errors()
            p.check_errors()
        assert t.tolist() == [[0, -1, -1], [1, -1, -1]]


@gpu
@pytest.mark.parametrize("shape,dtype,strided", [
    ((40, 16, 2, 64), torch.bfloat16, None), ((40, 8, 3, 5), torch.bfloat16, None),
    ((40, 1, 1, 1), torch.uint8, None), ((40, 4, 2, 64), torch.float32, "heads"),
    ((40, 16, 8, 128), torch.float16, "pairs"), ((9, 3, 1, 7), torch.uint8, "pairs")])
def test_copy_blocks(shape, dtype, strided):
    g = torch.Generator(device="cuda").manual_seed(1)

    def cache():
        n, bs, h, d = shape
        if strided == "heads":          # [blocks, heads, tokens, d] in memory
            return torch.randint(0, 255, (n, h, bs, d), generator=g,
                                 device="cuda").to(dtype).transpose(1, 2)
        if strided == "pairs":          # keys and values of a block side by side
            return torch.randint(0, 255, (n, 2, bs, h, d), generator=g,
                                 device="cuda").to(dtype)[:, 1]
        return torch.randint(0, 255, shape, generator=g, device="cuda").to(dtype)

    for n_caches in (1, 3, 70):
        caches = [cache() for _ in range(n_caches)]
        want = [c.clone() for c in caches]
        ids = torch.randperm(shape[0], generator=g, device="cuda").int()
        src, dst = ids[:4].clone(), ids[4:8].clone()
        src[1] = -1
        for w in want:
            for a, b in zip(src.tolist()[:3], dst.tolist()[:3]):
                if a >= 0:
                    w[b] = w[a]
        with paged(1, 16, 1) as p:
            p.copy_blocks(caches, src, dst, count=dev([3]))
            p.check_errors()
            for c, w in zip(caches, want):
                assert torch.equal(c, w)
            p.copy_blocks(caches, src, dst)
            for w in want:
                w[int(dst[3])] = w[int(src[3])]
            for c, w in zip(caches, want):
                assert torch.equal(c, w)
            p.copy_blocks(caches, src[:0], dst[:0])
            p.copy_blocks([], src, dst)
            p.check_errors()


@gpu
def test_copy_blocks_far_apart():
    """Blocks past 2^31 elements."""
    cache = torch.zeros((70000, 16, 2, 1024), dtype=torch.float16, device="cuda")
    assert cache.numel() > 1 << 31
    cache[3] = 1.5
    cache[69998] = 2.5
    with paged(1, 16, 1) as p:
        p.copy_blocks([cache], dev([3, 69998]), dev([69999, 5]))
        p.check_errors()
    assert (cache[69999] == 1.5).all() and (cache[5] == 2.5).all()
    assert (cache[69997] == 0).all() and (cache[6] == 0).all()


@gpu
def test_copy_blocks_bad_ids():
    from device_token_sampling_gb300 import VtError
    cache = torch.arange(4 * 8, device="cuda").view(4, 8).half()
    want = cache.clone()
    want[2] = want[1]
    with paged(1, 16, 1) as p:
        p.copy_blocks([cache], dev([1, 4, 0]), dev([2, 0, 7]))
        with pytest.raises(VtError, match="outside the cache"):
            p.check_errors()
    assert torch.equal(cache, want)


@gpu
def test_streams_and_graphs():
    """Fork, copies and release on a side stream, and captured and replayed."""
    g = np.random.default_rng(0)
    B, R, bs, cols, n = 6, 10, 8, 12, 200
    seq = g.integers(1, 60, B)
    held = -(-seq // bs)
    table = g.permutation(n)[:B * cols].reshape(B, cols)
    parents = g.integers(0, B, R)
    free = np.setdiff1d(np.arange(n), table)
    want = fork_reference(table, held, seq, parents, free, 0, bs, cols)
    cache0 = torch.randn((n, bs, 1, 64), device="cuda")
    moved = cache0.clone()
    for a, b in zip(want[4], want[5]):
        if a >= 0:
            moved[b] = cache0[a]
    rel = reclaim_reference(want[0], want[1], want[2], n, [], bs, cols)
    args = [dev(x) for x in (table, held, seq, parents, free, [0])]
    cache = cache0.clone()
    out = torch.empty((R, cols), dtype=torch.int32, device="cuda")
    with paged(R, bs, cols) as p:
        def step(stream=None):
            got = p.fork(*args, out, stream=stream)
            p.copy_blocks([cache], got[3], got[4], stream=stream)
            return got + tuple(p.release(out, got[0], got[1], n, stream=stream))

        def check(got):
            torch.cuda.synchronize()
            p.check_errors()
            np.testing.assert_array_equal(out.cpu(), rel[0])
            np.testing.assert_array_equal(got[7].cpu(), rel[2])
            assert got[8].item() == rel[3] and torch.equal(cache, moved)
            cache.copy_(cache0)
            out.zero_()
            torch.cuda.synchronize()

        torch.cuda.synchronize()
        check(step(torch.cuda.Stream()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for _ in range(2):
            graph.replay()
            check(got)


@gpu
def test_refusals():
    from device_token_sampling_gb300 import VtError
    t = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    two, one = dev([0, 0]), dev([0])
    with paged(2, 16, 4) as p:
        for bad in (lambda: p.fork(t, two, two, two, two, one, t[:1]),
                    lambda: p.fork(t, two, two.long(), two, two, one, t.clone()),
                    lambda: p.fork(t, one, two, two, two, one, t.clone()),
                    lambda: p.fork(t[:, :3], two, two, two, two, one, t.clone()),
                    lambda: p.fork(t.cpu(), two, two, two, two, one, t.clone()),
                    lambda: p.release(t, two, two, 0),
                    lambda: p.release(t, one, two, 8),
                    lambda: p.release(t, two, two, 8, out=(two.clone(), dev([0] * 7), one)),
                    lambda: p.compact(t, two, two, 8, out_table=t[:, :2]),
                    lambda: p.copy_blocks([t, t[:1]], two, two),
                    lambda: p.copy_blocks([t[:, ::2]], two, two),
                    lambda: p.copy_blocks([t.cpu()], two, two),
                    lambda: p.copy_blocks([t], two, one),
                    lambda: p.copy_blocks([t[0]], two, two)):
            with pytest.raises(ValueError):
                bad()
        for bad in (lambda: p.fork(t, two, two, two, two, one, t),
                    lambda: p.fork(t, two, two, dev([0, 0, 0]), two, one,
                                   torch.zeros((3, 4), dtype=torch.int32, device="cuda")),
                    lambda: p.fork(t, two, two, two, two, one, t.clone(),
                                   out=(two, dev([0, 0]), dev([0]), dev([0, 0]), dev([0, 0]),
                                        dev([0, 0]))),
                    lambda: p.release(t, two, two, (1 << 24) + 1,
                                      out=(dev([0, 0]), torch.empty((1 << 24) + 1,
                                                                    dtype=torch.int32,
                                                                    device="cuda"), one)),
                    lambda: p.release(t, two, two, 8, out=(two, dev([0] * 8), one))):
            with pytest.raises(VtError):
                bad()
