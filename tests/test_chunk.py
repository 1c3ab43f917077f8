"""PagedBatch.chunk_attention against a plain implementation in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from pagedlib import chunk_reference

gpu = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def batch(n, total, hq, hkv, d, bs, dtype, seed=0, spare=3, heads_first=False, q_scale=1.5):
    """Inputs of requests with n new of total tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    n, total = np.asarray(n), np.asarray(total)
    blocks = -(-np.maximum(total, 0) // bs)
    cols, n_cache = max(1, int(blocks.max())), int(blocks.sum()) + spare
    ids = rng.permutation(n_cache)
    table = np.full((len(n), cols), -1)
    at = 0
    for r, m in enumerate(blocks):
        table[r, :m] = ids[at:at + m]
        at += m
    shape = (n_cache, hkv, bs, d) if heads_first else (n_cache, bs, hkv, d)
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    if heads_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    q = (torch.randn((int(n.sum()), hq, d), generator=g, device="cuda") * q_scale).to(dtype)
    starts = np.concatenate([[0], np.cumsum(n)])
    return dict(q=q, starts=dev(starts), k_cache=k, v_cache=v, table=dev(table),
                seq_lens=dev(total))


def handle(x, bs, hkv=None):
    from device_token_sampling_gb300 import PagedBatch
    return PagedBatch(max_batch=x["seq_lens"].shape[0], block_size=bs,
                      max_blocks=x["table"].shape[1], q_heads=x["q"].shape[1],
                      kv_heads=x["k_cache"].shape[2], head_dim=x["q"].shape[2])


def compare(got, x, bs, scale):
    out, lse = got
    want, wlse, b_out, b_lse = chunk_reference(x["q"], x["starts"], x["k_cache"], x["v_cache"],
                                               x["table"], x["seq_lens"], bs, scale)
    T = want.shape[0]
    assert torch.isfinite(out[:T].float()).all()
    worst = ((out[:T].double() - want).abs() / b_out.clamp(min=1e-30)).max().item() if T else 0
    assert worst <= 1, f"out {worst:.2f} of its bound"
    empty = torch.isinf(wlse)
    assert torch.equal(torch.isinf(lse[:T]), empty)
    d = ((lse[:T].double() - wlse).abs() / b_lse.clamp(min=1e-30))[~empty]
    assert d.numel() == 0 or d.max().item() <= 1, f"lse {d.max().item():.2f} of its bound"
    assert (out[:T][empty] == 0).all()


def run(x, bs, scale=None):
    s = x["q"].shape[2] ** -0.5 if scale is None else scale
    with handle(x, bs) as p:
        got = p.chunk_attention(**x, scale=scale)
        p.check_errors()
    compare(got, x, bs, s)
    return got


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [1, 4, 8, 16, 64, 128, 256])
def test_block_sizes(bs, d, dtype):
    run(batch([1, 3, 17, 40], [1, 130, 129, 300], 8, 2, d, bs, dtype, seed=bs), bs)


@gpu
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (7, 1), (28, 4), (16, 2), (5, 5), (64, 1),
                                    (130, 1), (300, 1)])
def test_heads(hq, hkv):
    """Groups of every size, also of more heads than a tile has rows."""
    run(batch([1, 9, 33], [200, 9, 161], hq, hkv, 64, 16, torch.bfloat16, seed=hq), 16)


@gpu
@pytest.mark.parametrize("n,ctx", [
    ([1], [0]), ([1], [127]), ([1], [128]), ([2], [127]), ([128], [0]), ([129], [0]),
    ([127], [1]), ([256, 1], [0, 500]), ([300], [700]), ([1000], [0]), ([1, 2, 600, 5], [5, 0, 3, 900]),
    ([1] * 100, list(range(100))), ([513], [2000]), ([64], [64])])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(n, ctx, d):
    run(batch(n, np.add(n, ctx), 8, 2, d, 16, torch.bfloat16, seed=len(n)), 16)


@gpu
def test_one_long_request_among_short_ones():
    n = [1, 1, 700, 1, 2]
    run(batch(n, [1, 9000, 8000, 40, 2], 4, 1, 128, 64, torch.bfloat16), 64)


@gpu
@pytest.mark.parametrize("n,ctx,hq,hkv", [
    ([2048], [0], 16, 8), ([500, 700, 3], [0, 40, 900], 32, 8),       # whole units, several rounds
    ([5] * 20, [2000] * 20, 32, 8), ([1, 2, 3], [7000, 9000, 1], 16, 4),  # units cut into shares
    ([1500, 2900, 40], [900, 0, 4000], 16, 4)])                       # whole rounds and shares
def test_units_whole_and_cut(n, ctx, hq, hkv):
    run(batch(n, np.add(n, ctx), hq, hkv, 64, 64, torch.bfloat16, seed=hq), 64)


@gpu
def test_many_requests():
    g = np.random.default_rng(3)
    n = g.integers(0, 6, 1500)
    total = n + g.integers(0, 90, 1500)
    run(batch(n, total, 4, 2, 64, 16, torch.bfloat16), 16)


@gpu
def test_requests_without_tokens_and_rows_without_positions():
    """n = 0, and more new tokens than the request has: those before position 0 see nothing."""
    x = batch([3, 0, 5, 4, 0], [3, 40, 2, 0, 0], 4, 2, 64, 16, torch.bfloat16)
    out, lse = run(x, 16)
    assert (out[3:6] == 0).all() and torch.isinf(lse[3:6]).all()      # 5 new of 2
    assert (out[8:12] == 0).all() and torch.isinf(lse[8:12]).all()    # 4 new of 0
    x["seq_lens"][2] = -7
    out, lse = run(x, 16)
    assert (out[3:8] == 0).all() and torch.isinf(lse[3:8]).all()


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_rows_behind_the_last_request_are_left_alone(bs):
    x = batch([3, 2], [30, 50], 4, 2, 64, bs, torch.bfloat16)
    x["q"] = torch.cat([x["q"], torch.full_like(x["q"], float("nan"))])
    out = torch.full_like(x["q"], 7.0)
    lse = torch.full(x["q"].shape[:2], 9.0, device="cuda")
    with handle(x, bs) as p:
        p.chunk_attention(**x, out=out, lse=lse)
        p.check_errors()
    compare((out, lse), x, bs, 64 ** -0.5)
    assert (out[5:] == 7).all() and (lse[5:] == 9).all()


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_starts_that_are_no_rows(bs):
    """Decreasing starts and starts past q: the request is left out and reported."""
    from device_token_sampling_gb300 import VtError
    x = batch([3, 2, 4], [30, 50, 20], 4, 2, 64, bs, torch.bfloat16)
    for starts, fine in (([0, 3, 2, 9], [(0, 3)]), ([0, 3, 5, 10], [(0, 3), (3, 5)]),
                         ([-1, 3, 5, 9], [(3, 5), (5, 9)])):
        y = dict(x, starts=dev(starts))
        out = torch.full_like(x["q"], 7.0)
        lse = torch.zeros(x["q"].shape[:2], device="cuda")
        with handle(x, bs) as p:
            p.chunk_attention(**y, out=out, lse=lse)
            with pytest.raises(VtError, match="starts"):
                p.check_errors()
            want, _ = p.chunk_attention(**x)
            p.check_errors()
        # (starts[1] = 3 to 9 where the middle request is out: its rows are another's too)
        if starts[2] != 2:
            for a, b in fine:
                assert torch.equal(out[a:b], want[a:b])


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_lengths_past_the_tables_columns(bs):
    """Cut at the table: later rows see all of it."""
    x = batch([5], [64], 4, 2, 64, bs, torch.bfloat16)
    x["seq_lens"][0] = 66
    run(x, bs)
    x["table"] = x["table"][:, :32 // bs]
    run(x, bs)


@gpu
@pytest.mark.parametrize("bs", [4, 16, 64])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_blocks_outside_the_cache(bs, bad):
    """Their tokens are left out, and reported."""
    from device_token_sampling_gb300 import VtError
    x = batch([3, 200], [150, 400], 4, 2, 64, bs, torch.bfloat16)
    x["table"][0, 64 // bs] = bad
    x["table"][1, 192 // bs] = bad
    with handle(x, bs) as p:
        got = p.chunk_attention(**x)
        with pytest.raises(VtError, match="outside the cache"):
            p.check_errors()
        p.check_errors()
    compare(got, x, bs, 64 ** -0.5)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [4, 16, 128])
def test_values_that_are_not_finite(bs, dtype):
    """At positions that a row does not see they do not reach it: behind a request's end, and
    in the tokens of the chunk behind the row."""
    n, total = [40, 3, 1, 150], [100, 131, 77, 150]
    x = batch(n, total, 4, 2, 64, bs, dtype)
    clean = {k: v.clone() for k, v in x.items()}
    inf, nan = float("inf"), float("nan")

    def at(b, j):
        return int(x["table"][b, j // bs]), j % bs

    poisoned = {0: 90, 1: 130, 3: 60}        # visible to the rows from that position on
    for b, j in poisoned.items():
        i, o = at(b, j)
        x["v_cache"][i, o, :, ::3] = nan
        x["v_cache"][i, o, 0, 1] = inf
        x["v_cache"][i, o, 1, 2] = -inf
    for b in range(4):                       # the rest of the last blocks
        i, o = at(b, total[b] - 1)
        x["k_cache"][i, o + 1:] = nan
        x["v_cache"][i, o + 1:] = nan
    with handle(x, bs) as p:
        out, lse = p.chunk_attention(**x)
        want, wlse = p.chunk_attention(**clean)
        p.check_errors()
    s0 = 0
    for b, (m, t) in enumerate(zip(n, total)):
        sees = max(0, m - (t - poisoned[b])) if b in poisoned else m
        assert torch.equal(out[s0:s0 + sees], want[s0:s0 + sees]), b
        if sees < m:
            o = out[s0 + sees:s0 + m].float()
            assert torch.isnan(o[:, :, ::3]).all()
            assert torch.isinf(o[:, :2, 1]).all() and (o[:, :2, 1] > 0).all()
            assert (o[:, 2:, 2] == -inf).all()
            other = [c for c in range(64) if c % 3 and c > 2]
            err = (o[:, :, other] - want[s0 + sees:s0 + m][:, :, other].float()).abs().max()
            assert err <= 2 ** -5
        assert torch.equal(lse[s0:s0 + m], wlse[s0:s0 + m])
        s0 += m


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_scores_that_are_not_finite(bs):
    """A NaN key makes the rows that see it NaN, and no others."""
    x = batch([50], [90], 4, 2, 64, bs, torch.bfloat16)
    want, _ = run(x, bs)
    x["k_cache"][int(x["table"][0, 60 // bs]), 60 % bs, 1] = float("nan")
    with handle(x, bs) as p:
        out, lse = p.chunk_attention(**x)
    assert torch.equal(out[:20], want[:20]) and torch.equal(out[:, :2], want[:, :2])
    assert torch.isnan(out[20:, 2:].float()).all() and torch.isnan(lse[20:, 2:]).all()


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-3, 3.0])
@pytest.mark.parametrize("bs", [4, 16])
def test_scales(scale, bs):
    run(batch([5, 130], [70, 300], 4, 2, 64, bs, torch.bfloat16), bs, scale=scale)


@gpu
def test_growing_scores():
    """Each key longer than the last, so that the running maximum grows with every tile."""
    x = batch([3, 300], [900, 1300], 4, 2, 128, 16, torch.bfloat16)
    x["q"] = x["q"].abs()
    for b in range(2):
        t = int(x["seq_lens"][b])
        for j in range(0, t, 16):
            x["k_cache"][int(x["table"][b, j // 16])] = (
                x["k_cache"][int(x["table"][b, j // 16])].abs() * (0.02 + 0.5 * j / t))
    run(x, 16)


@gpu
@pytest.mark.parametrize("bs", [4, 32])
def test_strides(bs):
    """Heads before tokens in the cache, keys and values side by side, q as a part of a
    projection, a table that is a slice of a wider one."""
    x = batch([4, 140], [80, 333], 8, 2, 64, bs, torch.float16, heads_first=True)
    q = torch.randn((144, 12, 64), device="cuda").half()
    x["q"] = q[:, 2:10]
    wide = torch.full((2, x["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :x["table"].shape[1]] = x["table"]
    x["table"] = wide[:, :x["table"].shape[1]]
    run(x, bs)
    both = torch.randn((x["k_cache"].shape[0], 2, bs, 2, 64), device="cuda").half()
    x["k_cache"], x["v_cache"] = both[:, 0], both[:, 1]
    run(x, bs)


@gpu
def test_equal_to_single_tokens():
    """One token a request: the same inputs through ``attention``, within both bounds."""
    x = batch([1] * 20, list(range(50, 250, 10)), 8, 2, 128, 16, torch.bfloat16)
    with handle(x, 16) as p:
        a, la = p.chunk_attention(**x)
        b, lb = p.attention(x["q"], x["k_cache"], x["v_cache"], x["table"], x["seq_lens"])
        p.check_errors()
    compare((a, la), x, 16, 128 ** -0.5)
    compare((b, lb), x, 16, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("bs", [1, 2, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_small_blocks(bs, d):
    """Several copies a lane fetch a tile; blocks outside the cache inside it."""
    from device_token_sampling_gb300 import VtError
    x = batch([3, 150, 1], [700, 1000, 129], 8, 2, d, bs, torch.bfloat16, seed=bs)
    run(x, bs)
    bad = [5, 64 // bs, 700 // bs - 1]
    x["table"][0, bad] = torch.tensor([-1, 1 << 20, -5], dtype=torch.int32, device="cuda")
    with handle(x, bs) as p:
        out, lse = p.chunk_attention(**x)
        with pytest.raises(VtError, match="block"):
            p.check_errors()
    # the same without those tokens
    y = dict(x)
    keep = [j for j in range(700) if j // bs not in bad]
    rows = x["table"][0, torch.tensor(keep, device="cuda") // bs].long()
    at = torch.tensor(keep, device="cuda") % bs
    n = len(keep)
    one = dict(q=x["q"][2:3], starts=dev([0, 1]), k_cache=x["k_cache"][rows, at][:, None],
               v_cache=x["v_cache"][rows, at][:, None], table=dev(np.arange(n)[None]),
               seq_lens=dev([n]))
    compare((out[2:3], lse[2:3]), one, 1, d ** -0.5)


def spread(x):
    """One kv head for all, a stride of 0: what no tensor map holds."""
    x.update({k: x[k][:, :, :1].expand_as(x[k]) for k in ("k_cache", "v_cache")})
    return x


@gpu
@pytest.mark.parametrize("bs", [1, 16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_row_by_row(bs, d, dtype):
    run(spread(batch([1, 3, 40, 0, 5], [130, 700, 40, 9, 2], 8, 2, d, bs, dtype, seed=bs)), bs)
    run(spread(batch([20], [333], 28, 4, d, bs, dtype)), bs, scale=-0.2)


@gpu
def test_row_by_row_of_bad_blocks_and_values():
    """Blocks outside the cache are left out and reported; values that are not finite reach the
    rows that see them only; rows behind the last request stay."""
    from device_token_sampling_gb300 import VtError
    bs = 16
    x = batch([40, 3], [100, 131], 4, 2, 64, bs, torch.bfloat16)
    v = x["v_cache"].clone()
    v[int(x["table"][0, 5]), 10] = float("nan")          # token 90 of the first
    v[int(x["table"][1, 8]), 3:] = float("inf")          # behind the second's end
    y = spread(dict(x, v_cache=v))
    want, _ = run(spread(x), bs)
    y["q"] = torch.cat([x["q"], torch.full_like(x["q"], float("nan"))])
    out = torch.full_like(y["q"], 7.0)
    with handle(x, bs) as p:
        p.chunk_attention(**y, out=out)
        p.check_errors()
        assert torch.equal(out[:30], want[:30]) and torch.equal(out[40:43], want[40:])
        assert torch.isnan(out[30:40].float()).all() and (out[43:] == 7).all()
        y = dict(x, table=x["table"].clone())
        y["table"][1, 2] = 1 << 20
        out, _ = p.chunk_attention(**y)
        with pytest.raises(VtError, match="block"):
            p.check_errors()
    assert torch.equal(out[:40], want[:40]) and torch.isfinite(out.float()).all()
    assert not torch.equal(out[40:], want[40:])


@gpu
def test_far_blocks():
    """A cache past 2^31 elements."""
    bs, hkv, d = 64, 8, 128
    n_cache = (1 << 31) // (bs * hkv * d) + 40
    k = torch.zeros((n_cache, bs, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x = batch([3, 70], [200, 500], 16, hkv, d, bs, torch.bfloat16)
    m = x["k_cache"].shape[0]
    k[-m:], v[-m:] = x["k_cache"], x["v_cache"]
    with handle(x, bs) as p:
        want = p.chunk_attention(**x)
        y = dict(x, k_cache=k, v_cache=v, table=torch.where(x["table"] >= 0,
                                                            x["table"] + (n_cache - m), -1))
        got = p.chunk_attention(**y)
        p.check_errors()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_same_results_every_time():
    x = batch([5, 1, 260, 3], [3000, 70, 900, 2500], 8, 2, 128, 16, torch.bfloat16)
    with handle(x, 16) as p:
        first = p.chunk_attention(**x)
        for _ in range(5):
            again = p.chunk_attention(**x)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@gpu
def test_streams_and_graphs():
    """A side stream, and a captured call replayed on new lengths and rows."""
    x = batch([3, 4, 250], [40, 700, 300], 8, 2, 64, 16, torch.bfloat16, seed=1)
    y = batch([250, 3, 4], [300, 40, 700], 8, 2, 64, 16, torch.bfloat16, seed=2)
    with handle(x, 16) as p:
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = p.chunk_attention(**x, stream=side)
        side.synchronize()
        compare(got, x, 16, 64 ** -0.5)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = p.chunk_attention(**x)
        for k in x:
            x[k].copy_(y[k])
        for _ in range(2):
            got[0].zero_()
            graph.replay()
            torch.cuda.synchronize()
            compare(got, x, 16, 64 ** -0.5)
        p.check_errors()


@gpu
def test_two_handles_at_once():
    xs = [batch([3, 4, 250], [40, 700, 300], 8, 2, 64, 16, torch.bfloat16, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in xs]
    handles = [handle(x, 16) for x in xs]
    torch.cuda.synchronize()
    got = [[] for _ in xs]
    for _ in range(8):
        for i, (p, x, s) in enumerate(zip(handles, xs, streams)):
            got[i].append(p.chunk_attention(**x, stream=s))
    torch.cuda.synchronize()
    for i, p in enumerate(handles):
        p.check_errors()
        compare(got[i][0], xs[i], 16, 64 ** -0.5)
        for g in got[i][1:]:
            assert torch.equal(g[0], got[i][0][0])
        p.close()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_one_query_over_all_ctas(dtype):
    """One request of few rows and a long context: split over every CTA, joined from 64 parts."""
    for n, total in ((1, 70000), (5, 40001), (40, 33000)):
        run(batch([n], [total], 4, 1, 128, 64, dtype, seed=n), 64)


@gpu
def test_far_rows():
    """Query rows and results past 2^31 elements, starts that do not begin at 0."""
    bs, hq, T = 16, 32, 700_000
    x = batch([3, 200], [90, 333], hq, 8, 128, bs, torch.bfloat16)
    with handle(x, bs) as p:
        want, wlse = p.chunk_attention(**x)
        q = torch.empty((T, hq, 128), dtype=torch.bfloat16, device="cuda")
        q[-203:] = x["q"]
        y = dict(x, q=q, starts=dev([T - 203, T - 200, T]))
        out, lse = torch.full_like(q, 7.0), torch.full((T, hq), 9.0, device="cuda")
        p.chunk_attention(**y, out=out, lse=lse)
        p.check_errors()
    assert torch.equal(out[-203:], want) and torch.equal(lse[-203:], wlse)
    assert (out[:T - 203] == 7).all() and (lse[:T - 203] == 9).all()


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_one_query_for_all_heads_and_rows(bs):
    """q of stride 0."""
    x = batch([3, 140], [80, 333], 8, 2, 64, bs, torch.bfloat16)
    x["q"] = x["q"][:1, :1].expand(143, 8, 64)
    run(x, bs)


@gpu
@pytest.mark.parametrize("bs", [4, 16])
def test_outputs_at_odd_addresses(bs):
    """out and lse on 16 and 4 bytes only."""
    x = batch([3, 140], [80, 333], 8, 2, 64, bs, torch.bfloat16)
    want = run(x, bs)
    out = torch.zeros(143 * 8 * 64 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(143, 8, 64)
    lse = torch.zeros(143 * 8 + 1, device="cuda")[1:].view(143, 8)
    with handle(x, bs) as p:
        p.chunk_attention(**x, out=out, lse=lse)
        p.check_errors()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@gpu
@pytest.mark.parametrize("bs", [2, 16])
def test_without_log_sums(bs):
    """out_lse NULL at the C entry; whole units and parts."""
    from device_token_sampling_gb300.sampler import DTYPE_BF16
    x = batch([3, 140], [6000, 333], 8, 2, 64, bs, torch.bfloat16)
    want = run(x, bs)
    out = torch.empty_like(x["q"])
    with handle(x, bs) as p:
        kv = x["k_cache"].stride()
        rc = p._lib.vt_paged_chunk_attention(
            p._h, DTYPE_BF16, 2, 143, x["q"].data_ptr(), 512, 64, x["starts"].data_ptr(),
            x["k_cache"].data_ptr(), x["v_cache"].data_ptr(), x["k_cache"].shape[0], kv[0], kv[1],
            kv[2], x["table"].data_ptr(), x["table"].shape[1], x["table"].shape[1],
            x["seq_lens"].data_ptr(), 0.125, out.data_ptr(), None,
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        p.check_errors()
    assert torch.equal(out, want[0])


@gpu
def test_two_graphs_of_one_handle():
    """Two captured calls share the handle's workspaces: replayed one after another."""
    xs = [batch([3, 4, 250], [40, 700, 300], 8, 2, 64, 16, torch.bfloat16, seed=1),
          batch([1, 400, 2], [3000, 700, 90], 8, 2, 64, 16, torch.bfloat16, seed=2)]
    cols = max(x["table"].shape[1] for x in xs)
    from device_token_sampling_gb300 import PagedBatch
    with PagedBatch(3, 16, cols, 8, 2, 64) as p:
        graphs, got = [], []
        for x in xs:
            p.chunk_attention(**x)
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                got.append(p.chunk_attention(**x))
        for i in (0, 1, 1, 0, 1):
            got[i][0].zero_()
            graphs[i].replay()
            compare(got[i], xs[i], 16, 64 ** -0.5)
        p.check_errors()


@gpu
def test_waits_that_run_out(monkeypatch):
    """Every wait taken as run out: the call comes back and is reported, and another handle
    attends as before."""
    from device_token_sampling_gb300 import VtError, sampler
    x = batch([3, 4, 250, 1], [4000, 700, 300, 900], 8, 2, 128, 16, torch.bfloat16)
    want, wlse = run(x, 16)
    monkeypatch.setenv("VT_FAULT_INJECT", "wait")
    broken = handle(x, 16)
    monkeypatch.delenv("VT_FAULT_INJECT")
    for _ in range(2):
        broken.chunk_attention(**x)
        with pytest.raises(VtError) as e:
            broken.check_errors()
        assert e.value.code == sampler.VT_ERR_TIMEOUT
        broken.check_errors()
    broken.close()
    out, lse = run(x, 16)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@gpu
def test_refusals():
    from device_token_sampling_gb300 import PagedBatch, VtError
    x = batch([3, 2], [30, 50], 4, 2, 64, 16, torch.bfloat16)
    with handle(x, 16) as p:
        def bad(error=ValueError, **change):
            with pytest.raises(error):
                p.chunk_attention(**{**x, **change})

        bad(q=x["q"].float())
        bad(q=x["q"][:, :3])
        bad(q=x["q"].cpu())
        bad(k_cache=x["k_cache"].half())
        bad(v_cache=x["v_cache"][:, :8])
        bad(starts=x["starts"][:2])
        bad(starts=x["starts"].long())
        bad(seq_lens=x["seq_lens"].long())
        bad(table=x["table"][:1])
        bad(out=torch.empty((5, 4, 32), dtype=torch.bfloat16, device="cuda"))
        bad(lse=torch.empty((5, 3), device="cuda"))
        bad(VtError, scale=math.inf)
        odd = torch.zeros(x["q"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:]
        bad(VtError, q=odd.view_as(x["q"]))
        out, lse = p.chunk_attention(**{**x, "q": x["q"][:0]})
        assert out.shape == (0, 4, 64)
    with PagedBatch(1, 16, 4, 4, 2, 64) as p:
        bad(VtError)
    with PagedBatch(2, 16, 4) as p:
        bad()
