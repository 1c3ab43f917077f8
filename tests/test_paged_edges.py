"""The paged batch where blocks run short, requests share little, or values are not numbers."""
from __future__ import annotations

import numpy as np
import pytest

from pagedlib import attention_reference
from test_paged import BF, HF, make_attention

torch = pytest.importorskip("torch")


# ---- refused requests ----------------------------------------------------------------------------

def admitted(needs, free):
    """Which requests get their blocks, in request order: what is left of the free list after those
    before it, and a refused request uses none."""
    left, ok = free, []
    for n in needs:
        ok.append(n <= left)
        left -= n if n <= left else 0
    return np.array(ok), left


def test_admitted_by_hand():
    assert admitted([4, 40, 2], 10)[0].tolist() == [True, False, True]
    assert admitted([11, 10, 1, 0], 10)[0].tolist() == [False, True, False, True]


def build(needs, n_free, cursor=0, held=None, bs=4):
    """build_tables for requests that need `needs` blocks beyond `held`, all tokens new."""
    from device_token_sampling_gb300 import PagedBatch
    needs = np.asarray(needs)
    B = len(needs)
    h = np.zeros(B, np.int64) if held is None else np.asarray(held)
    blocks = h + needs
    cols = max(1, int(blocks.max()))
    seq = np.maximum(blocks * bs - np.arange(B) % bs, 0)
    seq = np.where(blocks > 0, seq, 0)
    query = np.where(needs > 0, seq - h * bs, 0)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    free = np.arange(cursor + n_free) + 1000
    table = np.full((B, cols), -1)
    for r in range(B):
        table[r, :h[r]] = r
    table = t(table)
    with PagedBatch(max_batch=B, block_size=bs, max_blocks=cols) as p:
        out = p.build_tables(table, t(seq), t(query), t(free), t([cursor]),
                             held=None if held is None else t(h), capacity=int(query.sum()))
        p.check_errors()
    got = dict(zip(("held", "cursor", "starts", "slots", "positions", "status"),
                   (x.cpu().numpy() for x in out)), table=table.cpu().numpy())
    ok, left = admitted(needs, n_free)
    np.testing.assert_array_equal(got["status"], np.where(ok, 0, 1))
    np.testing.assert_array_equal(got["held"], np.where(ok, blocks, h))
    assert got["cursor"][0] == cursor + n_free - left
    np.testing.assert_array_equal(got["starts"], np.concatenate([[0], np.cumsum(query)]))
    at = cursor
    slots = []
    for r in range(B):
        want = np.full(cols, -1)
        want[:h[r]] = r
        if ok[r]:
            want[h[r]:blocks[r]] = free[at:at + needs[r]]
            at += needs[r]
        np.testing.assert_array_equal(got["table"][r], want, err_msg=str(r))
        pos = np.arange(seq[r] - query[r], seq[r])
        slots.append(want[pos // bs] * bs + pos % bs if ok[r] else np.full(len(pos), -1))
    np.testing.assert_array_equal(got["slots"], np.concatenate(slots))
    return got


@pytest.mark.gpu
def test_a_request_that_does_not_fit_leaves_the_blocks_to_those_behind():
    assert build([4, 40, 2], 10)["status"].tolist() == [0, 1, 0]
    assert build([11, 10, 1, 0], 10, cursor=5)["status"].tolist() == [1, 0, 1, 0]
    build([1, 3, 1], 2, held=[2, 0, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("B,most,share", [(40, 9, 0.5), (511, 30, 0.9), (513, 3, 0.2), (1500, 200, 0.6),
                                          (4000, 2, 0.99), (1025, 60, 0.0), (16384, 3, 0.7)])
@pytest.mark.parametrize("step", [False, True])
def test_free_list_shorter_than_the_requests(B, most, share, step):
    """Several batches of the scan with refusals in them, needs of 0 among them."""
    g = np.random.default_rng(B + most)
    needs = g.integers(0, most + 1, B)
    if most > 20:                              # small requests behind very large ones
        needs = np.where(g.random(B) < 0.3, needs * 5, needs // 10)
    build(needs, int(needs.sum() * share), cursor=int(g.integers(0, 9)),
          held=g.integers(0, 4, B) if step else None)


# ---- values that are not numbers where a request does not attend ---------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,hq,hkv,d,bs,prefix", [(3, 4, 2, 64, 16, 96), (40, 8, 2, 128, 16, 300),
                                                  (33, 8, 1, 64, 64, 1029), (6, 2, 2, 128, 2, 70)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_past_a_short_request_do_not_reach_it(dtype, B, hq, hkv, d, bs, prefix, bad):
    """Requests shorter than the shared prefix beside longer ones: keys and values of the prefix
    that only the longer ones attend to are not finite."""
    from device_token_sampling_gb300 import PagedBatch
    seq = np.array([prefix + 5, prefix // 2, 1, 0, prefix, prefix - 1] * 7)[:B]
    seq[2] = min(seq[2], prefix // 3)
    c = make_attention(B + d, seq, hq, hkv, d, bs, prefix, dtype)
    p = PagedBatch(B, bs, c["cols"], hq, hkv, d)
    args = (c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], prefix)
    clean = [t.clone() for t in p.attention(*args)]
    pos = prefix // 2 + 1                      # past request 1, within the longest
    where = (int(c["pre"][pos // bs]), pos % bs)
    for cache in (c["v"], c["k"]):
        cache[where] = bad
        out, lse = p.attention(*args)
        p.check_errors()
        short = c["seq"] <= pos
        want, wlse, b_out, b_lse = attention_reference(
            c["q"][short], c["k"], c["v"], c["table"][short], c["seq"][short], c["pre"], prefix, bs,
            d ** -0.5)
        assert bool(((out[short].double() - want).abs() <= b_out).all())
        some = wlse > -float("inf")
        assert bool(((lse[short].double() - wlse).abs()[some] <= b_lse[some]).all())
        assert bool((lse[short][~some] == -float("inf")).all())
        assert bool((~out[~short].isfinite()).any(-1).all())
    c["v"][where] = 1.0
    c["k"][where] = 1.0
    again, _ = p.attention(*args)
    assert torch.equal(again[c["seq"] <= pos], clean[0][c["seq"] <= pos])


# ---- a table that is part of a wider one ---------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("B,prefix", [(3, 0), (20, 32)])
def test_lengths_past_a_narrowed_table_are_cut(B, prefix):
    """A column slice of a wider table, as a contiguous table of those columns: a length past the
    slice is cut there, whatever stands behind it."""
    from device_token_sampling_gb300 import PagedBatch
    c = make_attention(5, [80 + i % 3 for i in range(B)], 8, 2, 64, 16, prefix, BF)
    narrow = c["table"][:, :4].contiguous()    # 64 tokens
    wide = torch.zeros((B + 1, 12), dtype=torch.int32, device="cuda")
    wide[:B, 3:7] = narrow
    wide[:B, 7:9] = c["table"][:, 4:6].clamp(0, c["k"].shape[0] - 1)
    # (head-room in max_blocks, so that the lengths are not cut there)
    p = PagedBatch(B, 16, 16, 8, 2, 64)
    rest = (c["seq"], c["pre"], prefix)
    want, wlse = p.attention(c["q"], c["k"], c["v"], narrow, *rest)
    got, lse = p.attention(c["q"], c["k"], c["v"], wide[:B, 3:7], *rest)
    p.check_errors()
    assert torch.equal(got, want) and torch.equal(lse, wlse)


# ---- waits ---------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out(d, monkeypatch):
    """Every wait of the shared prefix's kernel taken as run out: the call comes back and is
    reported, and another handle attends as before."""
    from device_token_sampling_gb300 import PagedBatch, VtError, sampler
    c = make_attention(17, [700 + i for i in range(40)], 8, 2, d, 16, 690, BF)
    args = (c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], 690)
    with PagedBatch(40, 16, c["cols"], 8, 2, d) as p:
        want, wlse = p.attention(*args)
        p.check_errors()
    monkeypatch.setenv("VT_FAULT_INJECT", "wait")
    broken = PagedBatch(40, 16, c["cols"], 8, 2, d)
    monkeypatch.delenv("VT_FAULT_INJECT")
    for _ in range(2):
        broken.attention(*args)
        with pytest.raises(VtError) as e:
            broken.check_errors()
        assert e.value.code == sampler.VT_ERR_TIMEOUT
        broken.check_errors()
    with PagedBatch(40, 16, c["cols"], 8, 2, d) as p:
        out, lse = p.attention(*args)
        p.check_errors()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
