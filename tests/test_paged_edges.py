"""The paged batch where blocks run short, requests share little, or values are not numbers."""
from __future__ import annotations

import numpy as np
import pytest

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
