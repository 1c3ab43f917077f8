"""Block tables, slot maps and attention behind a shared prefix, against plain
references; the refusals."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from pagedlib import attention_reference, tables_reference

torch = pytest.importorskip("torch")


# ---- what needs no GPU --------------------------------------------------------------------------

@pytest.mark.parametrize("field,value", [
    ("max_batch", 0), ("max_batch", 16385), ("block_size", 0), ("block_size", 24),
    ("block_size", 2048), ("max_blocks", 0), ("max_blocks", 1 << 27), ("q_heads", 7),
    ("q_heads", 2048), ("kv_heads", 0), ("kv_heads", 3), ("head_dim", 96), ("device", -1)])
def test_create_refuses(field, value):
    from device_token_sampling_gb300 import sampler
    lib = sampler.load_library()
    cfg = sampler.PagedConfig(4, 16, 8, 8, 2, 64, 0)
    setattr(cfg, field, value)
    h = ctypes.c_void_p()
    assert lib.vt_paged_create(ctypes.byref(cfg), ctypes.byref(h)) == sampler.VT_ERR_INVALID_ARG
    assert not h.value


def test_null_handle_and_pointers():
    from device_token_sampling_gb300 import sampler
    lib = sampler.load_library()
    cfg = sampler.PagedConfig(4, 16, 8, 8, 2, 64, 0)
    assert lib.vt_paged_create(ctypes.byref(cfg), None) == sampler.VT_ERR_INVALID_ARG
    assert lib.vt_paged_create(None, ctypes.byref(ctypes.c_void_p())) == sampler.VT_ERR_INVALID_ARG
    lib.vt_paged_destroy(None)
    assert lib.vt_paged_last_error(None) == b"null handle"
    assert lib.vt_paged_check_errors(None) == sampler.VT_ERR_INVALID_ARG
    n = [None] * 30
    assert lib.vt_paged_tables(None, 1, *n[:4], 0, None, 0, None, None, 8, *n[:5], 0, None,
                               None) == sampler.VT_ERR_INVALID_ARG


def test_reference_tables_by_hand():
    """The host reference itself, on a case worked out by hand: blocks of 4, one shared block."""
    t, held, cur, starts, slots, pos, st = tables_reference(
        np.full((3, 3), -7), [5, 3, 9], [2, 3, 1], [10, 11, 12], 0, None, [20], 4, 3, 7)
    assert t.tolist() == [[20, 10, -1], [20, -1, -1], [20, 11, 12]]
    assert held.tolist() == [2, 1, 3] and cur == 3 and st.tolist() == [0, 0, 0]
    assert starts.tolist() == [0, 2, 5, 6]
    assert pos.tolist() == [3, 4, 0, 1, 2, 8, -1]
    assert slots.tolist() == [83, 40, 80, 81, 82, 48, -1]


# ---- tables --------------------------------------------------------------------------------------

def _tables_case(seed, B, bs, cols, prefix, max_len, max_query, scratch, short=0, extra_cols=0):
    g = np.random.default_rng(seed)
    seq = g.integers(0, max_len + 1, B)
    query = np.minimum(g.integers(0, max_query + 1, B), seq)
    held = np.where(seq - query > 0, -(-(seq - query) // bs), 0)
    need = int((-(-seq // bs)).sum())
    free = g.permutation(1 << 20)[:max(0, need - short)].astype(np.int32)
    table = g.integers(0, 1 << 20, (B, cols + extra_cols)).astype(np.int32)
    pre = g.integers(0, 1 << 20, prefix).astype(np.int32)
    return dict(table=table, seq=seq.astype(np.int32), query=query.astype(np.int32), free=free,
                cursor=np.array([min(3, len(free))], np.int32),
                held=None if scratch else held.astype(np.int32), prefix=pre)


def _run_tables(c, bs, cols, capacity, stream=None):
    from device_token_sampling_gb300 import PagedBatch
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    table = t(c["table"])
    with PagedBatch(max_batch=max(1, len(c["seq"])), block_size=bs, max_blocks=cols) as p:
        out = p.build_tables(table, t(c["seq"]), t(c["query"]), t(c["free"]), t(c["cursor"]),
                             held=t(c["held"]), prefix_blocks=t(c["prefix"]), capacity=capacity,
                             stream=stream)
        p.check_errors()
    return [x.cpu().numpy() for x in (table,) + out]


def _check_tables(c, bs, cols, capacity):
    got = _run_tables(c, bs, cols, capacity)
    want = tables_reference(c["table"], c["seq"], c["query"], c["free"], c["cursor"][0], c["held"],
                            c["prefix"], bs, cols, capacity)
    for g, w, name in zip(got, want, ("table", "held", "cursor", "starts", "slots", "positions",
                                      "status")):
        np.testing.assert_array_equal(g.reshape(-1), np.asarray(w).reshape(-1), err_msg=name)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("B,bs,cols,prefix,max_len,max_query,scratch", [
    (1, 16, 4, 0, 1, 1, True), (1, 1, 7, 2, 7, 7, True), (3, 8, 300, 5, 2000, 2000, True),
    (64, 16, 33, 4, 512, 1, False), (511, 16, 9, 0, 140, 3, False), (513, 4, 9, 3, 36, 36, True),
    (1025, 32, 5, 1, 150, 5, False), (2000, 128, 2, 1, 250, 9, True),
    (16384, 16, 3, 1, 40, 3, False)])
def test_tables(B, bs, cols, prefix, max_len, max_query, scratch):
    c = _tables_case(B, B, bs, cols, prefix, max_len, max_query, scratch)
    total = int(c["query"].sum())
    for capacity in {total, total + 5, max(0, total - 3), 0}:
        _check_tables(c, bs, cols, capacity)


@pytest.mark.gpu
@pytest.mark.parametrize("scratch", [True, False])
def test_tables_out_of_blocks_and_bad_lengths(scratch):
    c = _tables_case(5, 200, 16, 20, 2, 300, 20, scratch, short=400)
    c["seq"][7], c["seq"][90], c["query"][11] = -1, 20 * 16 + 1, 400
    got = _check_tables(c, 16, 20, 4000)
    assert set(got[-1].tolist()) == ({0, 1, 2} if scratch else {0, 2})


@pytest.mark.gpu
def test_tables_step_out_of_blocks():
    """A decode step whose free list runs out part of the way through the requests."""
    c = _tables_case(21, 300, 4, 20, 2, 70, 6, False)
    c["free"] = c["free"][:100]
    got = _check_tables(c, 4, 20, 1200)
    assert set(got[-1].tolist()) == {0, 1}


@pytest.mark.gpu
@pytest.mark.parametrize("cursor", [-1, -2 ** 31, 10 ** 9])
def test_tables_cursor_outside(cursor):
    c = _tables_case(6, 20, 16, 20, 2, 300, 20, True)
    c["cursor"][0] = cursor
    got = _check_tables(c, 16, 20, 400)
    assert got[2][0] == cursor


@pytest.mark.gpu
def test_tables_wide_rows_empty_arrays_and_steps():
    """A table wider than max_blocks, no free list, no prefix; then twenty decode steps that
    carry held and cursor on."""
    from device_token_sampling_gb300 import PagedBatch
    c = _tables_case(8, 9, 16, 6, 0, 90, 90, True, extra_cols=3)
    c["free"] = np.zeros(0, np.int32)
    c["cursor"][0] = 0
    got = _check_tables(c, 16, 6, 900)
    assert (got[0][:, 6:] == c["table"][:, 6:]).all()
    B, bs, cols = 33, 4, 16
    free = np.random.default_rng(3).permutation(1000).astype(np.int32)
    t = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    table = torch.empty((B, cols), dtype=torch.int32, device="cuda")
    tf = t(free)
    seq = np.random.default_rng(4).integers(1, 30, B)
    with PagedBatch(max_batch=B, block_size=bs, max_blocks=cols) as p:
        held, cur, *_ = p.build_tables(table, t(seq), t(seq), tf, t([0]), capacity=int(seq.sum()))
        for _ in range(20):
            seq = seq + 1
            held, cur, starts, slots, pos, st = p.build_tables(table, t(seq), t(np.ones(B)), tf, cur,
                                                               held=held)
            tab = table.cpu().numpy()
            want = [tab[r, (seq[r] - 1) // bs] * bs + (seq[r] - 1) % bs for r in range(B)]
            np.testing.assert_array_equal(slots.cpu().numpy(), want)
        used = np.concatenate([tab[r, :-(-seq[r] // bs)] for r in range(B)])
        assert len(set(used.tolist())) == len(used) == int(cur.item())


# ---- attention -----------------------------------------------------------------------------------

def make_attention(seed, seq, hq, hkv, d, bs, prefix_len, dtype, layout="NHD", poison=True,
                   value=1.0):
    """A cache whose unused tokens hold NaN, tables whose unused entries are far outside."""
    g = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    seq = np.asarray(seq)
    B = len(seq)
    n_shared, n_pre = prefix_len // bs, -(-prefix_len // bs)
    nblk = np.maximum(-(-seq // bs), n_shared)
    cols = max(1, int(nblk.max()), n_pre) + 2
    n_cache = n_pre + int((nblk - n_shared).sum()) + 2
    ids = g.permutation(n_cache).astype(np.int32)
    pre = ids[:n_pre]
    table = np.full((B, cols), 2 ** 31 - 1, np.int32)
    at = n_pre
    for r in range(B):
        table[r, :n_shared] = -5          # positions below prefix_len go by prefix_blocks alone
        n = nblk[r] - n_shared
        table[r, n_shared:n_shared + n] = ids[at:at + n]
        at += n
    shape = (n_cache, bs, hkv, d) if layout == "NHD" else (n_cache, hkv, bs, d)
    kv = []
    for _ in range(2):
        c = (torch.randn(shape, generator=gen, device="cuda") * value).to(dtype)
        if layout == "HND":
            c = c.transpose(1, 2)
        kv.append(c)
    used = np.zeros((n_cache, bs), bool)
    for p in range(prefix_len):
        used[pre[p // bs], p % bs] = True
    for r in range(B):
        for p in range(prefix_len, seq[r]):
            used[table[r, p // bs], p % bs] = True
    if poison:
        gone = torch.from_numpy(~used).cuda()
        for c in kv:
            c[gone] = float("nan")
    q = (torch.randn((B, hq, d), generator=gen, device="cuda") * 1.5).to(dtype)
    return dict(q=q, k=kv[0], v=kv[1], table=torch.from_numpy(table).cuda(),
                seq=torch.from_numpy(seq.astype(np.int32)).cuda(),
                pre=torch.from_numpy(np.ascontiguousarray(pre)).cuda(), cols=cols)


def check_attention(c, bs, prefix_len, scale=None, max_seq_len=0, max_batch=None, paged=None,
                    **kw):
    from device_token_sampling_gb300 import PagedBatch
    B, hq, d = c["q"].shape
    hkv = c["k"].shape[2]
    p = paged or PagedBatch(max_batch=max_batch or B, block_size=bs, max_blocks=c["cols"],
                            q_heads=hq, kv_heads=hkv, head_dim=d)
    out, lse = p.attention(c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], prefix_len,
                           scale=scale, max_seq_len=max_seq_len, **kw)
    p.check_errors()
    want, wlse, b_out, b_lse = attention_reference(
        c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], prefix_len, bs,
        d ** -0.5 if scale is None else scale)
    err = (out.double() - want).abs()
    assert bool((err <= b_out).all()), (float((err - b_out).max()), float(err.max()))
    empty = wlse == -float("inf")
    assert bool((lse[empty] == -float("inf")).all())
    el = (lse.double() - wlse).abs()[~empty]
    assert bool((el <= b_lse[~empty]).all()), float(el.max())
    return out, lse


BF, HF = torch.bfloat16, torch.float16


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("seq,hq,hkv,d,bs,prefix", [
    ([1], 1, 1, 64, 16, 0),                              # one token in all
    ([1, 2, 17, 0], 4, 4, 128, 16, 0),                   # nothing shared, an empty request
    ([64, 64], 8, 2, 64, 16, 64),                        # the prefix alone
    ([65, 64, 80, 300], 8, 2, 128, 16, 64),
    ([101, 140, 90, 0, 50, 100], 14, 2, 64, 8, 100),     # ends in a block; shorter ones, empty
    ([520, 513, 700], 32, 8, 128, 32, 513),
    ([1030, 1031], 24, 1, 64, 64, 1029),                 # 24 heads on one kv head
    ([37, 38, 39], 5, 5, 128, 1, 33),                    # blocks of one token
    ([2000] * 3, 16, 8, 128, 128, 1500),
    (list(range(400, 437)), 28, 4, 64, 16, 399)])
def test_attention(dtype, seq, hq, hkv, d, bs, prefix):
    check_attention(make_attention(len(seq) + d, seq, hq, hkv, d, bs, prefix, dtype), bs, prefix)


@pytest.mark.gpu
@pytest.mark.parametrize("B,G", [(1, 1), (4, 4), (5, 3), (16, 1), (17, 1), (33, 8), (65, 4), (130, 5)])
def test_attention_row_counts(B, G):
    """Rows behind the prefix below, at and above each tile size."""
    seq = 150 + np.arange(B) % 37
    check_attention(make_attention(B * G, seq, 2 * G, 2, 128, 16, 148, BF), 16, 148)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 63, 64, 127, 128, 129, 255, 257, 640, 1000])
def test_attention_prefix_lengths(prefix):
    seq = [prefix + 1, prefix, prefix + 30, max(0, prefix - 1), prefix // 2] * 9
    check_attention(make_attention(prefix, seq, 8, 2, 64, 16, prefix, HF), 16, prefix)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_attention_strides(layout):
    """A head-major cache, queries inside a wider projection, a table with spare columns."""
    seq = [300, 170, 222, 161]
    c = make_attention(7, seq, 8, 4, 128, 16, 160, BF, layout=layout)
    wide = torch.full((4, 16, 128 + 8), float("nan"), dtype=BF, device="cuda")
    wide[:, 3:11, :128] = c["q"]
    c["q"] = wide[:, 3:11, :128]
    t = torch.full((4, c["cols"] + 5), -1, dtype=torch.int32, device="cuda")
    t[:, :c["cols"]] = c["table"]
    c["table"] = t
    check_attention(c, 16, 160)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,layout,bs,d,B,G,prefix", [
    (BF, "HND", 16, 128, 40, 4, 300), (HF, "HND", 8, 64, 70, 2, 129), (BF, "NHD", 128, 64, 33, 8, 512),
    (HF, "NHD", 256, 128, 20, 4, 700), (BF, "HND", 1024, 64, 20, 3, 1500),
    (BF, "NHD", 4, 128, 20, 4, 77), (HF, "NHD", 32, 128, 300, 5, 2000), (BF, "NHD", 64, 128, 9, 32, 65),
    (BF, "NHD", 16, 64, 129, 1, 4097), (HF, "HND", 64, 64, 18, 16, 64)])
def test_attention_many_rows(dtype, layout, bs, d, B, G, prefix):
    """More than sixteen rows behind the prefix, in both layouts, every block size's way of copying
    a tile, one and several row tiles, splits that end inside a tile and inside a block."""
    g = np.random.default_rng(B)
    seq = prefix + g.integers(-prefix // 8, 80, B)
    seq[g.integers(0, B)] = 0
    check_attention(make_attention(B + d, seq, 2 * G, 2, d, bs, prefix, dtype, layout=layout), bs,
                    prefix)


@pytest.mark.gpu
def test_attention_one_head_odd_strides():
    """Dimensions of one element, whose strides say nothing."""
    c = make_attention(15, [50], 1, 1, 64, 16, 0, BF)
    one = torch.as_strided(c["q"], (1, 1, 64), (3, 5, 1))
    k, v = (torch.as_strided(t, t.shape, (16 * 64, 64, 7, 1)) for t in (c["k"], c["v"]))
    assert torch.equal(one, c["q"]) and torch.equal(k.nan_to_num(), c["k"].nan_to_num())
    check_attention({**c, "q": one, "k": k, "v": v}, 16, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 20])
@pytest.mark.parametrize("scale", [2.0, -0.3, 0.0])
def test_attention_scales(B, scale):
    seq = [200, 150, 140] + [190 + i for i in range(B - 3)]
    check_attention(make_attention(3, seq, 8, 2, 128, 16, 130, BF), 16, 130, scale=scale)


@pytest.mark.gpu
def test_attention_far_blocks():
    """A cache past 2^31 elements: offsets of the last blocks need 64 bits."""
    n, bs, hkv, d = 3000, 1024, 8, 128      # 3.1 G elements each
    kc = torch.zeros((n, bs, hkv, d), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(16)
    pre = torch.tensor([2999, 2], dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 0, 2998 - i] for i in range(20)], dtype=torch.int32, device="cuda")
    for b in pre.tolist() + table[:, 2].tolist():
        for c in (kc, vc):
            c[b] = torch.randn((bs, hkv, d), generator=gen, device="cuda").to(BF)
    q = torch.randn((20, 16, d), generator=gen, device="cuda").to(BF)
    seq = torch.arange(20, dtype=torch.int32, device="cuda") * 40 + 2048
    check_attention(dict(q=q, k=kc, v=vc, table=table, seq=seq, pre=pre, cols=3), bs, 2048)


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [0, 1, 200, 4000])
def test_attention_length_hint(hint):
    """The bound on the lengths shapes the launch only: a wrong one changes no result."""
    c = make_attention(9, [4000, 129, 2500, 0, 900], 8, 8, 64, 16, 128, BF)
    check_attention(c, 16, 128, max_seq_len=hint)


@pytest.mark.gpu
def test_attention_scales_and_large_scores():
    """Scores in the hundreds: weights underflow, the sums stay finite; negative and zero scale."""
    for scale in (2.0, -0.3, 0.0):
        check_attention(make_attention(3, [200, 150, 140], 8, 2, 128, 16, 130, BF), 16, 130,
                        scale=scale)


@pytest.mark.gpu
def test_attention_nan_and_inf_reach_their_rows_only():
    c = make_attention(4, [90, 90, 90], 4, 2, 64, 16, 64, BF)
    clean, _ = check_attention(c, 16, 64)
    c["q"][1, 2, 5] = float("nan")
    from device_token_sampling_gb300 import PagedBatch
    with PagedBatch(3, 16, c["cols"], 4, 2, 64) as p:
        out, lse = p.attention(c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], 64)
        p.check_errors()
    bad = torch.zeros((3, 4), dtype=torch.bool, device="cuda")
    bad[1, 2] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("B", [2, 40])
def test_attention_bad_blocks_are_left_out(B):
    from device_token_sampling_gb300 import PagedBatch, VtError
    c = make_attention(11, [200 + i for i in range(B)], 8, 2, 64, 16, 96, BF)
    c["pre"][2] = -1
    c["table"][0, 8] = c["k"].shape[0]
    c["table"][1, 12] = -2 ** 31
    p = PagedBatch(B, 16, c["cols"], 8, 2, 64)
    with pytest.raises(VtError, match="outside the cache"):
        check_attention(c, 16, 96, paged=p)
    out, lse = p.attention(c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], 96)
    want, wlse, b_out, b_lse = attention_reference(c["q"], c["k"], c["v"], c["table"], c["seq"],
                                                   c["pre"], 96, 16, 64 ** -0.5)
    assert bool(((out.double() - want).abs() <= b_out).all())
    assert bool(((lse.double() - wlse).abs() <= b_lse).all())
    with pytest.raises(VtError):
        p.check_errors()
    p.check_errors()  # reported once


@pytest.mark.gpu
def test_attention_repeats_streams_and_graph():
    """The same bits again, on another stream, and from a captured graph with new inputs."""
    from device_token_sampling_gb300 import PagedBatch
    c = make_attention(12, [400 + 7 * i for i in range(24)], 8, 2, 128, 16, 384, BF)
    p = PagedBatch(24, 16, c["cols"], 8, 2, 128)
    args = (c["q"], c["k"], c["v"], c["table"], c["seq"], c["pre"], 384)
    out, lse = p.attention(*args)
    for _ in range(3):
        o2, l2 = p.attention(*args)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, l2 = p.attention(*args, stream=s)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.attention(*args, out=o3, lse=l3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o3, out) and torch.equal(l3, lse)
    c["q"].copy_(c["q"].flip(0))
    c["seq"].sub_(5)
    g.replay()
    torch.cuda.synchronize()
    o4, l4 = p.attention(*args)
    assert torch.equal(o3, o4) and torch.equal(l3, l4) and not torch.equal(o3, out)


@pytest.mark.gpu
def test_refusals():
    from device_token_sampling_gb300 import PagedBatch, VtError, sampler
    c = make_attention(13, [40, 50], 4, 2, 64, 16, 32, BF)
    p = PagedBatch(2, 16, c["cols"], 4, 2, 64)
    ok = dict(q=c["q"], k_cache=c["k"], v_cache=c["v"], table=c["table"], seq_lens=c["seq"],
              prefix_blocks=c["pre"], prefix_len=32)
    p.attention(**ok)
    for bad in (dict(q=c["q"].float()), dict(q=c["q"][:, :3]), dict(q=c["q"].cpu()),
                dict(k_cache=c["k"].half()), dict(k_cache=c["k"][:, :8]),
                dict(v_cache=c["v"].transpose(1, 2).contiguous().transpose(1, 2)),
                dict(table=c["table"].long()), dict(seq_lens=c["seq"][:1]),
                dict(seq_lens=c["seq"].long()), dict(prefix_blocks=None),
                dict(prefix_blocks=c["pre"][:1]), dict(max_seq_len=10 ** 6),
                dict(out=torch.empty(2, 4, 64, device="cuda")),
                dict(lse=torch.empty(2, 3, device="cuda"))):
        with pytest.raises(ValueError):
            p.attention(**{**ok, **bad})
    odd = torch.zeros((2, 4, 65), dtype=BF, device="cuda")[:, :, 1:]
    for bad in (dict(q=odd), dict(prefix_len=-1), dict(scale=float("nan")), dict(max_seq_len=-1)):
        with pytest.raises(VtError) as e:
            p.attention(**{**ok, **bad})
        assert e.value.code == sampler.VT_ERR_INVALID_ARG
    three = make_attention(14, [40, 50, 60], 4, 2, 64, 16, 32, BF)
    with pytest.raises(VtError) as e:
        p.attention(three["q"], c["k"], c["v"], three["table"], three["seq"], c["pre"], 32)
    assert e.value.code == sampler.VT_ERR_CAPACITY
    with pytest.raises(ValueError):
        PagedBatch(2, 16, 8).attention(**ok)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    t = torch.empty((2, c["cols"]), dtype=torch.int32, device="cuda")
    good = dict(table=t, seq_lens=i32(3, 4), query_lens=i32(1, 1), free_blocks=i32(5, 6, 7),
                cursor=i32(0))
    p.build_tables(**good)
    held, cur = i32(0, 0), good["cursor"]
    full = p.build_tables(**good)
    for bad in (dict(table=t[:, :-1]), dict(table=t.long()), dict(query_lens=i32(1)),
                dict(cursor=i32(0, 0)), dict(capacity=-1), dict(free_blocks=i32(1).cpu()),
                dict(held=i32(0)), dict(out=full[:5] + (held,) + full)):
        with pytest.raises(ValueError):
            if "out" in bad:
                p.build_tables(**good, out=(held.long(),) + full[1:])
            p.build_tables(**{**good, **bad})
    for bad in (dict(held=held, out=(held,) + full[1:]),
                dict(out=(full[0], cur) + full[2:])):
        with pytest.raises(VtError) as e:
            p.build_tables(**{**good, **bad})
        assert e.value.code == sampler.VT_ERR_INVALID_ARG
