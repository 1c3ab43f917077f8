"""Cases for the operators of the parallel-sampling loop.

Three operators, named by a case's ``op``:

* ``given``  -- ``Sampler.sample_given``: temperature, min-p, top-k and top-p, then draws
  from given uniform numbers by inversion in vocabulary order;
* ``tables`` -- ``PagedBatch.build_tables``: block tables and slot maps from request lengths;
* ``prefix`` -- ``PagedBatch.attention``: one query token a request over a paged cache whose
  first tokens all requests share.

``run`` with ``own`` false computes them in elementary torch operations; with ``own`` true it
makes the calls of this package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# ---------------------------------------------------------------------------- the cases

def listed():
    return [
        # the first step of 16 continuations of one prompt: one row, 16 draws
        dict(name="given_fork16", op="given", B=1, V=151936, pad=0, dtype="bf16", draws=16,
             kind="topp"),
        # an odd vocabulary in rows that no vector load is aligned to
        dict(name="given_odd", op="given", B=5, V=32003, pad=0, dtype="f32", draws=3,
             kind="mixed"),
        # the package's b32 workload: T = 1, top-k 20, top-p 0.95
        dict(name="given_b32", op="given", B=32, V=151936, pad=0, dtype="bf16", draws=1,
             kind="b32"),
        # its b256 workload: greedy, top-k, top-p and all filters, by rows
        dict(name="given_b256", op="given", B=256, V=151936, pad=0, dtype="bf16", draws=1,
             kind="mixed"),
        # its large workload's shape, every kind of row (unfiltered ones too)
        dict(name="given_large", op="given", B=1024, V=248320, pad=0, dtype="f32", draws=1,
             kind="open"),
        # one decode step: each of 256 requests gets one token, one in 16 a new block
        dict(name="tables_decode", op="tables", B=256, block=16, cols=1024, prefix=64,
             max_len=8192, max_query=1, scratch=False),
        # prompts of ragged lengths coming in behind a shared system prompt
        dict(name="tables_prefill", op="tables", B=61, block=64, cols=160, prefix=16,
             max_len=8000, max_query=8000, scratch=True),
        # a whole serving state laid out anew
        dict(name="tables_large", op="tables", B=2048, block=16, cols=512, prefix=0,
             max_len=8192, max_query=8192, scratch=True),
        # four continuations of a short prompt: latency
        dict(name="prefix_small", op="prefix", B=4, hq=32, hkv=8, d=128, block=16, prefix=512,
             max_own=64, dtype="bf16"),
        # an odd batch, groups of 7 heads, a prefix that ends inside a block
        dict(name="prefix_odd", op="prefix", B=37, hq=28, hkv=4, d=64, block=16, prefix=3001,
             max_own=300, dtype="f16"),
        # an ordinary decode batch behind a long shared prompt
        dict(name="prefix_b64", op="prefix", B=64, hq=32, hkv=8, d=128, block=64, prefix=8192,
             max_own=512, dtype="bf16"),
        # many continuations of a long document
        dict(name="prefix_b256", op="prefix", B=256, hq=32, hkv=8, d=128, block=64,
             prefix=16384, max_own=1024, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["given", "tables", "prefix"])
    if op == "given":
        V = _log_int(rng, 1000, 248320)
        B = _log_int(rng, 1, min(1024, max(1, 250_000_000 // V)))
        return dict(op=op, B=B, V=V, pad=rng.choice([0, 0, 8, 13]),
                    dtype=rng.choice(["bf16", "f32"]), draws=rng.choice([1, 1, 2, 5, 16]),
                    kind=rng.choice(["topp", "b32", "mixed", "open"]))
    if op == "tables":
        block = rng.choice([8, 16, 32, 64, 128])
        B = _log_int(rng, 1, 2048)
        max_len = _log_int(rng, 16, min(65536, 16_000_000 // B))
        prefix = rng.randrange(0, max(1, max_len // (2 * block)) + 1)
        scratch = rng.random() < 0.5
        query = max_len if scratch else rng.choice([1, 1, 2, 5])
        cols = max(prefix, -(-max_len // block)) + rng.randrange(1, 9)
        return dict(op=op, B=B, block=block, cols=cols, prefix=prefix, max_len=max_len,
                    max_query=query, scratch=scratch)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    B = _log_int(rng, 1, 256)
    prefix = _log_int(rng, 1, min(32768, max(64, 130_000_000 // (B * hq))))
    return dict(op=op, B=B, hq=hq, hkv=hkv, d=d, block=rng.choice([16, 32, 64, 128]),
                prefix=prefix, max_own=_log_int(rng, 1, 1024),
                dtype=rng.choice(["bf16", "f16"]))


_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _given_params(case, seed):
    """Per-row parameters: numpy arrays (T, top_k, top_p, min_p)."""
    g = np.random.default_rng(seed)
    B, kind = case["B"], case["kind"]
    T = np.ones(B, np.float32)
    k = np.zeros(B, np.int32)
    p = np.ones(B, np.float32)
    mp = np.zeros(B, np.float32)
    if kind == "topp":
        T[:] = g.uniform(0.6, 1.0, B)
        p[:] = g.uniform(0.9, 0.98, B)
    elif kind == "b32":
        k[:] = 20
        p[:] = 0.95
    else:
        T[:] = g.uniform(0.3, 1.5, B)
        c = np.arange(B) % (4 if kind == "mixed" else 6)
        if B < 6:
            c = (c + seed) % (4 if kind == "mixed" else 6)
        T[c == 0] = 0.0                                  # greedy
        k[c == 1] = g.integers(1, 1025, B)[c == 1]
        p[c == 2] = g.uniform(0.5, 0.99, B).astype(np.float32)[c == 2]
        k[c == 3], p[c == 3], mp[c == 3] = 50, 0.95, 0.05
        # c == 4: no filter; c == 5: min-p alone
        mp[c == 5] = g.uniform(0.001, 0.2, B).astype(np.float32)[c == 5]
    return T, k, p, mp


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    g = np.random.default_rng([seed, 7])
    op, B = case["op"], case["B"]
    if op == "given":
        V = case["V"]
        ld = V + case["pad"]
        dt = _DT[case["dtype"]]
        x = torch.empty((B, ld), dtype=dt, device=dev)
        for r0 in range(0, B, 128):  # N(0, 1.5) with 8 columns a row raised by U(8, 12)
            r1 = min(B, r0 + 128)
            z = torch.randn((r1 - r0, ld), generator=gen, device=dev) * 1.5
            at = torch.randint(0, V, (r1 - r0, 8), generator=gen, device=dev)
            up = 8 + 4 * torch.rand((r1 - r0, 8), generator=gen, device=dev)
            z.scatter_add_(1, at, up)
            x[r0:r1] = z.to(dt)
        T, k, p, mp = _given_params(case, seed)
        u = torch.rand((B, case["draws"]), generator=gen, device=dev)
        st = dict(op=op, x=x[:, :V], u=u, T=T, k=k, p=p, mp=mp, V=V)
        if own:
            from device_token_sampling_gb300 import Sampler
            s = Sampler(max_batch=B, max_vocab=V)
            one, zero = np.ones(B, np.float32), np.zeros(B, np.float32)
            s.reset_params(T, k, p, mp, zero, zero, one, np.zeros(B, np.uint64))
            st["sampler"] = s
        else:
            greedy = (T == 0) | (k == 1) | (p == 0) | (mp == 1)
            inv_t = np.where(greedy, np.float32(1), np.float32(1) / np.where(T == 0, 1, T))
            st.update(greedy=torch.from_numpy(greedy).to(dev),
                      inv_t=torch.from_numpy(inv_t.astype(np.float32)).to(dev),
                      kk=torch.from_numpy(np.where((k <= 1) | (k >= V), V, k)).to(dev),
                      pp=torch.from_numpy(p.astype(np.float64)).to(dev),
                      lmp=torch.from_numpy(np.log(np.maximum(mp.astype(np.float64), 1e-300))
                                           ).to(dev),
                      has_mp=torch.from_numpy(mp > 0).to(dev))
        return st
    bs = case["block"]
    if op == "tables":
        ln, cap = _table_lens(case, g)
        q, ctx = ln["query"], ln["ctx"]
        n_free = int((-(-(ctx + q) // bs)).sum()) + 64
        ids = g.permutation(n_free + case["prefix"] + 8).astype(np.int32)
        held = -(-ctx // bs)
        table = np.full((B, case["cols"]), -1, np.int32)
        if not case["scratch"]:
            for r in range(B):
                table[r, :held[r]] = g.integers(0, n_free, held[r])
                n = min(held[r], case["prefix"])
                table[r, :n] = ids[n_free:n_free + n]
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        st = dict(op=op, table=t(table), seq=t((ctx + q).astype(np.int32)),
                  query=t(q.astype(np.int32)), free=t(ids[:n_free]),
                  cursor=t(np.array([min(7, n_free)], np.int32)),
                  held=None if case["scratch"] else t(held.astype(np.int32)),
                  prefix=t(ids[n_free:n_free + case["prefix"]]), bs=bs, cap=cap)
        if own:
            from device_token_sampling_gb300 import PagedBatch
            st["paged"] = PagedBatch(max_batch=B, block_size=bs, max_blocks=case["cols"])
        return st
    # prefix attention: a cache with the blocks of all requests in random order
    hq, hkv, d, P, dt = case["hq"], case["hkv"], case["d"], case["prefix"], _DT[case["dtype"]]
    own_len = g.integers(1, case["max_own"] + 1, B)
    nshared = P // bs                       # whole blocks are shared; a broken one is copied
    nP = -(-P // bs)
    total = P + own_len
    nblk = -(-total // bs)
    cols = int(nblk.max())
    n_own = int((nblk - nshared).sum())
    n_cache = nP + n_own + 3
    ids = g.permutation(n_cache).astype(np.int32)
    table = np.zeros((B, cols), np.int32)
    table[:, :nshared] = ids[:nshared]
    at = nP
    for r in range(B):
        n = nblk[r] - nshared
        table[r, nshared:nshared + n] = ids[at:at + n]
        at += n
    kc = torch.randn((n_cache, bs, hkv, d), generator=gen, device=dev).to(dt)
    vc = torch.randn((n_cache, bs, hkv, d), generator=gen, device=dev).to(dt)
    prefix_blocks = torch.from_numpy(ids[:nP]).to(dev)
    tab = torch.from_numpy(table).to(dev)
    if nP > nshared:  # the copies of the broken block
        kc[tab[:, nshared].long()] = kc[int(ids[nshared])].clone()
        vc[tab[:, nshared].long()] = vc[int(ids[nshared])].clone()
    q = (torch.randn((B, hq, d), generator=gen, device=dev) * 1.5).to(dt)
    st = dict(op=op, q=q, k=kc, v=vc, table=tab, prefix_blocks=prefix_blocks, P=P, bs=bs,
              seq=torch.from_numpy(total.astype(np.int32)).to(dev), max_len=int(total.max()),
              scale=1.0 / math.sqrt(d))
    if own:
        from device_token_sampling_gb300 import PagedBatch
        st["paged"] = PagedBatch(max_batch=B, block_size=bs, max_blocks=cols, q_heads=hq,
                                 kv_heads=hkv, head_dim=d)
    return st


def _table_lens(case, g):
    """Context and query lengths of a tables case, and the slot map's capacity."""
    B, ml, mq = case["B"], case["max_len"], case["max_query"]
    if case["scratch"]:
        q = g.integers(0, mq + 1, B)
        ctx = np.zeros(B, np.int64)
    else:
        q = g.integers(min(1, mq), mq + 1, B)
        ctx = g.integers(0, max(1, ml - mq + 1), B)
    return dict(query=q, ctx=ctx), B * mq

# ---------------------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if op == "given":
        if own:
            return state["sampler"].sample_given(state["x"], state["u"])
        return _plain_given(state)
    if op == "tables":
        if own:
            out = state["paged"].build_tables(
                state["table"], state["seq"], state["query"], state["free"], state["cursor"],
                held=state["held"], prefix_blocks=state["prefix"], capacity=state["cap"])
            return (state["table"],) + tuple(out)
        return _plain_tables(state)
    if own:
        return state["paged"].attention(
            state["q"], state["k"], state["v"], state["table"], state["seq"],
            state["prefix_blocks"], state["P"], scale=state["scale"],
            max_seq_len=state["max_len"])
    return _plain_prefix(state)


def _plain_given(s):
    """Sums of masses run in 64 bits: the token is decided by comparing them."""
    x, u, V = s["x"], s["u"], s["V"]
    B, N = u.shape
    tokens = torch.empty((B, N), dtype=torch.int32, device=x.device)
    logp = torch.empty((B, N), dtype=torch.float32, device=x.device)
    rank = torch.arange(V, device=x.device)
    for r0 in range(0, B, 128):
        r = slice(r0, min(B, r0 + 128))
        z = x[r].float() * s["inv_t"][r, None]
        m = z.max(1, keepdim=True).values
        d = z.double() - m.double()
        w = torch.exp(d)
        total = w.sum(1, keepdim=True)
        zs, order = torch.sort(z, dim=1, descending=True, stable=True)
        ds = zs.double() - m.double()
        keep = (rank < s["kk"][r, None]) & (~s["has_mp"][r, None] | (ds >= s["lmp"][r, None]))
        ws = torch.where(keep, torch.exp(ds), 0.0)
        before = torch.cumsum(ws, 1) - ws
        p = s["pp"][r, None]
        keep &= (p >= 1) | (before <= p * ws.sum(1, keepdim=True))
        keep = torch.where(s["greedy"][r, None], rank == 0, keep)
        kept = torch.zeros_like(keep).scatter_(1, order, keep)
        cdf = torch.cumsum(torch.where(kept, w, 0.0), 1)
        for n in range(N):
            t = u[r, n:n + 1].double() * cdf[:, -1:]
            tok = (cdf <= t).sum(1, keepdim=True)
            tokens[r, n:n + 1] = tok.int()
            logp[r, n:n + 1] = (d.gather(1, tok) - torch.log(total)).float()
    return tokens, logp


def _plain_tables(s):
    table, seq, q, free, bs = s["table"], s["seq"].long(), s["query"].long(), s["free"], s["bs"]
    B, cols = table.shape
    nP, cap = s["prefix"].shape[0], s["cap"]
    col = torch.arange(cols, device=table.device)
    blocks = (seq + bs - 1) // bs
    shared = torch.clamp(blocks, max=nP)
    old = torch.zeros_like(blocks) if s["held"] is None else s["held"].long()
    have = torch.maximum(old, shared)
    bad = (seq < 0) | (q < 0) | (q > seq) | (blocks > cols)
    need = torch.where(bad, 0, torch.clamp(blocks - have, min=0))
    off = torch.cumsum(need, 0) - need
    c0 = s["cursor"].long()
    full = (need > 0) & (c0 + off + need > free.shape[0])
    ok = ~bad & ~full
    # the table: shared blocks, then blocks off the free list, then -1 in a new table
    pre = torch.full((cols,), -1, dtype=torch.int32, device=table.device)
    pre[:min(nP, cols)] = s["prefix"][:cols]
    pos = (c0 + off - have)[:, None] + col
    new = free[pos.clamp(0, max(0, free.shape[0] - 1))]
    out = torch.where(col < have[:, None], pre, new)
    out = torch.where((col < blocks[:, None]) & ok[:, None], out, -1)
    if s["held"] is not None:
        out = torch.where((col >= old[:, None]) & (col < blocks[:, None]) & ok[:, None], out,
                          table)
    table.copy_(out)
    held = torch.where(ok, torch.maximum(old, blocks), old)
    cursor = c0 + torch.where(ok, need, 0).sum()
    starts = torch.zeros(B + 1, dtype=torch.int64, device=table.device)
    starts[1:] = torch.cumsum(torch.where(bad, 0, q), 0)
    t = torch.arange(cap, device=table.device)
    row = (starts[1:, None] <= t).sum(0) if B * cap <= 1 << 27 else _rows(starts, t)
    row = row.clamp(max=B - 1)
    live = (t < starts[-1]) & ok[row]
    position = seq[row] - q[row] + t - starts[row]
    block = table[row, torch.where(live, position // bs, 0)].long()
    slot = torch.where(live, block * bs + position % bs, -1)
    return (table, held.int(), cursor.int(), starts.int(), slot,
            torch.where(live, position, -1).int(), torch.where(bad, 2, full.int()).int())


def _rows(starts, t):
    """The row of each token by marking row ends and summing the marks."""
    n = t.shape[0]
    mark = torch.zeros(n + 1, dtype=torch.int64, device=t.device)
    mark.index_add_(0, starts[1:].clamp(max=n), torch.ones_like(starts[1:]))
    return torch.cumsum(mark, 0)[:n]


def _plain_prefix(s):
    """Scores, weights and sums in 32 bits; one matrix product over the shared part for all
    requests, and a padded one over each request's own part."""
    q, bs, P = s["q"], s["bs"], s["P"]
    B, hq, d = q.shape
    hkv = s["k"].shape[2]
    G = hq // hkv
    dev = q.device
    pos = torch.arange(P, device=dev)
    blk = s["prefix_blocks"][pos // bs].long()
    kp = s["k"][blk, pos % bs].float().permute(1, 0, 2)                    # [hkv, P, d]
    vp = s["v"][blk, pos % bs].float().permute(1, 0, 2)
    qh = q.float().view(B, hkv, G, d)
    qa = qh.permute(1, 0, 2, 3).reshape(hkv, B * G, d)
    sp = (torch.matmul(qa, kp.transpose(1, 2)) * s["scale"]).view(hkv, B, G, P)
    sp = sp.masked_fill(pos >= s["seq"][None, :, None, None], -math.inf)
    L = max(1, s["max_len"] - P)
    own_pos = P + torch.arange(L, device=dev)
    valid = own_pos < s["seq"][:, None]
    blk = torch.gather(s["table"].long(), 1, torch.where(valid, own_pos // bs, 0))
    ko = s["k"][blk, own_pos % bs].float().permute(0, 2, 3, 1)             # [B, hkv, d, L]
    vo = s["v"][blk, own_pos % bs].float().permute(0, 2, 1, 3)             # [B, hkv, L, d]
    so = torch.matmul(qh, ko) * s["scale"]                                 # [B, hkv, G, L]
    so = so.masked_fill(~valid[:, None, None, :], -math.inf)
    m = torch.maximum(sp.amax(-1).permute(1, 0, 2), so.amax(-1))           # [B, hkv, G]
    m0 = torch.where(m == -math.inf, 0.0, m)
    ep = torch.exp(sp - m0.permute(1, 0, 2)[..., None])
    eo = torch.exp(so - m0[..., None])
    tot = ep.sum(-1).permute(1, 0, 2) + eo.sum(-1)
    acc = torch.matmul(ep.view(hkv, B * G, P), vp).view(hkv, B, G, d).permute(1, 0, 2, 3)
    acc = acc + torch.matmul(eo, vo)
    out = acc / torch.where(tot == 0, 1.0, tot)[..., None]
    return out.reshape(B, hq, d).to(q.dtype), (m + torch.log(tot)).reshape(B, hq)

# ---------------------------------------------------------------------------- the work

def work(case):
    B = case["B"]
    if case["op"] == "given":
        es = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=B * case["V"] * es + B * case["draws"] * 12 + 24 * B,
                    flops=4 * B * case["V"])  # scale, subtract, exp, add: one of each an element
    if case["op"] == "tables":
        bs = case["block"]
        cap = B * case["max_query"]
        if case["scratch"]:
            entries = B * case["cols"]
            new = B * (case["max_query"] / 2 / bs)
        else:
            new = entries = B * max(1.0, (1 + case["max_query"]) / 2) / bs
        return dict(bytes=int(8 * B + 4 * new + 4 * entries + 12 * cap + 12 * B),
                    flops=int(4 * cap + 8 * B))
    es = 2
    own_len = (1 + case["max_own"]) / 2
    kv = (case["prefix"] + B * own_len) * case["hkv"] * case["d"] * 2 * es
    io = B * case["hq"] * (2 * case["d"] * es + 4)
    return dict(bytes=int(kv + io),
                flops=int(4 * B * case["hq"] * case["d"] * (case["prefix"] + own_len)))

# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "given":
        return _exact_given(s)
    if case["op"] == "prefix":
        return _exact_prefix(s)
    return None  # whole numbers throughout


def _exact_given(s):
    """Row by row, on the set itself: survivors, sorted, cut, put back in order."""
    x, V = s["x"], s["V"]
    u = s["u"].double()
    B, N = u.shape
    tokens = torch.empty((B, N), dtype=torch.int64, device=x.device)
    logp = torch.empty((B, N), dtype=torch.float64, device=x.device)
    for r in range(B):
        T, k, p, mp = float(s["T"][r]), int(s["k"][r]), float(s["p"][r]), float(s["mp"][r])
        greedy = T == 0 or k == 1 or p == 0 or mp == 1
        # the tempered logit is a 32-bit number by definition, everything after it is exact
        z = x[r].float() if greedy else x[r].float() * float(np.float32(1) / np.float32(T))
        z = z.double()
        m = z.max()
        lse = m + torch.log(torch.exp(z - m).sum())
        if greedy:
            tok = (z == m).nonzero()[0].expand(N)
        else:
            ids = torch.arange(V, device=x.device)
            if mp > 0:
                ids = (z - m >= math.log(mp)).nonzero()[:, 0]
            down = torch.sort(-z[ids], stable=True).indices
            ids = ids[down]
            if 1 < k < V:
                ids = ids[:k]
            if p < 1:
                c = torch.cumsum(torch.exp(z[ids] - m), 0)
                first_out = int((c <= p * c[-1]).sum())     # prefixes within p of the mass
                ids = ids[:first_out + 1]
            ids = ids.sort().values
            c = torch.cumsum(torch.exp(z[ids] - m), 0)
            tok = ids[torch.searchsorted(c, u[r] * c[-1], right=True)]
        tokens[r] = tok
        logp[r] = z[tok] - lse
    return tokens, logp


def _exact_prefix(s):
    """Request by request over its whole gathered context."""
    q, bs = s["q"].double(), s["bs"]
    B, hq, d = q.shape
    hkv = s["k"].shape[2]
    out = torch.zeros((B, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        n = int(s["seq"][b])
        if n == 0:
            continue
        at = torch.arange(n, device=q.device)
        ids = s["table"][b].long()[at // bs]
        k = s["k"][ids, at % bs].double()
        v = s["v"][ids, at % bs].double()
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            a = s["scale"] * (q[b, heads] @ k[:, h].T)
            lse[b, heads] = torch.logsumexp(a, 1)
            out[b, heads] = torch.softmax(a, 1) @ v[:, h]
    return out, lse
