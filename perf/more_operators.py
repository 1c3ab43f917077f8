"""Cases for the operators of a speculative and branching decode loop.

Four operators, named by a case's ``op``:

* ``verify``  -- ``Sampler.verify``: drafted tokens accepted or refused against the target's
  probabilities with given random numbers, and the token behind the accepted ones drawn from
  what is left;
* ``chunk``   -- ``PagedBatch.chunk_attention``: several new query tokens a request over its
  paged cache, each up to its own position;
* ``fork``    -- ``PagedBatch.fork`` and ``PagedBatch.copy_blocks``: rows of the next step that
  continue rows of this one, sharing whole blocks and copying the broken last one;
* ``reclaim`` -- ``PagedBatch.release``: blocks past the requests' lengths go back and the free
  list is made anew; or ``PagedBatch.compact`` and ``copy_blocks``: blocks in use move to the
  cache's low end.

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
        # one request with seven drafts: latency
        dict(name="verify_one", op="verify", B=1, K=7, V=151936, pad=0, dtype="bf16",
             drafter="model", ragged=False, flat=False, filtered=True),
        # drafts looked up in the prompt (no probabilities), an odd vocabulary in rows that no
        # vector load is aligned to
        dict(name="verify_odd", op="verify", B=29, K=4, V=32003, pad=0, dtype="f32",
             drafter="lookup", ragged=True, flat=False, filtered=False),
        # the package's b256 batch, four drafts a request, rows laid out token by token
        dict(name="verify_b256", op="verify", B=256, K=4, V=151936, pad=0, dtype="f32",
             drafter="model", ragged=True, flat=True, filtered=False),
        # four short requests, five tokens each: latency
        dict(name="chunk_small", op="chunk", B=4, hq=32, hkv=8, d=128, block=16, n_lo=5, n_hi=5,
             ctx_lo=100, ctx_hi=600, dtype="bf16"),
        # ragged prompts and single tokens in one batch, groups of 7 heads
        dict(name="chunk_odd", op="chunk", B=13, hq=28, hkv=4, d=64, block=16, n_lo=1, n_hi=201,
             ctx_lo=0, ctx_hi=3001, dtype="f16"),
        # a verification step of an ordinary batch over long contexts
        dict(name="chunk_b64", op="chunk", B=64, hq=32, hkv=8, d=128, block=64, n_lo=1, n_hi=8,
             ctx_lo=4096, ctx_hi=8192, dtype="bf16"),
        # chunks of long prompts behind what earlier chunks left in the cache
        dict(name="chunk_prefill", op="chunk", B=4, hq=32, hkv=8, d=128, block=64, n_lo=2048,
             n_hi=4096, ctx_lo=0, ctx_hi=16384, dtype="bf16"),
        # eight beams of one short request
        dict(name="fork_small", op="fork", B=8, rows=8, block=16, cols=64, max_len=600,
             kind="beams", layers=2, hkv=8, d=128, blocks=1024),
        # a large batch branching: 512 continuations of 128 requests
        dict(name="fork_large", op="fork", B=128, rows=512, block=64, cols=160, max_len=8192,
             kind="beams", layers=4, hkv=8, d=128, blocks=2048),
        # behind a verification step: the refused drafts' blocks of 256 requests
        dict(name="release_step", op="reclaim", B=256, block=16, cols=1024, max_len=8192,
             blocks=131072, compact=False, layers=0, hkv=0, d=0),
        # requests that ended, in a large serving state
        dict(name="release_large", op="reclaim", B=2048, block=16, cols=512, max_len=8192,
             blocks=1048576, compact=False, layers=0, hkv=0, d=0),
        # a cache half empty is packed to its low end
        dict(name="compact", op="reclaim", B=61, block=64, cols=160, max_len=8000, blocks=6000,
             compact=True, layers=2, hkv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "chunk", "fork", "reclaim"])
    if op == "verify":
        V = _log_int(rng, 1000, 248320)
        K = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        B = _log_int(rng, 1, min(1024, max(1, 190_000_000 // (V * (K + 1)))))
        return dict(op=op, B=B, K=K, V=V, pad=rng.choice([0, 0, 8, 13]),
                    dtype=rng.choice(["bf16", "f32"]), drafter=rng.choice(["model", "lookup"]),
                    ragged=rng.random() < 0.7, flat=rng.random() < 0.5,
                    filtered=rng.random() < 0.5)
    if op == "chunk":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        B = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, 16384)
        most = 1_800_000_000 // (B * hq)
        n = _log_int(rng, 1, min(4096, max(2, most // (ctx + 64)), int(math.sqrt(most))))
        return dict(op=op, B=B, hq=hq, hkv=hkv, d=d, block=rng.choice([8, 16, 32, 64, 128]),
                    n_lo=rng.choice([1, max(1, n // 2), n]), n_hi=n,
                    ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx,
                    dtype=rng.choice(["bf16", "f16"]))
    block = rng.choice([8, 16, 32, 64, 128])
    if op == "fork":
        B = _log_int(rng, 1, 512)
        rows = _log_int(rng, 1, 512)
        max_len = _log_int(rng, 4, 8192)
        blocks = B + rows + _log_int(rng, 64, 1024)
        return dict(op=op, B=B, rows=rows, block=block, cols=-(-max_len // block) + 2,
                    max_len=max_len, kind=rng.choice(["beams", "one"]),
                    layers=rng.choice([1, 2, 4]), hkv=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([64, 128]), blocks=blocks)
    compact = rng.random() < 0.5
    B = _log_int(rng, 1, 2048)
    max_len = _log_int(rng, 16, 8192)
    cols = -(-max_len // block) + rng.randrange(0, 4)
    layers, hkv, d = (rng.choice([1, 2]), rng.choice([1, 2]), 64) if compact else (0, 0, 0)
    most = 8192 if compact else 1048576
    blocks = min(most, max(64, int(B * cols * rng.uniform(0.6, 2.0))))
    return dict(op=op, B=B, block=block, cols=cols, max_len=max_len, blocks=blocks,
                compact=compact, layers=layers, hkv=hkv, d=d)


_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# ---------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g = np.random.default_rng([seed, 11])
    return _PREPARE[case["op"]](case, gen, g)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to("cuda")


def _probabilities(z, filtered):
    """Rows of probabilities; filtered: of the entries within 6 of the largest alone."""
    if filtered:
        z = z.masked_fill(z < z.amax(-1, keepdim=True) - 6, -math.inf)
    return torch.softmax(z, -1)


def _prepare_verify(case, gen, g):
    """Target rows: N(0, 1.5) logits with 8 columns a row raised by U(4, 12).  A drafting model's
    rows: the target's logits with N(0, 0.7) noise; its tokens are drawn from them.  Lookups: the
    target's likeliest token three times in four."""
    B, K, V, dt, dev = case["B"], case["K"], case["V"], _DT[case["dtype"]], "cuda"
    ld = V + case["pad"]
    lens = g.integers(0, K + 1, B) if case["ragged"] else np.full(B, K)
    rows = np.where(case["flat"], lens + 1, K + 1)
    starts = np.concatenate([[0], np.cumsum(rows)])
    T = int(starts[-1])
    model = case["drafter"] == "model"
    target = torch.zeros((T, ld), dtype=dt, device=dev)
    draft = torch.zeros((B, K, ld), dtype=dt, device=dev) if model else None
    tokens = torch.full((B, K), -1, dtype=torch.int32, device=dev)
    for r0 in range(0, B, 32):
        r1 = min(B, r0 + 32)
        z = torch.randn((r1 - r0, K + 1, V), generator=gen, device=dev) * 1.5
        at = torch.randint(0, V, (r1 - r0, K + 1, 8), generator=gen, device=dev)
        z.scatter_add_(2, at, 4 + 8 * torch.rand(at.shape, generator=gen, device=dev))
        p = _probabilities(z, case["filtered"])
        for r in range(r0, r1):
            target[starts[r]:starts[r + 1], :V] = p[r - r0, :rows[r]].to(dt)
        if model:
            z = z[:, :K]
            z += torch.randn(z.shape, generator=gen, device=dev) * 0.7
            q = _probabilities(z, case["filtered"]).to(dt)
            draft[r0:r1, :, :V] = q
            e = torch.empty(z.shape, device=dev).exponential_(generator=gen)
            tokens[r0:r1] = (q.float() / e).argmax(-1).int()
        else:
            best = p[:, :K].argmax(-1).int()
            other = torch.randint(0, V, best.shape, generator=gen, device=dev).int()
            keep = torch.rand(best.shape, generator=gen, device=dev) < 0.75
            tokens[r0:r1] = torch.where(keep, best, other)
    st = dict(op="verify", B=B, K=K, V=V, target=target[:, :V], draft=draft, tokens=tokens,
              u=torch.rand((B, K + 1), generator=gen, device=dev), lens=_i32(lens),
              starts=_i32(starts) if case["flat"] else None)
    if draft is not None:
        st["draft"] = draft[:, :, :V]
    if not case["flat"]:
        st["target"] = target.view(B, K + 1, ld)[:, :, :V]
    if own:
        from device_token_sampling_gb300 import Sampler
        st["sampler"] = Sampler(max_batch=B, max_vocab=V)
    return st


def _prepare_chunk(case, gen, g):
    """N(0, 1) keys and values in blocks in random order, N(0, 1.5) queries.  The chunks' lengths
    are the case's, in an order of the seed's."""
    B, hq, hkv, d, bs, dt = (case[k] for k in ("B", "hq", "hkv", "d", "block", "dtype"))
    dt = _DT[dt]
    n = g.permutation(np.random.default_rng([B, hq]).integers(case["n_lo"], case["n_hi"] + 1, B))
    total = g.integers(case["ctx_lo"], case["ctx_hi"] + 1, B) + n
    nblk = -(-total // bs)
    cols, n_cache = int(nblk.max()), int(nblk.sum()) + 3
    ids = g.permutation(n_cache)
    table = np.zeros((B, cols), np.int32)
    at = 0
    for r in range(B):
        table[r, :nblk[r]] = ids[at:at + nblk[r]]
        at += nblk[r]
    T = int(n.sum())
    k = torch.randn((n_cache, bs, hkv, d), generator=gen, device="cuda").to(dt)
    v = torch.randn((n_cache, bs, hkv, d), generator=gen, device="cuda").to(dt)
    q = (torch.randn((T, hq, d), generator=gen, device="cuda") * 1.5).to(dt)
    st = dict(op="chunk", q=q, k=k, v=v, table=_i32(table), bs=bs, seq=_i32(total),
              starts=_i32(np.concatenate([[0], np.cumsum(n)])), n=n, total=total,
              scale=1.0 / math.sqrt(d))
    if own:
        from device_token_sampling_gb300 import PagedBatch
        st["paged"] = PagedBatch(max_batch=B, block_size=bs, max_blocks=cols, q_heads=hq,
                                 kv_heads=hkv, head_dim=d)
    return st


def _caches(case, gen):
    shape = (case["blocks"], case["block"], case["hkv"], case["d"])
    return [torch.randn(shape, generator=gen, device="cuda").bfloat16()
            for _ in range(2 * case["layers"])]


def _paged(case, rows):
    from device_token_sampling_gb300 import PagedBatch
    return PagedBatch(max_batch=rows, block_size=case["block"], max_blocks=case["cols"])


def _prepare_fork(case, gen, g):
    """Requests whose last blocks are their own and whose others are of a common pool."""
    B, R, bs, cols, blocks = (case[k] for k in ("B", "rows", "block", "cols", "blocks"))
    seq = g.integers(1, case["max_len"] + 1, B)
    held = -(-seq // bs)
    ids = g.permutation(blocks)
    table = np.where(np.arange(cols) < held[:, None], g.choice(ids[B + R:], (B, cols)), -1)
    table[np.arange(B), held - 1] = ids[:B]
    # beams: the better half of the rows continues, each several times
    parents = (np.zeros(R, np.int64) if case["kind"] == "one"
               else g.integers(0, max(1, (B + 1) // 2), R) * 2 % B)
    st = dict(op="fork", table=_i32(table), held=_i32(held), seq=_i32(seq), bs=bs,
              parents=_i32(parents), free=_i32(ids[B:B + R]), cursor=_i32([0]),
              caches=_caches(case, gen),
              out_table=torch.full((R, cols), -1, dtype=torch.int32, device="cuda"))
    if own:
        st["paged"] = _paged(case, max(B, R))
    return st


def _prepare_reclaim(case, gen, g):
    """Tables filled to their columns, or as far as the cache goes, of requests that keep a part."""
    B, bs, cols, blocks = (case[k] for k in ("B", "block", "cols", "blocks"))
    each = min(cols, -(-case["max_len"] // bs), max(1, (blocks - 8) // B))
    each = min(each, max(1, (blocks - 8) * 3 // (4 * B) + 1))
    held = np.minimum(g.integers(max(1, each // 2), each + 1, B), each)
    ids = g.permutation(blocks)
    table = np.full((B, cols), -1, np.int32)
    at = (np.cumsum(held) - held) % max(1, blocks - 8 - each)
    for r in range(B):
        table[r, :held[r]] = ids[8 + at[r]:8 + at[r] + held[r]]
    keep = np.where(g.random(B) < 0.3, 0, held * bs - g.integers(0, 3 * bs, B)).clip(0)
    st = dict(op="reclaim", table=_i32(table), held=_i32(held), seq=_i32(keep), bs=bs,
              blocks=blocks, prefix=_i32(ids[:8]), compact=case["compact"],
              caches=_caches(case, gen))
    if case["compact"]:
        st["out_table"] = torch.empty_like(st["table"])
    if own:
        st["paged"] = _paged(case, B)
    return st


_PREPARE = dict(verify=_prepare_verify, chunk=_prepare_chunk, fork=_prepare_fork,
                reclaim=_prepare_reclaim)

# ---------------------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if not own:
        return _PLAIN[op](state)
    if op == "verify":
        return state["sampler"].verify(state["target"], state["tokens"], state["u"],
                                       draft_probs=state["draft"], draft_lens=state["lens"],
                                       starts=state["starts"])
    p = state["paged"]
    if op == "chunk":
        return p.chunk_attention(state["q"], state["starts"], state["k"], state["v"],
                                 state["table"], state["seq"], scale=state["scale"])
    if op == "fork":
        out = p.fork(state["table"], state["held"], state["seq"], state["parents"],
                     state["free"], state["cursor"], state["out_table"])
        p.copy_blocks(state["caches"], out[3], out[4])
        return (state["out_table"],) + tuple(out) + tuple(state["caches"])
    if not state["compact"]:
        out = p.release(state["table"], state["held"], state["seq"], state["blocks"],
                        prefix_blocks=state["prefix"])
        return (state["table"],) + tuple(out)
    out = p.compact(state["table"], state["held"], state["seq"], state["blocks"],
                    prefix_blocks=state["prefix"], out_table=state["out_table"])
    p.copy_blocks(state["caches"], out[3], out[4], count=out[5])
    return (state["out_table"],) + tuple(out) + tuple(state["caches"])


def _plain_verify(s):
    """Products and sums in 64 bits: an acceptance and a token are decided by comparing them."""
    p, q, tok, u, K, V = s["target"], s["draft"], s["tokens"].long(), s["u"], s["K"], s["V"]
    B, dev = s["B"], p.device
    row = torch.arange(B, device=dev)
    step = torch.arange(K, device=dev)
    if s["starts"] is None:
        p = p.reshape(B * (K + 1), V)
        base = row * (K + 1)
    else:
        base = s["starts"][:-1].long()
    lens = s["lens"].long()
    at = (base[:, None] + step).clamp(max=p.shape[0] - 1)
    px = p[at, tok.clamp(0)].double()
    qx = (torch.ones_like(px) if q is None else
          torch.gather(q, 2, tok.clamp(0)[..., None])[..., 0].double())
    yes = (u[:, :K].double() * qx < px) & (step < lens[:, None])
    accepted = torch.cumprod(yes.long(), 1).sum(1)
    out = torch.where(step < accepted[:, None], tok, -1).int()
    out = torch.cat([out, torch.full((B, 1), -1, dtype=torch.int32, device=dev)], 1)
    new = torch.empty((B,), dtype=torch.int64, device=dev)
    for r0 in range(0, B, 128):
        r = slice(r0, min(B, r0 + 128))
        w = p[base[r] + accepted[r]].double()
        short = (accepted[r] < lens[r])[:, None]
        j = accepted[r].clamp(max=K - 1)
        if q is None:
            w.scatter_(1, tok[row[r], j][:, None],
                       torch.where(short, 0.0, w.gather(1, tok[row[r], j][:, None])))
        else:
            w -= torch.where(short, q[row[r], j].double(), 0.0)
            w.clamp_(min=0.0)
        cdf = torch.cumsum(w, 1)
        new[r] = (cdf <= u[r, K:].double() * cdf[:, -1:]).sum(1)
    out.scatter_(1, accepted[:, None], new[:, None].int())
    return out, accepted.int()


def _plain_chunk(s):
    """Requests padded to the longest of a few; scores, weights and sums in 32 bits."""
    q, bs, n, total = s["q"], s["bs"], s["n"], s["total"]
    T, hq, d = q.shape
    hkv = s["k"].shape[2]
    G = hq // hkv
    dev = q.device
    out = torch.empty((T, hq, d), dtype=torch.float32, device=dev)
    lse = torch.empty((T, hq), dtype=torch.float32, device=dev)
    B = len(n)
    b0 = 0
    while b0 < B:
        b1 = b0 + 1  # as many requests as 2^31 scores hold
        while b1 < B and ((b1 + 1 - b0) * hq * int(n[b0:b1 + 1].max())
                          * int(total[b0:b1 + 1].max())) <= 1 << 31:
            b1 += 1
        N, L = int(n[b0:b1].max()), int(total[b0:b1].max())
        r = slice(b0, b1)
        first, last = s["starts"][b0:b1].long(), s["starts"][b0 + 1:b1 + 1].long()
        seq = s["seq"][r].long()
        i = torch.arange(N, device=dev)
        j = torch.arange(L, device=dev)
        there = j < seq[:, None]
        blk = torch.gather(s["table"][r].long(), 1, torch.where(there, j // bs, 0))
        k = s["k"][blk, j % bs].float().permute(0, 2, 3, 1)                  # [b, hkv, d, L]
        rows = (first[:, None] + i).clamp(max=T - 1)
        live = first[:, None] + i < last[:, None]
        x = q[rows].float().view(-1, N, hkv, G, d).permute(0, 2, 3, 1, 4)     # [b, hkv, G, N, d]
        a = torch.matmul(x.reshape(-1, hkv, G * N, d), k).view(-1, hkv, G, N, L)
        a *= s["scale"]
        end = seq[:, None] - (last - first)[:, None] + i                      # last one seen
        a.masked_fill_((j > end[..., None])[:, None, None], -math.inf)
        m = a.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        a -= m
        a.exp_()
        tot = a.sum(-1, keepdim=True)
        v = s["v"][blk, j % bs].float().permute(0, 2, 1, 3)                   # [b, hkv, L, d]
        o = torch.matmul(a.view(-1, hkv, G * N, L), v).view(-1, hkv, G, N, d)
        o /= torch.where(tot == 0, 1.0, tot)
        ls = (m + torch.log(tot))[..., 0]
        out[rows[live]] = o.permute(0, 3, 1, 2, 4).reshape(-1, N, hq, d)[live]
        lse[rows[live]] = ls.permute(0, 3, 1, 2).reshape(-1, N, hq)[live]
        b0 = b1
    return out.to(q.dtype), lse


def _plain_copy(caches, src, dst):
    some = src >= 0
    a, b = src[some].long(), dst[some].long()
    for c in caches:
        c[b] = c[a]


def _plain_fork(s):
    table, bs, free = s["table"], s["bs"], s["free"]
    B, cols = table.shape
    par = s["parents"].long()
    R, dev = par.shape[0], table.device
    r = torch.arange(R, device=dev)
    col = torch.arange(cols, device=dev)
    first = torch.full((B,), R, device=dev).scatter_reduce_(0, par, r, "amin")
    stays = first[par] == r              # the child that keeps the parent's row as it is
    seq, held = s["seq"].long()[par], s["held"].long()[par]
    blocks = (seq + bs - 1) // bs
    need = ~stays & (seq % bs != 0)
    c0 = s["cursor"].long()
    at = c0 + torch.cumsum(need, 0) - need.long()
    full = need & (at >= free.shape[0])
    ok = ~full
    new = free[at.clamp(max=free.shape[0] - 1)]
    mine = torch.where(ok, torch.where(stays, held, blocks), 0)
    out = torch.where(col < mine[:, None], table[par], -1)
    fresh = need & ok
    src = torch.where(fresh, table[par, (blocks - 1).clamp(0)], -1)
    dst = torch.where(fresh, new, -1)
    out = torch.where(fresh[:, None] & (col == blocks[:, None] - 1), new[:, None], out)
    s["out_table"].copy_(out)
    _plain_copy(s["caches"], src, dst)
    return (s["out_table"], mine.int(), torch.where(ok, seq, 0).int(),
            (c0 + fresh.sum()).int(), src, dst, full.int()) + tuple(s["caches"])


def _plain_reclaim(s):
    table, bs, N = s["table"], s["bs"], s["blocks"]
    cols = table.shape[1]
    dev = table.device
    kept = torch.minimum((s["seq"].long() + bs - 1) // bs, s["held"].long())
    inside = torch.arange(cols, device=dev) < kept[:, None]
    used = torch.zeros(N + 1, dtype=torch.bool, device=dev)
    used[torch.where(inside, table, N).reshape(-1).long()] = True
    used[s["prefix"].long()] = True
    used = used[:N]
    ids = torch.arange(N, device=dev)
    before = torch.cumsum(used, 0) - used.long()            # used blocks of lower ids
    n_used = used.sum()
    if not s["compact"]:
        table.copy_(torch.where(inside, table, -1))
        blocks = torch.empty(N, dtype=torch.int32, device=dev)
        blocks[torch.where(used, before, n_used + ids - before)] = ids.int()
        return table, kept.int(), blocks, n_used.int().reshape(1)
    most = N // 2
    moves = used & (ids >= n_used)
    hole = ~used & (ids < n_used)
    below = torch.cumsum(moves, 0) - moves.long()
    holes = torch.cumsum(hole, 0) - hole.long()
    src = torch.full((N + 1,), -1, dtype=torch.int32, device=dev)
    dst = src.clone()
    src[torch.where(moves, below, N)] = ids.int()
    dst[torch.where(hole, holes, N)] = ids.int()
    src, dst = src[:most].contiguous(), dst[:most].contiguous()
    now = torch.where(moves, dst[below.clamp(max=most - 1)], ids).int()
    s["out_table"].copy_(torch.where(inside, now[table.long().clamp(0)], -1))
    _plain_copy(s["caches"], src, dst)
    return (s["out_table"], kept.int(), ids.int(), n_used.int().reshape(1), src, dst,
            moves.sum().int().reshape(1), now[s["prefix"].long()]) + tuple(s["caches"])


_PLAIN = dict(verify=_plain_verify, chunk=_plain_chunk, fork=_plain_fork, reclaim=_plain_reclaim)

# ---------------------------------------------------------------------------- the work

def work(case):
    op, B = case["op"], case["B"]
    if op == "verify":
        # one row a request is read: with a model's drafts two of four are refused at some
        # place, and then the drafter's row as well
        es = 4 if case["dtype"] == "f32" else 2
        rows = 1.5 if case["drafter"] == "model" else 1.0
        K = case["K"]
        return dict(bytes=int(B * (rows * case["V"] * es + K * (4 + 4 + 2 * es) + 8 * K + 16)),
                    flops=int(2 * B * rows * case["V"]))
    if op == "chunk":
        es, hq, hkv, d = 2, case["hq"], case["hkv"], case["d"]
        n = (case["n_lo"] + case["n_hi"]) / 2
        ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
        return dict(bytes=int(B * ((ctx + n) * hkv * d * 2 * es + n * hq * (2 * d * es + 4))),
                    flops=int(4 * B * hq * d * n * (ctx + n / 2)))
    block_bytes = 2 * case["layers"] * case["block"] * case["hkv"] * case["d"] * 2
    if op == "fork":
        R = case["rows"]
        parents = 1 if case["kind"] == "one" else max(1, (B + 1) // 2)
        copies = R - parents * (1 - (1 - 1 / parents) ** R)
        entries = R * case["max_len"] / 2 / case["block"]
        return dict(bytes=int(2 * copies * block_bytes + 4 * (entries + R * case["cols"]) + 40 * R),
                    flops=R)
    each = min(case["cols"], -(-case["max_len"] // case["block"]),
               max(1, (case["blocks"] - 8) * 3 // (4 * B) + 1))
    entries = 0.75 * each * B * 0.7
    n = min(case["blocks"], entries)
    free = case["blocks"] - n
    moves = n * free / case["blocks"] if case["compact"] else 0
    columns = B * case["cols"] if case["compact"] else 0.3 * entries
    return dict(bytes=int(4 * entries + 4 * columns + 12 * B + 4 * case["blocks"]
                          + 2 * moves * block_bytes),
                flops=int(case["blocks"]))

# ---------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "verify":
        return _exact_verify(prepare(case, seed))
    if case["op"] == "chunk":
        return _exact_chunk(prepare(case, seed))
    return None  # whole numbers, and blocks copied as they are


def _exact_verify(s):
    """Request by request: the first refused draft, then the draw on the row's support."""
    B, K = s["B"], s["K"]
    out = torch.full((B, K + 1), -1, dtype=torch.int64)
    accepted = torch.zeros(B, dtype=torch.int64)
    lens, tok, u = s["lens"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    starts = s["starts"].tolist() if s["starts"] is not None else None
    for b in range(B):
        rows = s["target"][b] if starts is None else s["target"][starts[b]:starts[b + 1]]
        a = 0
        while a < lens[b]:
            x = tok[b][a]
            q = 1.0 if s["draft"] is None else float(s["draft"][b, a, x])
            if not u[b][a] * q < float(rows[a, x]):
                break
            out[b, a] = x
            a += 1
        w = rows[a].double()
        if a < lens[b]:
            q = torch.zeros_like(w)
            if s["draft"] is None:
                q[tok[b][a]] = math.inf
            else:
                q = s["draft"][b, a].double()
            w = torch.relu(w - q)
        ids = w.nonzero()[:, 0]
        c = torch.cumsum(w[ids], 0)
        t = u[b][K] * c[-1]
        out[b, a] = ids[torch.searchsorted(c, t.reshape(1), right=True)[0]]
        accepted[b] = a
    return out, accepted


def _exact_chunk(s):
    """Request by request and head by head over the gathered context."""
    q, bs = s["q"].double(), s["bs"]
    T, hq, d = q.shape
    hkv = s["k"].shape[2]
    G = hq // hkv
    out = torch.zeros((T, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=q.device)
    t0 = 0
    for b, (n, L) in enumerate(zip(s["n"].tolist(), s["total"].tolist())):
        j = torch.arange(L, device=q.device)
        ids = s["table"][b].long()[j // bs]
        k, v = s["k"][ids, j % bs].double(), s["v"][ids, j % bs].double()
        hidden = j[None] > j[L - n:, None]
        for h in range(hq):
            a = s["scale"] * (q[t0:t0 + n, h] @ k[:, h // G].T)
            a[hidden] = -math.inf
            lse[t0:t0 + n, h] = torch.logsumexp(a, 1)
            out[t0:t0 + n, h] = torch.softmax(a, 1) @ v[:, h // G]
        t0 += n
    return out, lse
