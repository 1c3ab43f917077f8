"""Plain references for the paged batch: the block tables one request at a time
on the host, the attention in 64 bits over each request's gathered context."""
from __future__ import annotations

import math

import numpy as np


def tables_reference(table, seq, query, free, cursor, held, prefix, block_size, max_blocks,
                     capacity):
    """Returns (table, held, cursor, starts, slots, positions, status) as int64 arrays."""
    B = len(seq)
    new = held is None
    table = np.array(table, np.int64)
    if new:
        table[:, :max_blocks] = -1
    out_held = np.zeros(B, np.int64) if new else np.array(held, np.int64)
    status = np.zeros(B, np.int64)
    starts = np.zeros(B + 1, np.int64)
    slots = np.full(capacity, -1, np.int64)
    positions = np.full(capacity, -1, np.int64)
    at = int(cursor)
    usable = 0 <= at <= len(free)
    asked = at if usable else len(free)
    at_out = at
    for r in range(B):
        s, q = int(seq[r]), int(query[r])
        blocks = -(-s // block_size)
        if s < 0 or q < 0 or q > s or blocks > max_blocks:
            status[r] = 2
            starts[r + 1] = starts[r]
            continue
        starts[r + 1] = starts[r] + q
        have = max(int(out_held[r]), min(blocks, len(prefix)))
        need = max(0, blocks - have)
        if need and asked + need > len(free):
            status[r] = 1
            asked += need
            continue
        for c in range(int(out_held[r]), blocks):
            table[r, c] = prefix[c] if c < have else free[asked + c - have]
        asked += need
        if need:
            at_out = asked
        out_held[r] = max(int(out_held[r]), blocks)
        for i in range(q):
            t, p = starts[r] + i, s - q + i
            if t < capacity:
                slots[t] = table[r, p // block_size] * block_size + p % block_size
                positions[t] = p
    return table, out_held, at_out, starts, slots, positions, status


def attention_reference(q, k_cache, v_cache, table, seq, prefix_blocks, prefix_len, block_size,
                        scale):
    """(out, lse, bound_out, bound_lse) in float64 on q's device.

    The bounds count what the operator rounds: the result once and each weight once to q's
    type (half a step each, the weights' own rounding in absolute terms below the smallest
    normal number), and fp32 accumulation of the head_dim and of the sequence's terms."""
    import torch
    B, hq, d = q.shape
    hkv = k_cache.shape[2]
    G = hq // hkv
    dev = q.device
    half = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * half
    out = torch.zeros((B, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device=dev)
    b_out = torch.zeros_like(out)
    b_lse = torch.zeros_like(lse)
    for b in range(B):
        n = int(seq[b])
        if n <= 0:
            continue
        pos = torch.arange(n, device=dev)
        ids = torch.where(pos < prefix_len,
                          prefix_blocks[(pos.clamp(max=max(prefix_len - 1, 0))) // block_size]
                          if prefix_len else torch.zeros_like(pos).int(),
                          table[b][pos // block_size]).long()
        ok = (ids >= 0) & (ids < k_cache.shape[0])
        pos, ids = pos[ok], ids[ok]
        if pos.numel() == 0:
            continue
        k = k_cache[ids, pos % block_size].double()
        v = v_cache[ids, pos % block_size].double()
        for h in range(hkv):
            heads = slice(h * G, (h + 1) * G)
            qq = q[b, heads].double()
            s = scale * (qq @ k[:, h].T)
            w = torch.softmax(s, 1)
            out[b, heads] = w @ v[:, h]
            lse[b, heads] = torch.logsumexp(s, 1)
            err_s = (abs(scale) * (qq.abs() @ k[:, h].abs().T)).amax(1) * d * 2.0 ** -23 + 2.0 ** -21
            err_s = err_s + pos.numel() * 2.0 ** -23
            mag = w @ v[:, h].abs()
            peak = torch.exp(s.amax(1) - lse[b, heads])       # 1 over the sum of the weights
            b_out[b, heads] = (half * out[b, heads].abs() + (half + 2 * err_s[:, None]) * mag
                               + tiny * peak[:, None] * v[:, h].abs().sum(0) + tiny)
            b_lse[b, heads] = err_s + 2.0 ** -23 * lse[b, heads].abs()
    return out, lse, b_out, b_lse
