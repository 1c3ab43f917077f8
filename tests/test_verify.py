"""Sampler.verify against a plain implementation in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


def reference(target, tokens, u, draft, lens):
    """One request: p [n + 1.., V], x [K], u [K + 1], q [K, V] or None.  Returns (accepted, row),
    the row that the next token is drawn from (zeros: none)."""
    K, V = len(tokens), target.shape[1]
    u = np.where(u > 0, u, 0).astype(np.float64)
    a = 0
    while a < lens:
        x = int(tokens[a])
        if not 0 <= x < V:
            break
        q = 1.0 if draft is None else float(draft[a, x])
        if not u[a] * q < float(target[a, x]):
            break
        a += 1
    p = target[a].astype(np.float64)
    r = np.maximum(p, 0)
    if a < lens:
        if draft is not None:
            r = np.maximum(p - np.maximum(draft[a].astype(np.float64), 0), 0)
        elif 0 <= tokens[a] < V:
            r[tokens[a]] = 0
        if not r.any():
            r = np.maximum(p, 0)
    return a, r


def check(got, accepted, target, tokens, u, draft, lens):
    """Tokens and counts of one request.  The kernel's sums are exact but for entries below
    2^-31, cut to 2^-54 each; this float64 cumsum of V terms is off by V 2^-53 of the total."""
    a, r = reference(target, tokens, u, draft, lens)
    K = len(tokens)
    assert accepted == a
    assert (got[:a] == tokens[:a]).all()
    assert (got[a + 1:] == -1).all()
    V = len(r)
    total = r.sum()
    if total == 0:
        assert got[a] == -1
        return
    tok = int(got[a])
    assert 0 <= tok < V and r[tok] > 0
    c = np.cumsum(r)
    slack = V * 2.0 ** -53 * total + V * 2.0 ** -54
    v = float(u[K])
    if v >= 1:
        assert tok == np.nonzero(r)[0][-1]
        return
    t = (v if v > 0 else 0.0) * c[-1]
    assert c[tok] > t - slack and (tok == 0 or c[tok - 1] <= t + slack), (tok, t)


def make(B, K, V, dtype, lookup, ragged, flat, pad, seed, sharp=3.0):
    """Inputs on the device, and the host's copies of them."""
    g = torch.Generator().manual_seed(seed)
    lens = (torch.randint(0, K + 1, (B,), generator=g) if ragged
            else torch.full((B,), K)).int()
    rows = lens + 1 if flat else torch.full((B,), K + 1).int()
    starts = torch.cat([torch.zeros(1), torch.cumsum(rows, 0)]).int()
    T = int(starts[-1])
    z = torch.randn((T, V), generator=g) * sharp
    p = torch.zeros((T, V + pad))
    p[:, :V] = torch.softmax(z, 1)
    p = p.to(dtype)
    q = torch.zeros((B, K, V + pad), dtype=dtype)
    x = torch.zeros((B, K), dtype=torch.int32)
    for b in range(B):
        for i in range(K):
            t = int(starts[b]) + min(i, int(rows[b]) - 1)
            q[b, i, :V] = torch.softmax(z[t] + torch.randn(V, generator=g), 0).to(dtype)
            x[b, i] = torch.multinomial(q[b, i, :V].float() + 1e-30, 1, generator=g)
    u = torch.rand((B, K + 1), generator=g)
    host = dict(p=p[:, :V].float().numpy(), q=None if lookup else q[:, :, :V].float().numpy(),
                x=x.numpy(), u=u.numpy(), lens=lens.numpy(), starts=starts.numpy())
    dp = p.cuda()[:, :V]
    if not flat:
        dp = p.cuda().view(B, K + 1, V + pad)[:, :, :V]
    args = dict(target_probs=dp, draft_tokens=x.cuda(), uniforms=u.cuda(),
                draft_probs=None if lookup else q.cuda()[:, :, :V],
                draft_lens=lens.cuda(), starts=starts.cuda() if flat else None)
    return args, host


def check_all(out, host):
    tok, acc = out[0].cpu().numpy(), out[1].cpu().numpy()
    for b in range(len(acc)):
        p = host["p"][host["starts"][b]:host["starts"][b + 1]]
        check(tok[b], acc[b], p, host["x"][b], host["u"][b],
              None if host["q"] is None else host["q"][b], int(host["lens"][b]))


def sampler(B, V):
    from device_token_sampling_gb300 import Sampler
    return Sampler(max_batch=B, max_vocab=V)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("B,K,V,pad,flat", [
    (1, 1, 1, 0, False), (1, 1, 7, 0, True), (3, 2, 128, 0, True), (2, 5, 1000, 24, False),
    (5, 3, 4099, 13, True), (1, 7, 32003, 0, False), (4, 4, 50000, 16, True),
    (700, 2, 513, 0, True), (2, 40, 300, 4, False), (1, 2, 151936, 0, False)])
def test_against_reference(B, K, V, pad, flat, lookup, dtype):
    for seed in range(2):
        args, host = make(B, K, V, dtype, lookup, seed == 0, flat, pad, seed * 100 + V)
        with sampler(B, V) as s:
            out = s.verify(**args)
            status = s.row_status(B)
            s.check_device_errors()
        check_all(out, host)
        assert (status == 0).all()


@gpu
def test_large_vocabulary_bounds_of_the_draw():
    """u at both ends, and where a row's mass is in one place only."""
    V = 248320
    p = torch.zeros((4, 1, V), device="cuda")
    p[0, 0, 7], p[0, 0, V - 1] = 0.5, 0.5
    p[1, 0, V - 2] = 1.0
    p[2] = 1.0 / V
    p[3, 0, 5] = 2.0 ** -40
    p[3, 0, 100000] = 2.0 ** -41
    x = torch.zeros((4, 0), dtype=torch.int32, device="cuda")
    top = 1 - 2.0 ** -24
    with sampler(4, V) as s:
        for u, want in ((0.0, [7, V - 2, 0, 5]), (top, [V - 1, V - 2, V - 1, 100000]),
                        (1.0, [V - 1, V - 2, V - 1, 100000]), (5.0, [V - 1, V - 2, V - 1, 100000]),
                        (float("nan"), [7, V - 2, 0, 5]), (-1.0, [7, V - 2, 0, 5]),
                        (0.5, [V - 1, V - 2, V // 2, 5]),
                        (0.75, [V - 1, V - 2, V // 4 * 3, 100000])):
            tok, acc = s.verify(p, x, torch.full((4, 1), u, device="cuda"))
            assert tok[:, 0].tolist() == [w if r != 2 else tok[2, 0].item()
                                          for r, w in enumerate(want)], u
            # 1 / V is rounded to 24 bits: V equal masses, exact in any order
            assert abs(tok[2, 0].item() - want[2]) <= 1
            assert (acc == 0).all()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_edges(dtype):
    """Equal rows, no mass, values that are no probabilities, tokens outside the vocabulary."""
    V, K = 2000, 2
    g = torch.Generator().manual_seed(5)
    base = torch.softmax(torch.randn((V,), generator=g) * 2, 0).to(dtype)
    B = 12
    p = base.expand(B, K + 1, V).clone()
    q = base.expand(B, K, V).clone()
    x = torch.full((B, K), 11, dtype=torch.int32)
    u = torch.full((B, K + 1), 0.5)
    lens = torch.full((B,), K, dtype=torch.int32)
    p[0, 0, 11] = 0                       # refused; nothing left of p - q elsewhere: from p
    q[0, 0, 11] = base[11]
    p[1] = 0                              # no mass at all
    p[2, 0, 5] = float("nan")             # refused by x, and its row holds a NaN
    p[2, 0, 11] = 0
    p[3, 0, 5] = float("inf")
    p[3, 0, 11] = 0
    q[4, 0, 5] = float("nan")
    p[4, 0, 11] = 0
    x[5, 0] = -1                          # no such token
    x[6, 1] = V
    p[7, 0, 11] = float("nan")            # compares with nothing: refused
    lens[8] = -3
    lens[9] = 1000
    u[10, 0] = float("nan")
    p[11, 0, 3] = -0.25                   # below 0 counts as 0
    p[11, 0, 11] = 0
    with sampler(B, V) as s:
        tok, acc = s.verify(p.cuda(), x.cuda(), u.cuda(), draft_probs=q.cuda(),
                            draft_lens=lens.cuda())
        status = s.row_status(B).tolist()
    tok, acc = tok.cpu().numpy(), acc.cpu().numpy()
    assert status == [0, 2, 1, 1, 1, 0, 0, 1, 0, 0, 0, 0]
    for b in range(B):
        n = min(max(int(lens[b]), 0), K)
        if status[b] == 1:
            assert acc[b] == 0 and (tok[b] == -1).all()
            continue
        check(tok[b], acc[b], p[b].float().numpy(), x[b].numpy(), u[b].numpy(),
              q[b].float().numpy(), n)


@gpu
def test_sums_that_are_no_distribution():
    """A row that sums to 512 and more is refused by its status, not drawn from wrongly."""
    V = 1 << 20
    p = torch.full((1, 1, V), 1.9, device="cuda")
    x = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    u = torch.full((1, 1), 0.5, device="cuda")
    with sampler(1, V) as s:
        tok, _ = s.verify(p, x, u)
        assert tok.item() == -1 and s.row_status(1).item() == 1
        p.fill_(2.0 ** -13)                # 128 in all: fine
        tok, _ = s.verify(p, x, u)
        assert tok.item() == V // 2 and s.row_status(1).item() == 0


@gpu
def test_starts():
    """Rows by starts: requests without rows, fewer rows than drafts, rows that are not there."""
    V, K, B = 600, 3, 6
    g = torch.Generator().manual_seed(2)
    p = torch.softmax(torch.randn((8, V), generator=g), 1)
    x = p[:1].argmax(1).int().expand(B, K).contiguous()
    starts = torch.tensor([0, 4, 4, 6, 5, 9, 9], dtype=torch.int32)
    u = torch.full((B, K + 1), 0.25)
    u[:, :K] = 0
    with sampler(B, V) as s:
        tok, acc = s.verify(p.cuda(), x.cuda(), u.cuda(), starts=starts.cuda())
        status = s.row_status(B).tolist()
    # request 1: no rows; 3: decreasing; 4: rows 5..8 of 8; 5: no rows
    assert status == [0, 2, 0, 2, 2, 2]
    tok, acc = tok.cpu().numpy(), acc.cpu().numpy()
    for b, n in ((0, 3), (2, 1)):
        check(tok[b], acc[b], p[int(starts[b]):int(starts[b + 1])].numpy(), x[b].numpy(),
              u[b].numpy(), None, n)
    assert acc.tolist() == [3, 0, 1, 0, 0, 0]
    assert (tok[[1, 3, 4, 5]] == -1).all()


@gpu
@pytest.mark.parametrize("lookup", [False, True])
def test_the_tokens_have_the_targets_distribution(lookup):
    """First tokens of 200,000 requests: counts within 6 standard deviations of the target's."""
    B, V = 1 << 14, 7
    g = torch.Generator(device="cuda").manual_seed(3)
    p = torch.softmax(torch.randn(V, generator=g, device="cuda") * 1.2, 0)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda") * 1.2, 0)
    counts = torch.zeros(V, device="cuda")
    with sampler(B, V) as s:
        for _ in range(12):
            if lookup:
                x = torch.full((B, 1), 2, dtype=torch.int32, device="cuda")
            else:
                x = torch.multinomial(q, B, replacement=True, generator=g).int()[:, None]
            u = torch.rand((B, 2), generator=g, device="cuda")
            tok, _ = s.verify(p.expand(B, 2, V).contiguous(), x.contiguous(), u,
                              draft_probs=None if lookup else q.expand(B, 1, V).contiguous())
            counts += torch.bincount(tok[:, 0].long(), minlength=V)
    n = 12 * B
    sd = (n * p * (1 - p)).sqrt()
    assert ((counts - n * p).abs() <= 6 * sd).all(), (counts / n, p)


@gpu
def test_strides_streams_graphs():
    """Strided rows, a stream of the caller's, and a captured call replayed on new inputs."""
    B, K, V = 4, 3, 5000
    args, host = make(B, K, V, torch.float32, False, True, False, 8, 1)
    wide = torch.zeros((K + 1, B, V + 8), device="cuda")   # step-major rows
    wide[:, :, :V] = args["target_probs"].transpose(0, 1)
    drafts = torch.zeros((K, B, V + 8), device="cuda")
    drafts[:, :, :V] = args["draft_probs"].transpose(0, 1)
    args["target_probs"] = wide.transpose(0, 1)[:, :, :V]
    args["draft_probs"] = drafts.transpose(0, 1)[:, :, :V]
    with sampler(B, V) as s:
        check_all(s.verify(**args), host)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        out = s.verify(**args, stream=side)
        side.synchronize()
        check_all(out, host)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.verify(**args)
        new, host2 = make(B, K, V, torch.float32, False, True, False, 8, 9)
        for k in ("target_probs", "draft_probs", "draft_tokens", "uniforms", "draft_lens"):
            args[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        check_all(out, host2)


@gpu
def test_refusals():
    from device_token_sampling_gb300 import VtError
    B, K, V = 2, 2, 100
    args, _ = make(B, K, V, torch.float32, False, False, False, 0, 0)
    with sampler(B, V) as s:
        def bad(error=ValueError, **change):
            with pytest.raises(error):
                s.verify(**{**args, **change})

        bad(target_probs=args["target_probs"].half())
        bad(target_probs=args["target_probs"][:, :K])
        bad(target_probs=args["target_probs"].cpu())
        bad(target_probs=args["target_probs"].transpose(1, 2).contiguous().transpose(1, 2))
        bad(draft_probs=args["draft_probs"].bfloat16())
        bad(draft_probs=args["draft_probs"][:, :1])
        bad(draft_tokens=args["draft_tokens"].long())
        bad(draft_tokens=args["draft_tokens"][0])
        bad(uniforms=args["uniforms"][:, :K])
        bad(uniforms=args["uniforms"].double())
        bad(draft_lens=args["draft_lens"].long())
        bad(starts=torch.zeros(B + 1, dtype=torch.int32, device="cuda"))     # 3-D target
        bad(out=(torch.empty((B, K), dtype=torch.int32, device="cuda"),
                 torch.empty(B, dtype=torch.int32, device="cuda")))
    with sampler(1, V) as s:
        bad(VtError)
    with sampler(B, V - 1) as s:
        bad(VtError)
