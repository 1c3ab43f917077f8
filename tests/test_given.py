"""Draws from given uniform numbers, against the definition in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

EMPTY = dict(T=1.0, k=0, p=1.0, mp=0.0)


def reference_row(x, u, T=1.0, k=0, p=1.0, mp=0.0):
    """One row in float64 from the definition: (tokens, near, logprobs, kept).  ``near[i]`` holds
    the tokens either side when u * W is within 1e-9 of W of a boundary between two."""
    V = len(x)
    greedy = T == 0 or k == 1 or p == 0 or mp == 1
    inv_t = np.float32(1) if greedy else np.float32(1) / np.float32(T)
    with np.errstate(over="ignore"):
        z = (x.astype(np.float32) * inv_t).astype(np.float32).astype(np.float64)
    m = z.max()
    if np.isnan(z).any() or m == np.inf or m == -np.inf:
        return [-1] * len(u), [set()] * len(u), [math.nan] * len(u), 0
    lse = math.log(np.exp(z - m).sum())
    if greedy:
        j = int(np.argmax(z))
        return [j] * len(u), [{j}] * len(u), [-lse] * len(u), 1
    ids = np.nonzero(z > -np.inf)[0]
    if mp > 0:
        ids = ids[z[ids] - m >= math.log(float(np.float32(mp)))]
    order = ids[np.argsort(-z[ids], kind="stable")]
    if 1 < k < V:
        order = order[:k]
    if p < 1:
        c = np.cumsum(np.exp(z[order] - m))
        order = order[np.concatenate([[0.0], c[:-1]]) <= float(np.float32(p)) * c[-1]]
    kept = np.sort(order)
    c = np.cumsum(np.exp(z[kept] - m))
    tok, near, lp = [], [], []
    for v in u:
        v = float(v)
        v = 0.0 if not v > 0 else min(v, 1 - 2.0 ** -40)
        t = v * c[-1]
        pick = [int(kept[min(np.searchsorted(c, t + e, side="right"), len(kept) - 1)])
                for e in (0.0, -1e-9 * c[-1], 1e-9 * c[-1])]
        tok.append(pick[0])
        near.append(set(pick))
        lp.append(z[pick[0]] - m - lse)
    return tok, near, lp, len(kept)


def run(x, u, rows, V=None, stream=None, check=True, **kw):
    """x [B, ld] float32 or bf16 CUDA tensor, rows: B dicts of parameters."""
    from device_token_sampling_gb300 import Sampler
    B = x.shape[0]
    V = V or x.shape[1]
    a = {n: np.array([{**EMPTY, **r}[n] for r in rows]) for n in ("T", "k", "p", "mp")}
    s = Sampler(max_batch=B, max_vocab=V)
    s.reset_params(a["T"], a["k"], a["p"], a["mp"], np.zeros(B), np.zeros(B), np.ones(B),
                   np.zeros(B, np.uint64))
    tok, lp = s.sample_given(x, u, V=V, stream=stream, **kw)
    torch.cuda.synchronize()
    s.check_device_errors()
    st = s.row_status(B).cpu().numpy()
    if check:
        xs, us = x[:, :V].float().cpu().numpy(), u.cpu().numpy().reshape(B, -1)
        t, l = tok.cpu().numpy().reshape(B, -1), lp.cpu().numpy().reshape(B, -1)
        for r in range(B):
            want, near, wlp, kept = reference_row(xs[r], us[r], **{**EMPTY, **rows[r]})
            for i in range(us.shape[1]):
                assert t[r, i] == want[i] or t[r, i] in near[i], (r, i, t[r, i], want[i], rows[r], kept)
                if want[i] < 0:
                    assert np.isnan(l[r, i]) and st[r] in (1, 2)
                elif t[r, i] == want[i]:
                    # fp32: the difference and the logarithm round once each (half a unit at
                    # their size), the sum of V exponentials by at most 2^-22 each, the exponent
                    # of each by 2^-23 of |z - m|, which the weights keep near ln V + its value
                    tol = 2.0 ** -23 * (abs(wlp[i]) * 3 + 2 * math.log(V + 1) + 40)
                    assert abs(l[r, i] - wlp[i]) <= tol, (r, i, l[r, i], wlp[i], tol)
                    assert st[r] == 0
    return tok, lp, st


def logits(seed, B, ld, dtype, sigma=1.5, raised=8):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((B, ld), generator=g, device="cuda") * sigma
    n = min(raised, ld)
    z.scatter_add_(1, torch.randint(0, ld, (B, n), generator=g, device="cuda"),
                   8 + 4 * torch.rand((B, n), generator=g, device="cuda"))
    return z.to(dtype)


def uniforms(seed, B, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 99)
    return torch.rand((B, n), generator=g, device="cuda")


ROWS = [dict(T=0.0), dict(T=0.7, k=40), dict(T=1.3, p=0.9), dict(T=1.0, k=50, p=0.95, mp=0.05),
        dict(T=0.9), dict(T=1.1, mp=0.02), dict(k=1), dict(T=0.3, p=0.5), dict(T=1.5, k=1000, p=0.99),
        dict(p=0.0), dict(mp=1.0), dict(T=0.8, k=2), dict(T=1.0, k=3000, p=0.97), dict(T=2.0, p=0.999)]


def test_reference_by_hand():
    """The reference, on three tokens of masses 1/2, 1/4, 1/4 and hand-worked numbers."""
    x = np.log(np.array([1.0, 2.0, 1.0], np.float32)).astype(np.float32)
    assert reference_row(x, [0.0, 0.2, 0.26, 0.74, 0.76, 0.999])[0] == [0, 0, 1, 1, 2, 2]
    assert reference_row(x, [0.1, 0.4], k=2)[0] == [0, 1]       # the tie goes to index 0
    assert reference_row(x, [0.9], p=0.4)[0] == [1]
    assert reference_row(x, [0.9], T=0.0)[0] == [1]


def test_null_and_state():
    from device_token_sampling_gb300 import sampler
    lib = sampler.load_library()
    assert lib.vt_sample_given(None, None, 0, 1, 1, 1, None, 1, None, None,
                               None) == sampler.VT_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld", [(1, 1), (2, 8), (3, 3), (511, 511), (512, 512), (513, 520),
                                  (1000, 1000), (4097, 4104), (32003, 32003), (50257, 50264),
                                  (151936, 151936), (248320, 248320)])
def test_every_kind_of_row(dtype, V, ld):
    B = len(ROWS)
    x = logits(V, B, ld, dtype)
    if ld > V:
        x[:, V:] = float("nan")
    run(x, uniforms(V, B, 3), ROWS, V=V)


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(1 << 20, torch.bfloat16), (1 << 20, torch.float32),
                                     (600001, torch.float32)])
def test_large_vocabulary(V, dtype):
    """Rows that no cluster's shared memory holds, read again from global memory."""
    rows = [ROWS[1], ROWS[2], ROWS[4], ROWS[12], ROWS[0]]
    run(logits(3, 5, V, dtype), uniforms(3, 5, 2), rows)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 2, 37, 76, 153, 300])
def test_batch_sizes(B):
    """Every cluster size."""
    rows = [ROWS[i % len(ROWS)] for i in range(B)]
    run(logits(B, B, 20000, torch.bfloat16), uniforms(B, B, 1), rows)


@pytest.mark.gpu
@pytest.mark.parametrize("draws", [1, 2, 16, 17, 1000, 65536])
def test_draw_counts(draws):
    rows = [ROWS[2], ROWS[4], ROWS[1], ROWS[0]]
    tok, _, _ = run(logits(draws, 4, 3001, torch.float32), uniforms(draws, 4, draws), rows,
                    check=draws <= 1000)
    if draws > 1000:
        # u = (i + 1/2) / n steps through the distribution: every token as often as its share
        x = logits(draws, 4, 3001, torch.float32)
        u = ((torch.arange(draws, device="cuda") + 0.5) / draws).expand(4, -1).contiguous()
        tok, _, _ = run(x, u, rows, check=False)
        assert bool((tok[1].diff() >= 0).all())
        share = torch.softmax((x[1] * float(np.float32(1) / np.float32(0.9))).double(), 0)
        got = torch.bincount(tok[1].long(), minlength=3001).double()
        assert float((got - share * draws).abs().max()) <= 1.5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_flat_and_steep_rows(dtype):
    """Rows of equal values, of two values, of few values many times; one column alone; a row
    whose masses all but one underflow; a row 60 below its maximum."""
    V = 9000
    x = torch.zeros((8, V), dtype=dtype, device="cuda")
    x[1] = torch.arange(V, device="cuda") % 2
    x[2] = (torch.arange(V, device="cuda") % 7).to(dtype)
    x[3] = -60000.0
    x[3, 777] = 5.0
    x[4] = -60.0
    x[4, 8999] = 0.0
    x[5] = float("-inf")
    x[5, 1234] = -3.0
    x[6] = float("-inf")
    x[6, 100:140] = 2.0
    x[7] = -0.0
    x[7, ::3] = 0.0
    u = uniforms(5, 8, 9)
    u[:, 0], u[:, 1], u[:, 2] = 0.0, 1 - 2.0 ** -24, 0.5
    for kind in (dict(), dict(k=17), dict(p=0.3), dict(k=4000, p=0.7), dict(mp=0.4), dict(T=0.01),
                 dict(T=50.0, k=100), dict(k=8999), dict(k=V), dict(T=0.6, k=33, p=0.5, mp=0.1)):
        run(x, u, [kind] * 8)


@pytest.mark.gpu
def test_masked_columns_and_broken_rows():
    """-inf columns are never drawn; NaN and +inf rows, rows of -inf give no token."""
    V = 5000
    x = logits(1, 9, V, torch.float32)
    x[0, ::2] = float("-inf")
    x[1, 4321] = float("nan")
    x[2, 0] = float("inf")
    x[3] = float("-inf")
    x[4, 1:] = float("-inf")
    x[5, :-1] = float("-inf")
    x[6] = 3.0e38                               # overflows at T = 0.5
    x[7] *= 1e30
    u = uniforms(1, 9, 4)
    for kind in (dict(T=0.5), dict(T=0.5, k=3000), dict(T=0.5, p=0.9), dict(T=0.0)):
        _, _, st = run(x, u, [kind] * 9)
        assert st.tolist()[1:4] == [1, 1, 2]


@pytest.mark.gpu
def test_uniforms_outside_and_on_the_edges():
    x = logits(2, 2, 700, torch.float32)
    u = torch.tensor([[0.0, -1.0, float("nan"), 1e-30, 1e-44, float("-inf")],
                      [1.0, 7.0, float("inf"), 1 - 2.0 ** -24, 2.0 ** -24, 0.5]], device="cuda")
    tok, _, _ = run(x, u, [dict(p=0.9)] * 2)
    t = tok.cpu().numpy()
    assert (t[0] == t[0, 0]).all() and (t[1, :4] == t[1, 0]).all()


@pytest.mark.gpu
def test_top_p_boundary():
    """Prefix ratios 1e-6 either side of p: the kept set, read off by u next to 1 and by the set
    of tokens that a ladder of u reaches."""
    V = 64
    x = torch.full((1, V), -30.0, device="cuda")
    w = np.array([0.5, 0.25, 0.125, 0.0625, 0.0625])
    x[0, [9, 3, 30, 20, 50]] = torch.tensor(np.log(w), dtype=torch.float32, device="cuda")
    u = ((torch.arange(4096, device="cuda") + 0.5) / 4096)[None]
    for p, kept in ((0.749999, {9, 3}), (0.750001, {9, 3, 30}), (0.874999, {9, 3, 30}),
                    (0.875001, {9, 3, 30, 20}), (0.4, {9})):
        tok, _, _ = run(x, u, [dict(p=p)])
        assert set(tok[0].tolist()) == kept, p


@pytest.mark.gpu
def test_shapes_streams_graph_and_repeats():
    from device_token_sampling_gb300 import Sampler
    B, V = 24, 30000
    x, u = logits(4, B, V, torch.bfloat16), uniforms(4, B, 1)
    rows = [ROWS[i % len(ROWS)] for i in range(B)]
    tok, lp, _ = run(x, u, rows)
    tok1, lp1, _ = run(x, u[:, 0].contiguous(), rows)
    assert tok1.shape == (B,) and torch.equal(tok1, tok[:, 0]) and torch.equal(lp1, lp[:, 0])
    # the same bits as int16, unaligned rows, another stream
    odd = torch.empty((B, V + 1), dtype=torch.bfloat16, device="cuda")[:, 1:]
    odd.copy_(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t2, l2, _ in (run(x.view(torch.int16), u, rows, check=False),
                      run(odd, u, rows, check=False), run(x, u, rows, check=False, stream=s)):
        assert torch.equal(t2, tok) and torch.equal(l2, lp)
    smp = Sampler(max_batch=B, max_vocab=V)
    a = {n: np.array([{**EMPTY, **r}[n] for r in rows]) for n in ("T", "k", "p", "mp")}
    smp.reset_params(a["T"], a["k"], a["p"], a["mp"], np.zeros(B), np.zeros(B), np.ones(B),
                     np.zeros(B, np.uint64))
    out = (torch.empty_like(tok), torch.empty_like(lp))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        smp.sample_given(x, u, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], tok) and torch.equal(out[1], lp)
    u.copy_(1 - u)
    g.replay()
    torch.cuda.synchronize()
    t3, l3 = smp.sample_given(x, u)
    assert torch.equal(out[0], t3) and torch.equal(out[1], l3) and not torch.equal(t3, tok)
    # the seeds stay, and sample() works on as before
    assert (smp.seeds(B) == 0).all()
    no_lp, none = smp.sample_given(x, u, out=(torch.empty_like(tok), None))
    assert none is None and torch.equal(no_lp, t3)


@pytest.mark.gpu
def test_refusals():
    from device_token_sampling_gb300 import Sampler, VtError, sampler
    x, u = logits(5, 4, 1000, torch.float32), uniforms(5, 4, 2)
    one, zero, none = np.ones(4), np.zeros(4), np.zeros(4, np.int32)
    s = Sampler(max_batch=4, max_vocab=1000, max_history=8)
    with pytest.raises(VtError) as e:
        s.sample_given(x, u)
    assert e.value.code == sampler.VT_ERR_STATE
    s.reset_params(one[:3], none[:3], one[:3], zero[:3], zero[:3], zero[:3], one[:3],
                   np.zeros(3, np.uint64))
    with pytest.raises(VtError) as e:
        s.sample_given(x, u)
    assert e.value.code == sampler.VT_ERR_STATE
    for pen, decay in ((0.5, None), (0.0, 0.9 * one)):
        s.reset_params(one, none, 0.9 * one, zero, pen * one, zero, one, np.zeros(4, np.uint64),
                       top_p_decay=decay)
        with pytest.raises(VtError) as e:
            s.sample_given(x, u)
        assert e.value.code == sampler.VT_ERR_INVALID_ARG
    s.reset_params(one, none, one, zero, zero, zero, one, np.zeros(4, np.uint64))
    s.sample_given(x, u)
    big = logits(5, 4, 1001, torch.float32)
    with pytest.raises(VtError) as e:
        s.sample_given(big, u)
    assert e.value.code == sampler.VT_ERR_CAPACITY
    with pytest.raises(VtError) as e:
        s.sample_given(x, torch.empty((4, 0), device="cuda"))
    assert e.value.code == sampler.VT_ERR_INVALID_ARG
    for args, kw in (((x.half(), u), {}), ((x[0], u), {}), ((x.cpu(), u), {}), ((x.T, u), {}),
                     ((x, u.double()), {}), ((x, u.cpu()), {}), ((x, u[:3]), {}),
                     ((x, u.T.contiguous().T), {}), ((x, u), dict(V=1001)),
                     ((x, u), dict(out=(u, u))),
                     ((x, u), dict(out=(torch.empty((4, 1), dtype=torch.int32, device="cuda"),
                                        None)))):
        with pytest.raises(ValueError):
            s.sample_given(*args, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("B,V", [(1, 151936), (3, 40000), (5, 5000), (160, 9000)])
def test_top_p_of_half_precision_rows_with_many_equal_values(B, V):
    """bf16 rows of few patterns under top-p: the boundary falls among equal elements, within a
    segment and between two, on values of either sign and among the tiny ones; temperatures that
    make patterns equal."""
    g = torch.Generator(device="cuda").manual_seed(B + V)
    x = torch.empty((B, V), dtype=torch.bfloat16, device="cuda")
    for r in range(B):
        n = torch.randint(0, 7, (V,), generator=g, device="cuda")
        if r % 5 == 0:
            x[r] = n.to(torch.bfloat16) - 3                     # seven values
        elif r % 5 == 1:
            x[r] = (n - 3).float() * 2.0 ** -14                 # all tiny
            x[r, ::3] = 1.5
        elif r % 5 == 2:
            x[r] = -1.0 - (n % 2).float() / 128                 # two neighbouring patterns below 0
        elif r % 5 == 3:
            x[r] = torch.where(torch.arange(V, device="cuda") < 2048, 2.0, -8.0)
        else:
            x[r] = torch.where(n < 3, 0.5, -100.0 * n.float())  # spread over many octaves
    u = uniforms(B, B, 5)
    u[:, 0], u[:, 1] = 1 - 2.0 ** -24, 0.0
    for kind in (dict(p=0.31), dict(p=0.77), dict(p=0.999), dict(p=1e-4), dict(T=0.7, p=0.6),
                 dict(T=20.0, p=0.9), dict(T=1e30, p=0.45), dict(T=1e-3, p=0.45),
                 dict(p=0.6, mp=0.2), dict(p=0.6, k=2000)):
        run(x, u, [kind] * B)
