"""Calls on a stream of their own, while the current stream and that one are both busy: outputs
made by a call lie in no memory that pending work still uses, and inputs live until they are read."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

N = 1 << 22  # elements of the outputs: an allocation of its own


def busy():
    """About 50 ms of products, enqueued on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    for _ in range(60):
        torch.mm(a, a, out=b)
    return b


def make_given():
    from device_token_sampling_gb300 import Sampler
    B, V, draws = 64, 5000, N // 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((B, V), generator=g, device="cuda")
    u = torch.rand((B, draws), generator=g, device="cuda")
    s = Sampler(max_batch=B, max_vocab=V)
    one, zero = np.ones(B), np.zeros(B)
    s.reset_params(one, zero, one, zero, zero, zero, one, np.zeros(B, np.uint64))
    return s, lambda t, stream: s.sample_given(t[0], t[1], stream=stream), (x, u)


def make_tables():
    from device_token_sampling_gb300 import PagedBatch
    B, bs = 64, 16
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = torch.full((B,), 1000, dtype=torch.int32, device="cuda")
    p = PagedBatch(B, bs, 64)
    table = torch.zeros((B, 64), dtype=torch.int32, device="cuda")
    free = torch.arange(B * 64, dtype=torch.int32, device="cuda")
    return (p, lambda i, stream: p.build_tables(table, i[0], i[0], i[1], t(0) if stream is None else
                                                i[2], capacity=N, stream=stream),
            (lens, free, t(0)))


def make_attention():
    from device_token_sampling_gb300 import PagedBatch
    B, hq, d = 1024, 64, 64
    p = PagedBatch(B, 16, 4, hq, hq, d)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((8, 16, hq, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, hq, d), generator=g, device="cuda").bfloat16()
    table = torch.randint(0, 8, (B, 4), generator=g, device="cuda").int()
    lens = torch.full((B,), 20, dtype=torch.int32, device="cuda")
    return (p, lambda i, stream: p.attention(i[0], k, v, i[1], i[2], stream=stream),
            (q, table, lens))


def greedy(B=4096, V=4096, **kw):
    """A sampler whose draws are the same every time, and its logits."""
    from device_token_sampling_gb300 import Sampler
    s = Sampler(max_batch=B, max_vocab=V, **kw)
    one, zero = np.ones(B), np.zeros(B)
    s.reset_params(zero, zero, one, zero, zero, zero, one, np.zeros(B, np.uint64))
    g = torch.Generator(device="cuda").manual_seed(3)
    return s, torch.randn((B, V), generator=g, device="cuda")


def make_sample():
    s, x = greedy(max_logprobs=8)
    return s, lambda i, stream: s.sample(i[0], num_logprobs=8, stream=stream), (x,)


def make_partials():
    s, x = greedy()
    return s, lambda i, stream: (s.shard_partials(i[0], 0, 4096, 32, stream=stream),), (x,)


def make_merge():
    s, x = greedy(max_logprobs=8)
    parts = s.shard_partials(x, 0, 4096, 32)[None]
    return s, lambda i, stream: s.shard_merge(i[0], 4096, 32, 8, stream=stream), (parts,)


CALLS = [make_given, make_tables, make_attention, make_sample, make_partials, make_merge]


@pytest.mark.parametrize("make", CALLS)
def test_outputs_wait_for_pending_work_on_the_current_stream(make):
    """A tensor is freed while a copy of it is still pending on the current stream; the call on
    another stream makes outputs of the same size."""
    handle, call, inputs = make()
    sizes = {t.numel() * t.element_size() for t in call(inputs, None)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    held = [torch.full((n // 4,), 7, dtype=torch.int32, device="cuda") for n in sizes if n >= 1 << 16]
    assert held
    keep = busy()
    copies = [h.clone() for h in held]
    del held
    out = call(inputs, side)
    torch.cuda.synchronize()
    assert keep is not None and out
    for c in copies:
        assert bool((c == 7).all())


@pytest.mark.parametrize("make", CALLS)
def test_inputs_live_until_the_call_has_read_them(make):
    """Inputs that the caller drops at once, with the call still pending on its stream."""
    handle, call, inputs = make()
    want = [t.clone() for t in call(inputs, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        keep = busy()
    temps = [t.clone() for t in inputs]
    shapes = [(t.shape, t.dtype) for t in temps]
    torch.cuda.current_stream().synchronize()
    got = call(temps, side)
    del temps
    over = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]
    torch.cuda.synchronize()
    assert keep is not None and len(over) == len(inputs)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("make", CALLS)
def test_outputs_used_on_the_current_stream_live_until_it_is_done(make):
    """Outputs handed over to the current stream, read there by pending work and dropped; the
    next call on the other stream makes outputs of the same size."""
    handle, call, inputs = make()
    want = [t.clone() for t in call(inputs, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(inputs, side)
    torch.cuda.current_stream().wait_stream(side)
    keep = busy()
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    assert keep is not None and over
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
