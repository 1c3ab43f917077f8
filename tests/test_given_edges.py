"""Draws from given uniform numbers where logits are large, flat or far apart, against the
definition in 64 bits of ``test_given``."""
from __future__ import annotations

import os

import numpy as np
import pytest

from test_given import EMPTY, ROWS, logits, run, uniforms

torch = pytest.importorskip("torch")

F32_MIN = float(np.finfo(np.float32).min)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [5000, 40000, 151936])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_flat_rows_of_large_magnitude(dtype, V):
    """Every logit at one value whose neighbours are further away than a histogram bin: a mask's
    fill value, the type's lowest number.  Top-k takes the lowest indices."""
    values = [-1e9, F32_MIN if dtype == torch.float32 else float(torch.finfo(dtype).min), 1e6,
              -65504.0, 2.0 ** 17, 2.0 ** 17 + 1024.0, -2.0 ** 24, 3e38]
    x = torch.empty((len(values), V), dtype=dtype, device="cuda")
    for r, v in enumerate(values):
        x[r] = v
    u = uniforms(V, len(values), 4)
    u[:, 0], u[:, 1] = 0.0, 1 - 2.0 ** -24
    for kind in (dict(k=50), dict(k=2), dict(k=30, p=0.5), dict(k=20, mp=0.1), dict(k=1000),
                 dict(T=0.7, k=20), dict(T=1.5, k=20)):
        tok, _, st = run(x, u, [kind] * len(values))
        ok = torch.from_numpy(st == 0).cuda()
        assert bool(ok.any())
        assert bool(((tok >= 0) & (tok < kind["k"]))[ok].all())


@pytest.mark.gpu
@pytest.mark.parametrize("at", [1e6, -1e6, 2.0 ** 17, 2.0 ** 20])
@pytest.mark.parametrize("T", [1.0, 0.7, 1.5])
def test_neighbouring_values_of_large_magnitude(at, T):
    """Logits a few representable steps apart far from zero: the k-th value is among them, and
    tempering makes neighbours equal, which then go by index."""
    V = 40000
    step = float(np.spacing(np.float32(abs(at))))
    j = torch.arange(V, device="cuda")
    x = torch.empty((4, V), dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(int(abs(at)))
    x[0] = at + step * ((j // 64) % 97)
    x[1] = at + step * (j % 5)
    x[2] = at + step * torch.randint(0, 2000, (V,), generator=g, device="cuda")
    x[3] = at - step * (j // 64)
    u = uniforms(7, 4, 6)
    for kind in (dict(k=50), dict(k=7), dict(k=300, p=0.8), dict(k=100, mp=0.3)):
        run(x, u, [dict(kind, T=T)] * 4)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [3000, 9000, 151936])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_faint_tail(dtype, V):
    """One logit, and all others so far below it that each has next to no mass while a stretch of
    them has some: numbers at the ends of [0, 1) fall into such stretches.  Every draw is a
    token."""
    x = torch.empty((12, V), dtype=dtype, device="cuda")
    for r, low in enumerate((-36.0, -37.0, -38.0, -40.0)):
        for i, peak in enumerate((0, V // 2, V - 1)):
            x[3 * r + i] = low
            x[3 * r + i, peak] = 0.0
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 1e-30, 0.5], device="cuda").repeat(12, 1)
    for kind in (dict(), dict(T=0.99), dict(p=1 - 2.0 ** -24), dict(mp=1e-30), dict(k=V - 1)):
        tok, _, st = run(x, u, [kind] * 12)
        assert (st == 0).all()
        assert bool(((tok >= 0) & (tok < V)).all()), kind
    # without a filter the first logit has mass of its own: a number of 0 draws the first token
    # wherever a stretch of the tail has any
    tok, _, _ = run(x[:6], u[:6], [dict()] * 6)
    if V == 9000:
        assert bool((tok[:, 0] == 0).all())


class OnDevice:
    """A tensor of another GPU, as far as its attributes go."""
    is_cuda = True

    def __init__(self, shape, index):
        self.shape, self.index, self.dtype = shape, index, torch.float32
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self.shape[1] if i == 0 else 1

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def element_size(self):
        return self.dtype.itemsize


class Stream:
    """The default stream of device 0, as far as its attributes go."""
    cuda_stream, device, device_index = 0, torch.device("cuda", 0), 0


@pytest.fixture
def recorder():
    """A sampler on device 0 whose library only records its calls."""
    from device_token_sampling_gb300 import Sampler
    called = []

    class Lib:
        def vt_sample_given(self, *a):
            called.append(a)
            return 0

    s = Sampler.__new__(Sampler)
    s._lib, s._h, s.device = Lib(), None, 0
    return s, called


def test_tensors_of_another_gpu_are_refused(recorder):
    """Their addresses mean nothing on the handle's device: nothing is called with them."""
    s, called = recorder
    x, u = OnDevice((4, 100), 1), OnDevice((4, 2), 1)
    tok, lp = OnDevice((4, 2), 1), OnDevice((4, 2), 1)
    tok.dtype = torch.int32
    with pytest.raises(ValueError):
        s.sample_given(x, u, out=(tok, lp), stream=Stream())
    assert not called


@pytest.mark.parametrize("have,given", [(torch.bfloat16, 0), (torch.float32, 1), (torch.uint8, 1),
                                        (torch.float16, 0)])
def test_logits_of_another_size_than_the_given_dtype_are_refused(recorder, have, given):
    """A dtype wider than the tensor's elements would read past its end."""
    s, called = recorder
    x, u = OnDevice((4, 100), 0), OnDevice((4, 2), 0)
    x.dtype = have
    tok, lp = OnDevice((4, 2), 0), OnDevice((4, 2), 0)
    tok.dtype = torch.int32
    with pytest.raises(ValueError):
        s.sample_given(x, u, out=(tok, lp), stream=Stream(), dtype=given)
    assert not called


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_waits_that_run_out(dtype, monkeypatch):
    """Every wait for a copy taken as run out: the call is reported and its draws are right, on
    rows that come by copies throughout and on rows with a ragged end, several segments a warp."""
    from device_token_sampling_gb300 import Sampler, VtError, sampler
    for B, V in ((300, 20480), (700, 5000), (1, 4096)):
        x, u = logits(B, B, V, dtype), uniforms(B, B, 3)
        rows = [ROWS[i % len(ROWS)] for i in range(B)]
        tok, lp, _ = run(x, u, rows, check=False)
        monkeypatch.setenv("VT_FAULT_INJECT", "wait")
        s = Sampler(max_batch=B, max_vocab=V)
        monkeypatch.delenv("VT_FAULT_INJECT")
        a = {n: np.array([{**EMPTY, **r}[n] for r in rows]) for n in ("T", "k", "p", "mp")}
        s.reset_params(a["T"], a["k"], a["p"], a["mp"], np.zeros(B), np.zeros(B), np.ones(B),
                       np.zeros(B, np.uint64))
        got, got_lp = s.sample_given(x, u)
        with pytest.raises(VtError) as e:
            s.check_device_errors()
        assert e.value.code == sampler.VT_ERR_TIMEOUT
        s.check_device_errors()
        assert torch.equal(got, tok) and torch.equal(got_lp, lp)


def test_masses_as_modelled():
    """The kernel's mass arithmetic step by step in NumPy (an FMA as a product and a sum in long
    double, rounded once): within half a unit of 2^-30 for each of its two roundings, the cubic
    term that the quadratic leaves out and the error of the reduced argument, 1.1e-9 together; the
    two roundings' variance over mantissas 2^f, f uniform, makes 2.8e-10 rms."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "device_token_sampling_gb300", "csrc", "vt_given.cu")) as f:
        source = f.read()
    for constant in ("x *= 1.0013547198921082", "double x = 1073741824.0", "1.92596303e-8f",
                     "__fmaf_rn(r, 0.240226507f, 0.693147181f)", "kMagic = 12582912.f",
                     "kMagic512 = 24576.f"):
        assert constant in source, constant
    f32, long = np.float32, np.longdouble

    def fma(a, b, c):
        return (a.astype(long) * b.astype(long) + c.astype(long)).astype(f32)

    table, as_float, x = [], [], 1073741824.0
    for _ in range(512):
        table.append(int(x + 0.5))
        bits = ((127 + 30) << 23) + int((x - 1073741824.0) / 128.0 + 0.5)
        as_float.append(np.uint32(bits).view(f32))
        x *= 1.0013547198921082
    table, as_float = np.array(table, np.int64), np.array(as_float, f32)
    g = np.random.default_rng(0)
    for low, high in ((-1, 0), (-40, 0), (20, 30), (-300, -280), (4000, 4800)):
        z = g.uniform(low, high, 400000).astype(f32)
        log2e = np.full_like(z, 1.4426950408889634)
        k = fma(z, log2e, np.full_like(z, 24576)) - f32(24576)
        r = fma(z, log2e, -k)
        r = fma(z, np.full_like(z, 1.92596303e-8), r)
        q = r * fma(r, np.full_like(z, 0.240226507), np.full_like(z, 0.693147181))
        n = np.rint(k.astype(np.float64) * 512).astype(np.int64)
        up = fma(q, as_float[n & 511], np.full_like(z, 12582912)).astype(np.float64) - 12582912
        mantissa = table[n & 511] + up.astype(np.int64)
        exact = np.exp2(z.astype(long) / np.log(long(2)) - (n >> 9))
        error = np.abs(mantissa / (exact * 2.0 ** 30) - 1)
        assert error.max() <= 1.1e-9 and np.sqrt((error ** 2).mean()) <= 3e-10
