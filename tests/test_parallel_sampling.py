"""The example's decode loop, each step checked against plain computations on its own tensors."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

from pagedlib import attention_reference
from test_given import reference_row

torch = pytest.importorskip("torch")
EXAMPLES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")


@pytest.mark.gpu
@pytest.mark.parametrize("n,prompt,steps", [(5, 37, 20), (32, 1000, 6), (3, 64, 4), (2, 9, 12)])
def test_loop(n, prompt, steps):
    sys.path.insert(0, EXAMPLES)
    import parallel_sampling as ex
    seen = []

    def watch(s):
        seen.append(s["step"])
        assert (s["status"] == 0).all()
        logits = s["logits"].float().cpu().numpy()
        u = s["uniforms"].cpu().numpy()
        for i in range(n):
            row, v = (logits[0], u[0, i]) if s["step"] == 0 else (logits[i], u[i])
            tok, near, _, _ = reference_row(row, [v], T=0.9, k=200, p=0.95, mp=0.01)
            assert int(s["tokens"][i]) in near[0] | {tok[0]}
        if s["step"] == 0:
            return
        want, wlse, b_out, b_lse = attention_reference(
            s["q"], s["keys"], s["values"], s["table"], s["lens"], s["prefix"],
            s["prefix"].shape[0] * ex.BLOCK, ex.BLOCK, ex.HEAD_DIM ** -0.5)
        assert bool(((s["attended"].double() - want).abs() <= b_out).all())
        assert bool(((s["lse"].double() - wlse).abs() <= b_lse).all())

    tokens = ex.generate(n, prompt, steps, seed=n, watch=watch)
    assert seen == list(range(steps)) and tokens.shape == (n, steps)
    assert len({tuple(r) for r in tokens.tolist()}) == n  # different numbers, different texts
    assert torch.equal(ex.generate(n, prompt, steps, seed=n), tokens)


def test_reference_shares_nothing_with_the_kernels():
    """The references are plain torch and numpy."""
    here = os.path.dirname(os.path.abspath(__file__))
    text = open(os.path.join(here, "pagedlib.py")).read()
    assert "device_token_sampling" not in text
    assert np.isfinite(reference_row(np.zeros(4, np.float32), [0.5])[2][0])
