"""Gated delta rule, bf16 rows, where sums cancel: keys (and queries) that share a
direction, values that the state predicts, slow forgetting; gradients that come from
the last tokens alone.

Tolerances. What a value of fp32 arithmetic carries in the end is its rounding to
bf16, 2^-8 / sqrt(3) = 2.3e-3 of a two-norm. Operands of every product before it are two
bf16 parts, off by 2^-16 of themselves; where a sum's terms are up to a hundred times the
sum, 1.5e-3 of it. Together under 2^-8. States are the sum of those products without
the rounding: 2^-15 of their two-norm, for terms that are twice it (with
independent keys 1e-5, test_gpu_gated.py).
"""

import numpy as np
import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import to_dev, to_host
from oracle import gated

pytestmark = pytest.mark.gpu

ROUNDED, STATE = 2.0 ** -8, 2.0 ** -15


def near(got, want, tol, name):
    err, size = np.linalg.norm(got - want), np.linalg.norm(want)
    assert np.isfinite(got).all() and err <= tol * size, f"{name}: {err / max(size, 1e-300):.2e} of the two-norm, {tol:.1e} allowed"


def alike(H, N, dk, dv, common, slow, queries, values, seed):
    """Unit keys with `common` times a shared direction in them (1, 3, 10: cosines
    of 1/2, 0.9, 0.99), queries too or not; values around one of their own, or at random."""
    r = np.random.default_rng(seed)
    shared = r.normal(size=(1, H, 1, dk))
    q = r.normal(size=(1, H, N, dk)) + (common * shared if queries else 0)
    k = r.normal(size=(1, H, N, dk)) + common * shared
    q, k = [x / np.linalg.norm(x, axis=-1, keepdims=True) for x in (q, k)]
    v = r.normal(size=(1, H, N, dv)) * (0.1 if values else 1) + (r.normal(size=(1, H, 1, dv)) if values else 0)
    if slow:
        g, beta = np.full((1, H, N), -1e-3), 1 - 0.01 * r.uniform(size=(1, H, N))
    else:
        g = -np.exp(r.uniform(-5, 0, size=(H, 1))) * np.log1p(np.exp(r.normal(size=(1, H, N))))
        beta = 1 / (1 + np.exp(-r.normal(size=(1, H, N))))
    dev = [to_dev(x.astype(np.float32), "bf16") for x in (q, k, v)] + [to_dev(x.astype(np.float32), "f32") for x in (g, beta)]
    return dev, r


CASES = [(0, False, False, False), (0, True, False, False), (1, False, False, False), (3, False, False, False), (3, True, True, False),
         (10, False, True, False), (10, True, True, False), (3, True, False, True), (10, True, True, True)]
SIZES = [(3, 320, 128, 128), (5, 200, 64, 64), (3, 150, 64, 128), (50, 260, 128, 128), (80, 260, 128, 128), (160, 130, 64, 64), (90, 140, 128, 64)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, case):
    H, N, dk, dv = size
    dev, r = alike(H, N, dk, dv, *case, seed=N + dk)
    some = [0, H // 2, H - 1]
    want, S_want = gated.forward(*[to_host(x)[:, some] for x in dev], dk ** -0.5)
    out, S = la.forward_gated_delta(*dev, return_state=True)
    near(to_host(out)[:, some], want, ROUNDED, "out")
    near(to_host(S)[:, some], S_want, STATE, "state")
    # a state that is asked for changes no output
    assert torch.equal(la.forward_gated_delta(*dev), out)
    # packed: two sequences are each as by themselves
    at = (0, 70, N)
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    want, S_want = gated.forward(*[to_host(x)[:, some] for x in dev], dk ** -0.5, None, at)
    out, S = la.forward_gated_delta(*dev, offsets=off, return_state=True)
    near(to_host(out)[:, some], want, ROUNDED, "packed out")
    near(to_host(S)[:, some], S_want, STATE, "packed state")
