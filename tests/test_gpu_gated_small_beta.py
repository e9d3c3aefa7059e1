"""dbeta of tokens that write nothing (beta = 0) or next to nothing, from small
gradients: those of a mean over many tokens.

Tolerance as in test_gpu_gated.py: up to twelve roundings to bf16, 2^-7 of the
two-norm, of all tokens and of those with a small beta by themselves. Every gradient
is linear in dout, so that its scale (a power of two) changes nothing in it.
"""

import numpy as np
import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import to_dev, to_host
from oracle import gated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [0, -30, -60, -90])
@pytest.mark.parametrize("heads, d", [(3, 128), (4, 64), (24, 128)])
def test_small_beta(heads, d, power):
    N, r = 320, np.random.default_rng(heads + d)
    q, k = [x / np.linalg.norm(x, axis=-1, keepdims=True) for x in r.normal(size=(2, 1, heads, N, d))]
    g = -np.exp(r.uniform(-5, 0, size=(heads, 1))) * np.log1p(np.exp(r.normal(size=(1, heads, N))))
    beta = 1 / (1 + np.exp(-r.normal(size=(1, heads, N))))
    small = r.uniform(size=beta.shape) < 0.3
    beta[small] = r.choice([0.0, 0.0, 1e-38, -1e-20, 1e-12, 1e-9, 1e-6], size=int(small.sum()))
    dev = [to_dev(x.astype(np.float32), "bf16") for x in (q, k, r.normal(size=q.shape))]
    dev += [to_dev(x.astype(np.float32), "f32") for x in (g, beta)]
    do = to_dev(r.normal(size=q.shape).astype(np.float32), "bf16")
    want = gated.backward(*[to_host(x)[:, :3] for x in dev], to_host(do)[:, :3], d ** -0.5)
    got = la.backward_gated_delta(*dev, do * 2.0 ** power)
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        x = to_host(x)[:, :3] * 2.0 ** -power
        assert np.linalg.norm(x - y) <= 2.0 ** -7 * np.linalg.norm(y), name
        if name == "dbeta":
            x, y = x[small[:, :3]], y[small[:, :3]]
            assert np.linalg.norm(x - y) <= 2.0 ** -7 * np.linalg.norm(y)
