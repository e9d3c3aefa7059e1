"""Gated delta rule, bf16 rows, where sums cancel: keys (and queries) that share a
direction, values that the state predicts, slow forgetting; gradients that come from
the last tokens alone.

Tolerances. What a value of fp32 arithmetic carries in the end is its rounding to
bf16, 2^-8 / sqrt(3) = 2.3e-3 of a two-norm. Operands of every product before it are two
bf16 parts, off by 2^-16 of themselves; where a sum's terms are up to a hundred times the
sum, 1.5e-3 of it. Together under 2^-8. dg has larger ones: it is the sum, from its token to the
chunk's end, of q.dq - dv.(v - e) - beta dbeta (S'^T k = v - e) and of one product at the end.
With their magnitudes' sums m, 2600 times dg where keys and queries are nearly equal and the
state predicts the values, the products, off by 2^-18 of their terms in the root mean square
(two parts of 2^-9 each, lo lo left out), put dg off by 2^-18 m beside its rounding: the larger of
that and 2^-8 is allowed. States are the sum of those products without
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


def terms_of_dg(dev, some, want):
    """The two-norm of the sums of the magnitudes of dg's terms, over that of dg."""
    q, k, v, g, beta = [to_host(x)[:, some] for x in dev]
    e = np.stack([t[1] for t in gated.forward(q, k, v, g, beta, q.shape[-1] ** -0.5, keep=True)[2][0]], 1)[None]
    x = np.abs((q * want[0]).sum(-1)) + np.abs((want[2] * (v - e)).sum(-1)) + np.abs(beta * want[4])
    for c in range(0, x.shape[-1], 64):
        x[..., c:c + 64] = x[..., c:c + 64][..., ::-1].cumsum(-1)[..., ::-1]
    return np.linalg.norm(x) / np.linalg.norm(want[3])


def gradients(dev, do, dS, some, scale):
    got = la.backward_gated_delta(*dev, do, dS=dS)
    want = gated.backward(*[to_host(x)[:, some] for x in dev], to_host(do)[:, some], scale, None, None if dS is None else to_host(dS)[:, some])
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        near(to_host(x)[:, some], y, max(ROUNDED, ROUNDED / 3 ** 0.5 + 2.0 ** -18 * terms_of_dg(dev, some, want)) if name == "dg" else ROUNDED, name)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("size", [(3, 320, 128, 128), (5, 200, 64, 64), (3, 150, 64, 128), (2, 100, 128, 64), (24, 260, 128, 128),
                                  (50, 130, 64, 64), (45, 140, 64, 128), (45, 140, 128, 64)], ids=str)
def test_backward(size, case):
    H, N, dk, dv = size
    dev, r = alike(H, N, dk, dv, *case, seed=3 * N + dv)
    do = to_dev(r.normal(size=(1, H, N, dv)).astype(np.float32), "bf16")
    gradients(dev, do, None, [0, H - 1], dk ** -0.5)


@pytest.mark.parametrize("last", [1, 8, 65])
@pytest.mark.parametrize("case", [CASES[0], CASES[3], CASES[4]], ids=str)
@pytest.mark.parametrize("H, N, d", [(1, 33, 128), (1, 320, 128), (3, 640, 128), (2, 70, 64), (30, 257, 128), (1, 64, 64)])
def test_gradients_of_the_last_tokens(H, N, d, case, last):
    dev, r = alike(H, N, d, d, *case, seed=N + last)
    do = r.normal(size=(1, H, N, d))
    do[:, :, :max(N - last, 0)] = 0
    gradients(dev, to_dev(do.astype(np.float32), "bf16"), None, [0, H - 1] if H > 1 else [0], d ** -0.5)


@pytest.mark.parametrize("H, N, d", [(1, 320, 128), (24, 130, 64)])
def test_initial_state_gradient(H, N, d):
    dev, r = alike(H, N, d, d, 3, True, True, False, seed=N)
    S0, dS = [to_dev((r.normal(size=(1, H, d, d)) * d ** -0.5).astype(np.float32), "f32") for _ in range(2)]
    do = to_dev(r.normal(size=(1, H, N, d)).astype(np.float32), "bf16")
    got = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    some = [0, H - 1]
    want = gated.backward(*[to_host(x)[:, some] for x in dev], to_host(do)[:, some], d ** -0.5, to_host(S0)[:, some], to_host(dS)[:, some])
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        near(to_host(x)[:, some], y, ROUNDED, name)
    near(to_host(got[5])[:, some], want[5], STATE, "dS0")
    # without a state's gradient asked for, the other gradients keep their bits
    zero = torch.zeros_like(S0)
    assert all(torch.equal(x, y) for x, y in zip(la.backward_gated_delta(*dev, do, S0=zero)[:5], la.backward_gated_delta(*dev, do)))
