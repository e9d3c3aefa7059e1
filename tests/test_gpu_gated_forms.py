"""The backward of the gated delta rule by four warps of each chain a CTA (many heads):
against the fp64 definition, repeated bit for bit, beside another form's bits for the same
rows within rounding, and its bounded waits. Fewer heads take eight warps on 16 columns,
which the other tests of the gated delta rule do.

Tolerances: test_gpu_gated_keys.py."""

import time

import numpy as np
import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import to_dev, to_host
from oracle import gated

pytestmark = pytest.mark.gpu

SIZES = [(48, 200, 128, 128), (64, 129, 64, 64), (64, 70, 64, 128), (80, 65, 128, 64)]


def inputs(H, N, dk, dv):
    r = np.random.default_rng(H + N)
    q, k = [x / np.linalg.norm(x, axis=-1, keepdims=True) for x in r.normal(size=(2, 1, H // 2, N, dk))]
    v, do = r.normal(size=(2, 1, H, N, dv))
    g = -np.exp(r.uniform(-5, 0, size=(H, 1))) * np.log1p(np.exp(r.normal(size=(1, H, N))))
    beta = 1 / (1 + np.exp(-r.normal(size=(1, H, N))))
    dev = [to_dev(x.astype(np.float32), "bf16") for x in (q, k, v)] + [to_dev(x.astype(np.float32), "f32") for x in (g, beta)]
    S0, dS = [to_dev((r.normal(size=(1, H, dk, dv)) * dk ** -0.5).astype(np.float32), "f32") for _ in range(2)]
    return dev, to_dev(do.astype(np.float32), "bf16"), S0, dS


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradients(size):
    H, N, dk, dv = size
    dev, do, S0, dS = inputs(*size)
    got = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    some = [slice(0, 1), slice(H // 2 - 1, H // 2)]          # key heads: value heads 2 h, 2 h + 1
    for s in some:
        w = slice(2 * s.start, 2 * s.stop)
        x = [to_host(y)[:, s if i < 2 else w] for i, y in enumerate(dev)]
        want = gated.backward(*x, to_host(do)[:, w], dk ** -0.5, to_host(S0)[:, w], to_host(dS)[:, w])
        for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, want):
            a = to_host(a)[:, s if name in ("dq", "dk") else w]
            assert np.linalg.norm(a - b) <= (2.0 ** -15 if name == "dS0" else 2.0 ** -8) * np.linalg.norm(b), name
    again = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # the first heads by themselves take the other form: the same sums in another order
    few = la.backward_gated_delta(*[y[:, :2 if i < 2 else 4].contiguous() for i, y in enumerate(dev)], do[:, :4].contiguous(),
                                  S0=S0[:, :4].contiguous(), dS=dS[:, :4].contiguous())
    for a, b in zip(few, got):
        b = b[:, :a.shape[1]].double()
        assert (a.double() - b).norm() <= 2.0 ** -8 * b.norm()


@pytest.mark.parametrize("gradients", [0, 1])
@pytest.mark.parametrize("size", [SIZES[0], SIZES[1]], ids=str)
def test_waits_give_up_and_the_next_call_runs(size, gradients):
    dev, do, S0, dS = inputs(*size)
    want = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK
    la.la_test_timeout_next_gated(gradients)
    t0 = time.perf_counter()
    la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    torch.cuda.synchronize()
    assert 1.5 < time.perf_counter() - t0 < 30.0
    assert la.la_device_status(True) == la.LA_ERR_TIMEOUT
    got = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N", [1, 2, 7, 16, 32])
@pytest.mark.parametrize("H, dk, dv", [(4, 128, 128), (64, 64, 64), (2, 64, 128), (80, 128, 64)])
def test_gradients_of_short_sequences(H, dk, dv, N):
    dev, do, S0, dS = inputs(H, N, dk, dv)
    got = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    x = [to_host(y)[:, :1 if i < 2 else 2] for i, y in enumerate(dev)]
    want = gated.backward(*x, to_host(do)[:, :2], dk ** -0.5, to_host(S0)[:, :2], to_host(dS)[:, :2])
    for name, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, want):
        a = to_host(a)[:, :1 if name in ("dq", "dk") else 2]
        assert np.linalg.norm(a - b) <= (2.0 ** -15 if name == "dS0" else 2.0 ** -8) * np.linalg.norm(b), name
