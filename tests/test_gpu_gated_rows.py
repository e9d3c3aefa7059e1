"""Gated delta rule on the tensor cores: rows that are not finite beside packed
sequences in every form of the chains, and differences of the forward along v.

Which form is taken goes by the heads: eight warps on 16 columns up to 38 (forward)
or 19 (backward) of them, then pairs of warps, or for the backward one warp for 16 columns."""

import numpy as np
import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import to_dev, to_host

pytestmark = pytest.mark.gpu


def inputs(H, N, d, seed):
    r = np.random.default_rng(seed)
    q, k = [x / np.linalg.norm(x, axis=-1, keepdims=True) for x in r.normal(size=(2, 1, H, N, d))]
    g = -np.exp(r.uniform(-5, 0, size=(H, 1))) * np.log1p(np.exp(r.normal(size=(1, H, N))))
    beta = 1 / (1 + np.exp(-r.normal(size=(1, H, N))))
    dev = [to_dev(x.astype(np.float32), "bf16") for x in (q, k, r.normal(size=q.shape))]
    dev += [to_dev(x.astype(np.float32), "f32") for x in (g, beta)]
    S0, dS = [to_dev((r.normal(size=(4, H, d, d)) * d ** -0.5).astype(np.float32), "f32") for _ in range(2)]
    return dev, S0, dS, to_dev(r.normal(size=q.shape).astype(np.float32), "bf16"), r


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [(5, 69, 69, 100, 190), (3, 70, 135, 199, 300)], ids=str)
@pytest.mark.parametrize("heads, d", [(2, 128), (50, 128), (90, 64), (80, 128)])
def test_rows_of_other_sequences(heads, d, at, value):
    """Nothing outside the sequences, and nothing of sequence 2 from its 12th token on,
    reaches another sequence or an earlier token."""
    N = at[-1] + 10
    dev, S0, dS, do, _ = inputs(heads, N, d, seed=heads)
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    want, S_want = la.forward_gated_delta(*dev, S0=S0, return_state=True, offsets=off)
    grads = la.backward_gated_delta(*dev, do, S0=S0, dS=dS, offsets=off)
    cut = at[2] + 11
    bad = [x.clone() for x in dev] + [do.clone()]
    for x in bad:
        x[:, :, :at[0]] = value
        x[:, :, at[4]:] = value
        x[:, :, cut:at[3]] = value
    out = torch.full_like(want, 7.0)
    _, S = la.forward_gated_delta(*bad[:5], S0=S0, return_state=True, offsets=off, out=out)
    assert torch.equal(out[:, :, at[0]:cut], want[:, :, at[0]:cut]) and torch.equal(out[:, :, at[3]:at[4]], want[:, :, at[3]:at[4]])
    assert (out[:, :, :at[0]] == 7).all() and (out[:, :, at[4]:] == 7).all()
    assert torch.equal(S[[0, 1, 3]], S_want[[0, 1, 3]])
    got = la.backward_gated_delta(*bad[:5], bad[5], S0=S0, dS=dS, offsets=off)
    for x, y in zip(got[:5], grads[:5]):
        assert torch.equal(x[:, :, at[0]:at[2]], y[:, :, at[0]:at[2]]) and torch.equal(x[:, :, at[3]:at[4]], y[:, :, at[3]:at[4]])
        assert not x[:, :, :at[0]].any() and not x[:, :, at[4]:].any()
    assert torch.equal(got[5][[0, 1, 3]], grads[5][[0, 1, 3]])


@pytest.mark.parametrize("heads", [2, 24, 50])
def test_differences_along_values(heads):
    """The forward is linear in v and S0: along a step of both, the outputs and states move
    by what dv and dS0 say. Outputs, values and gradients are rounded to bf16, each value by
    itself: by 2^-8 / sqrt(3) in the root mean square, so that a sum of n products is off by
    that times the root of its squared terms; six times that, for the two of the loss and the one of dv."""
    N, d = 200, 128
    dev, S0, dS, do, r = inputs(heads, N, d, seed=heads + 1)
    S0, dS = S0[:1].contiguous(), dS[:1].contiguous()
    got = la.backward_gated_delta(*dev, do, S0=S0, dS=dS)
    dv, dS0 = got[2].double(), got[5].double()
    v2 = to_dev(r.normal(size=dev[2].shape).astype(np.float32), "bf16")
    step = to_dev((r.normal(size=S0.shape) * d ** -0.5).astype(np.float32), "f32")
    a, Sa = la.forward_gated_delta(*dev, S0=S0, return_state=True)
    b, Sb = la.forward_gated_delta(dev[0], dev[1], v2, dev[3], dev[4], S0=step, return_state=True)
    moved = ((b.double() - a.double()) * do.double()).sum() + ((Sb - Sa).double() * dS.double()).sum()
    said = (dv * (v2.double() - dev[2].double())).sum() + (dS0 * (step - S0).double()).sum()
    rms = 2.0 ** -8 / 3 ** 0.5
    terms = [x.double().square().mul(do.double().square()).sum() for x in (a, b)] + [(dv * (v2.double() - dev[2].double())).square().sum()]
    states = 1e-5 * ((Sa.double().norm() + Sb.double().norm()) * dS.double().norm() + dS0.norm() * (step - S0).double().norm())
    assert abs(moved - said).item() <= 6 * rms * sum(terms).sqrt().item() + states.item()


@pytest.mark.parametrize("heads", [3, 50, 80])
def test_large_beta_and_positive_decay(heads):
    """beta up to 2 (a token may overshoot) and g above zero: the formula as it stands."""
    from oracle import gated
    N, d = 180, 128
    dev, S0, dS, do, r = inputs(heads, N, d, seed=7)
    dev[4] = dev[4] * 2
    dev[3] = dev[3] + 0.02
    some = [0, heads - 1]
    host = [to_host(x)[:, some] for x in dev]
    out, S = la.forward_gated_delta(*dev, return_state=True)
    want, S_want = gated.forward(*host, d ** -0.5)
    assert np.linalg.norm(to_host(out)[:, some] - want) <= 2.0 ** -8 * np.linalg.norm(want)
    assert np.linalg.norm(to_host(S)[:, some] - S_want) <= 2.0 ** -15 * np.linalg.norm(S_want)
    got = la.backward_gated_delta(*dev, do)
    for x, y in zip(got, gated.backward(*host, to_host(do)[:, some], d ** -0.5)):
        assert np.linalg.norm(to_host(x)[:, some] - y) <= 2.0 ** -7 * np.linalg.norm(y)


def test_gradients_beyond_32_bits():
    """17 million rows of 256 bytes, 262146 chunks' states of 32 KiB: the last sequence's
    gradients as by itself."""
    n, tail, d = (1 << 24) + 70, 150, 128
    dev, _, _, do, _ = inputs(1, tail, d, seed=8)
    want = la.backward_gated_delta(*dev, do)
    big = [torch.zeros(x.shape[:2] + (n,) + x.shape[3:], dtype=x.dtype, device="cuda") for x in dev + [do]]
    for x, y in zip(big, dev + [do]):
        x[:, :, n - tail:] = y
    off = torch.tensor([0, n - tail, n], dtype=torch.int32, device="cuda")
    got = la.backward_gated_delta(*big[:5], big[5], offsets=off)
    for x, y in zip(got, want):
        assert torch.equal(x[:, :, n - tail:], y) and not x[:, :, :n - tail].any()
