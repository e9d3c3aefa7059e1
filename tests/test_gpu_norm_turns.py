"""Sines and cosines of the rotation, fp32 rows: a row with one component of 1
comes out as its norm's reciprocal times a cosine and a sine.

An angle's top 32 bits of a turn, less the quarter turns in it, are at most 2^29
of 2^-32 turns: as a float off by half a step, 2^-25 of pi / 4, beside the 2^-32 of a turn
cut off: under 2^-25. The sine and cosine of that are off by 2 steps (2^-22 of the
value), the reciprocal root by 2 (2^-22), the product by a half: together
2^-20.8 of the value and 2^-25. Double positions times fp32 frequencies: 2^-53 of angles up to
2^20, 2^-33."""

import numpy as np
import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 64), (128, 32), (16, 16)])
def test_sines_and_cosines(d, rot, interleaved):
    N = 3000
    freqs = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    freqs[::2] *= -1
    pos = torch.arange(N, dtype=torch.int32) * 331 - 7000
    pos[:40] = torch.arange(40)
    rows = torch.zeros(1, N, rot // 2, d)
    first = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    second = first + 1 if interleaved else first + rot // 2
    rows[:, :, np.arange(rot // 2), first] = 1.0
    x = rows.cuda()
    how = dict(positions=pos[None].cuda(), freqs=torch.from_numpy(freqs).cuda(), norm="l2", eps=0.0, interleaved=interleaved)
    out, back = la.qk_norm_rotate(x, x.clone(), **how)
    assert torch.equal(out, back)
    angle = pos.numpy().astype(np.float64)[:, None] * freqs.astype(np.float64)          # [N, pairs]

    def check(got, want):
        assert (np.abs(got - want) <= 2.0 ** -20.8 * np.abs(want) + 2.0 ** -25 + 2.0 ** -33).all(), np.abs(got - want).max()

    h = np.arange(rot // 2)
    z = to_host(out)[0]                                                               # [pairs, N, d]
    check(z[h, :, first].T, np.cos(angle))
    check(z[h, :, second].T, np.sin(angle))
    # the gradient turns back: dx of the partner is what dz's first component sends there
    dz = rows.transpose(1, 2).contiguous().cuda()
    dx = to_host(la.qk_norm_rotate_backward(x, x, dz, torch.zeros_like(dz), **how)[0])[0]     # [N, pairs, d]
    check(dx[:, h, second], -np.sin(angle))
