"""Draws from rows of many dense weights, next to a border, and acceptance tests
next to a tie.

Every weight there is a whole number of units, so that the sums are known exactly
in 64-bit integers and one weight can be set such that the draw lies a chosen
distance from the border between two tokens. The stated bound of the kernel's
sums (2^-38 of the row's sum up to 2^18 tokens, 2^-35 up to 2^24) is the distance.
The batches are large enough that a sequence gets a single CTA, where a lane sums
the most values; the small ones spread over eight.
"""

import numpy as np
import pytest

import causal_linear_attention_la_gb300 as la
from helpers import build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build_lib()
    la.lib()
    yield
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK


def base_row(kind, V, rng):
    """Weights as whole numbers of units, each exact in fp32 after division by
    the unit."""
    if kind == "equal":
        return np.full(V, 11184811, np.int64), 2.0 ** -25            # fp32's 1 / 3
    m = rng.integers(1 << 23, 1 << 24, V)                            # 24 bits, over a range of 2^12
    return m << rng.integers(0, 13, V), 2.0 ** -40


def near_a_border(cum, bits, rng, step=1, most=1 << 24):
    """(token, what its weight grows by, u, answer) for a row of whole weights
    with prefix sums `cum`: u times the sum then lies 2^-bits of the sum before
    the end of `token` or behind it, and more than that away from the other
    borders. The new weight is below `most`, and grows by a multiple of `step`."""
    total = int(cum[-1])
    least = max(1 << 20, 3 * (total >> bits))
    while True:
        k = int(rng.integers(1 << 20, 1 << 23))                      # u = k / 2^24 in [1/16, 1/2)
        t = int(np.searchsorted(cum, k * total // 2 ** 24))
        if not 0 < t < len(cum) - 3:
            continue
        side = int(rng.integers(0, 2)) * 2 - 1
        # cum_t + d - u (total + d) = side 2^-bits total
        d = ((side * total << 24 >> bits) - ((int(cum[t]) << 24) - k * total)) // (2 ** 24 - k) // step * step
        if not least <= int(cum[t]) - int(cum[t - 1]) + d < most or int(cum[t + 1]) - int(cum[t]) < least:
            continue
        gap = (int(cum[t]) + d << 24) - k * (total + d)              # exactly, in units of 2^-24
        assert gap * side > 0 and abs((abs(gap) >> 24) - (total >> bits)) <= step + 2
        return t, d, k / 2 ** 24, t if side > 0 else t + 1


@pytest.mark.parametrize("kind", ["equal", "spread"])
@pytest.mark.parametrize("V,B,bits", [(1 << 18, 200, 38), (250007, 200, 38), (1 << 24, 160, 35), ((1 << 24) - 3, 160, 35),
                                      (1 << 18, 3, 38), (1 << 24, 3, 35)])
def test_draw_next_to_a_border(V, B, bits, kind):
    import torch
    rng = np.random.default_rng(V + B)
    w, unit = base_row(kind, V, rng)
    row = torch.from_numpy((w * unit).astype(np.float32)).cuda()
    assert np.array_equal(row.double().cpu().numpy()[:1000], (w * unit)[:1000])
    p = row.expand(B, 1, V).contiguous()
    u, want, cum = np.zeros((B, 1), np.float32), [], np.cumsum(w)
    for b in range(B):
        t, d, u[b, 0], answer = near_a_border(cum, bits, rng)
        p[b, 0, t] = (int(w[t]) + d) * unit
        want.append(answer)
    path, accepted, nxt = la.verify_tree(p, *[torch.zeros((B, 0), dtype=torch.int32, device="cuda")] * 2, torch.from_numpy(u).cuda())
    assert np.array_equal(nxt.cpu().numpy(), want)


@pytest.mark.parametrize("V,B,bits", [(1 << 18, 200, 38), (1 << 22, 160, 35), ((1 << 22) + 5, 160, 35)])
def test_draw_from_the_rest_next_to_a_border(V, B, bits):
    """The same for what a draft leaves, p - q: weights that no single fp32 word
    holds."""
    import torch
    rng = np.random.default_rng(V)
    q = 3                                                            # units of 2^-33, p in units of 2^-25
    w = np.full(V, 11184811 * 256 - q, np.int64)
    p = torch.full((V,), 11184811 * 2.0 ** -25, device="cuda").expand(B, 2, V).contiguous()
    u, want, cum = np.zeros((B, 2), np.float32), [], np.cumsum(w)
    for b in range(B):
        t, d, r, answer = near_a_border(cum, bits, rng, 256, 1 << 32)      # (p stays a multiple of 256 units)
        p[b, 0, t] = (int(w[t]) + d + q) * 2.0 ** -33
        u[b] = 0.5, r
        want.append(answer)
    draft = torch.full((B, 1, V), q * 2.0 ** -33, device="cuda")
    tokens = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")       # no token of the vocabulary: it falls
    accepted, nxt = la.verify_chain(p, draft, tokens, torch.from_numpy(u).cuda())
    assert not accepted.any() and np.array_equal(nxt.cpu().numpy(), want)


def test_acceptance_next_to_a_tie():
    """u q < p exactly (64 bits hold the product of two fp32 numbers), for numbers
    of any size: p is the rounded product, one step below or one above."""
    import torch
    rng = np.random.default_rng(2)
    u, q, p = [], [], []
    for eu, eq in [(0, 0), (-24, -10), (-30, -59), (-30, -62), (-60, -30), (-100, -30), (-120, -20), (-140, 0), (-148, 40), (-60, -85),
                   (-10, -130), (-90, 59), (-125, 70)]:
        for _ in range(40):
            a = np.float32(2.0 ** (eu - 1) * (1 + rng.random()))
            b = np.float32(2.0 ** eq * (1 + rng.random()))
            x = np.float32(np.float64(a) * np.float64(b))
            u += [a] * 3
            q += [b] * 3
            p += [x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(np.inf))]
    u += [np.float32(2.0 ** -100)]                       # 2^-130 (1 - 2^-24), a subnormal 2^-130 once rounded
    q += [np.float32(2.0 ** -30 * (1 - 2.0 ** -24))]
    p += [np.float32(2.0 ** -130)]
    u, q, p = (np.array(x, np.float32) for x in (u, q, p))
    B, V = len(u), 8
    target, draft = np.zeros((B, 2, V), np.float32), np.zeros((B, 1, V), np.float32)
    target[:, 0, 3], target[:, 1, 5], draft[:, 0, 3] = p, 1.0, q
    uniform = np.stack([u, np.full(B, 0.5, np.float32)], 1)
    tokens = torch.full((B, 1), 3, dtype=torch.int32, device="cuda")
    accepted, _ = la.verify_chain(*(torch.from_numpy(x).cuda() for x in (target, draft)), tokens, torch.from_numpy(uniform).cuda())
    want = u.astype(np.float64) * q.astype(np.float64) < p.astype(np.float64)
    assert want[-1] and 0.2 < want.mean() < 0.8
    assert np.array_equal(accepted.cpu().numpy(), want.astype(np.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 50001])
def test_rows_that_sum_past_fp32(V, dtype):
    """Finite weights whose sum is beyond 3.4e38 give no token, wherever they lie;
    just below it they are drawn from, and so are sums of 2^-110."""
    import torch
    from helpers import to_dev
    w = np.zeros((6, 2, V), np.float32)
    w[0, :, [0, V - 1]] = 2.0 ** 127                     # 2^128
    w[1, :, ::7] = 2.0 ** 126
    w[2, :, [0, V - 1]] = 2.0 ** 126                     # 2^127: drawn from
    w[3, :, [1, V - 2]] = 2.0 ** -111
    w[4, :, :30] = 2.0 ** 124                            # 30 of 16
    w[5, :, :15] = 2.0 ** 124                            # 15 of 16: drawn from
    u = np.full((6, 2), 0.75, np.float32)
    want = [-1, -1, V - 1, V - 2, -1, 11]
    p = to_dev(w, dtype)
    none = torch.full((6, 1), -1, dtype=torch.int32, device="cuda")
    accepted, nxt = la.verify_chain(p, torch.zeros_like(p[:, :1]), none, torch.from_numpy(u).cuda())
    assert not accepted.any() and nxt.tolist() == want
    path, accepted, nxt = la.verify_tree(p, none, none, torch.from_numpy(u).cuda())
    assert not accepted.any() and nxt.tolist() == want and torch.all(path == -1)
