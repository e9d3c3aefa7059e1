"""The error bounds that the delta-rule kernels are held to can be met and can be
missed: the tensor-core kernels' arithmetic, restated on the CPU, stays within
them, and the same with any one operand's low part left out does not. Host only.
"""

import numpy as np
import pytest

from oracle import spec
from causal_linear_attention_la_gb300 import synth

HALF_BF16 = 2.0 ** -8


def inputs(T, dk, dv, seed, H=2, correlated=0.0):
    """A state after 24 tokens, and T rows with keys of norm 1 that share a
    direction where they are correlated; a path, a star, a random tree."""
    rng = np.random.default_rng(seed)

    def keys(n):
        k = rng.standard_normal((3, H, n, dk)) + correlated * rng.standard_normal((3, H, 1, dk))
        return k / np.linalg.norm(k, axis=-1, keepdims=True)

    k0, v0 = keys(24), rng.standard_normal((3, H, 24, dv)) * dv ** -0.5
    S = np.einsum("bhtk,bhtv->bhkv", k0, v0).astype(np.float32)
    q, v = (rng.standard_normal((3, H, T, d)) * d ** -0.5 for d in (dk, dv))
    q, k, v = (synth.round_to_bf16(x.astype(np.float32)).astype(np.float64) for x in (q, keys(T), v))
    i = np.arange(T)
    parent = np.stack([i - 1, np.full(T, -1), np.minimum((rng.random(T) ** 0.5 * (i + 1)).astype(int), i) - 1])
    return S, q, k, v, parent


def bf16(x):
    return synth.round_to_bf16(np.asarray(x, np.float32)).astype(np.float64)


def tree_in_parts(S, q, k, v, parent, without=""):
    """One head by the tensor-core kernels' steps: blocks of 16 nodes, two bf16
    parts an operand (the low part of the operands named in `without` left out),
    products without lo lo, fp32 in between."""
    def parts(x, name):
        x = np.asarray(x, np.float32).astype(np.float64)
        return bf16(x), np.zeros_like(x) if name in without else bf16(x - bf16(x))

    def product(a, b):
        return (a[0] @ b[0] + a[1] @ b[0] + a[0] @ b[1]).astype(np.float32).astype(np.float64)

    T = len(q)
    n = (T + 15) // 16 * 16
    q, k, v = (np.concatenate([x, np.zeros((n - T, x.shape[1]))]) for x in (q, k, v))
    on = np.zeros((n, n), bool)
    for i in range(T):
        on[i, spec.path_of(parent, i)] = True
    A = np.where(on & ~np.eye(n, dtype=bool), k @ k.T, 0.0).astype(np.float32).astype(np.float64)
    W, minus, state = parts(np.where(on, q @ k.T, 0.0), "W"), parts(-A, "A"), parts(S, "S")
    R = v - k @ state[0] - k @ state[1]
    U = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    for b in range(0, n, 16):
        own = slice(b, b + 16)
        left = R[own]
        for c in range(0, b, 16):
            left = left + product((minus[0][own, c:c + 16], minus[1][own, c:c + 16]), (U[0][c:c + 16], U[1][c:c + 16]))
        X = parts(np.linalg.inv(np.eye(16) + A[own, own]), "X")
        U[0][own], U[1][own] = parts(product(X, parts(left, "R")), "U")
    return bf16(q @ state[0] + q @ state[1] + product(W, U))[:T]


def worst(T, d, without, correlated=0.0):
    """The largest error over the bound, for each of the three trees."""
    S, q, k, v, parent = inputs(T, d, d, T + d, correlated=correlated)
    want, _ = spec.decode_tree_delta(S, q, k, v, parent)
    bound = HALF_BF16 * np.abs(want) + spec.decode_tree_delta_bound(S, q, k, v, parent, parts=True)
    got = np.stack([[tree_in_parts(S[b, h], q[b, h], k[b, h], v[b, h], parent[b], without) for h in range(S.shape[1])]
                    for b in range(3)])
    return (np.abs(got - want) / bound).max(axis=(1, 2, 3))


@pytest.mark.parametrize("correlated", [0.0, 2.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 9, 17, 32, 64])
def test_two_parts_stay_within_the_bound(T, d, correlated):
    assert worst(T, d, "", correlated).max() <= 1.0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [17, 32, 64])
def test_a_missing_low_part_does_not(T, d):
    assert worst(T, d, "SAXRUW").min() > 2.0               # high parts alone: in every tree
    for operand in "SRUW":
        assert worst(T, d, operand).max() > 1.0, operand
    if T > 17:                                              # the key products too, once they are large
        for operand in "AX":
            assert worst(T, d, operand, 2.0).max() > 1.0, operand


def test_the_bound_means_something():
    """Below a hundredth of the largest output after a path of 64 tokens, in fp32
    below a 500th."""
    for d in (64, 128):
        S, q, k, v, parent = inputs(64, d, d, d)
        want, scale = spec.decode_tree_delta(S, q, k, v, parent)
        top = np.abs(want).max(axis=(1, 2, 3))
        assert np.all(spec.decode_tree_delta_bound(S, q, k, v, parent, parts=True).max(axis=(1, 2, 3)) < 1e-2 * top)
        assert np.all(spec.decode_tree_delta_bound(S, q, k, v, parent).max(axis=(1, 2, 3)) < 2e-3 * top)


@pytest.mark.parametrize("d", [16, 128])
@pytest.mark.parametrize("T", [1, 20, 100])
def test_advance_bound(T, d):
    """fp32 steps stay within the bound; with the state held in bf16, or without
    the last token, they do not."""
    S0, _, k, v, _ = inputs(T, d, d, T, H=1)
    want, _ = spec.advance_delta(S0, k, v)
    bound = spec.advance_delta_bound(S0, k, v)
    assert bound.max() < 2e-3 * np.abs(want).max()
    for held, n in ((np.float32, T), (bf16, T), (np.float32, T - 1)):
        S = S0.copy()
        for t in range(n):
            kt, vt = k[:, :, t].astype(np.float32), v[:, :, t].astype(np.float32)
            u = np.einsum("bhkv,bhk->bhv", S, kt)
            S = held(S + kt[..., None] * (vt - u)[..., None, :]).astype(np.float32)
        right = np.abs(S - want) <= bound
        assert right.all() if held is np.float32 and n == T else not right.all()
