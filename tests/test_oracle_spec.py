"""The oracle of the speculative-decoding operators against what they mean: a
tree of one path is a sequence of steps, the verified tokens follow the target's
law, packed values are the nearest ones. Host logic only."""

import numpy as np
import pytest

import oracle as orc
from oracle import spec
from causal_linear_attention_la_gb300 import synth


def _state(B, H, dk, dv, seed):
    q, k, v = synth.qkv(B, H, 12, dk, dv, seed=seed, dtype="f32")
    _, S, z = orc.forward_recurrent(q, k, v, return_state=True)
    return S, z


@pytest.mark.parametrize("alpha", [None, [0.5, 0.9, 1.0]])
def test_a_tree_of_one_path_is_a_sequence(alpha):
    B, H, T, dk, dv = 2, 3, 6, 16, 32
    S, z = _state(B, H, dk, dv, 1)
    q, k, v = synth.qkv(B, H, T, dk, dv, seed=2, dtype="f32")
    parent = np.tile(np.arange(T) - 1, (B, 1))
    out, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
    a = np.ones((1, H)) if alpha is None else np.array(alpha)[None]
    S2, z2, want = orc.decode_steps_decay(S, z, q, k, v, alpha=a)
    assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
    assert np.all(scale >= np.abs(out) * (1 - 1e-12))
    S3, z3, A = spec.advance(S, z, k, v, alpha=alpha)
    assert np.allclose(S3, S2, rtol=1e-12) and np.allclose(z3, z2, rtol=1e-12)
    S4, _ = spec.advance_delta(S, k, v)
    S5, want = orc.decode_steps_delta(S, q, k, v)
    assert np.allclose(S4, S5, rtol=1e-10, atol=1e-12)
    out, _ = spec.decode_tree_delta(S, q, k, v, parent)
    assert np.allclose(out, want, rtol=1e-10, atol=1e-12)


def test_siblings_do_not_meet():
    S, z = _state(1, 2, 16, 16, 3)
    q, k, v = synth.qkv(1, 2, 5, 16, 16, seed=4, dtype="f32")
    parent = np.array([[-1, 0, 0, 1, 9]])          # node 4: no earlier node, so a child of the root
    out, _ = spec.decode_tree(S, z, q, k, v, parent)
    for i, path in enumerate([[0], [0, 1], [0, 2], [0, 1, 3], [4]]):
        assert spec.path_of(parent[0], i) == path
        one = np.arange(len(path))[None] - 1
        want, _ = spec.decode_tree(S, z, q[:, :, path], k[:, :, path], v[:, :, path], one)
        assert np.allclose(out[:, :, i], want[:, :, -1], rtol=1e-13)


def test_rows_of_a_path_end_at_an_entry_outside():
    assert spec._rows([[2, 0, 7, 1]], [4], 0, 3) == [2, 0]
    assert spec._rows([[2, 0, -1, 1]], [9], 0, 4) == [2, 0]
    assert spec._rows(None, [-3], 0, 4) == []
    assert spec._rows(None, None, 0, 3) == [0, 1, 2]


def test_chain_follows_the_target():
    """Over a fine grid of random numbers the first token out of a chain of one
    (drafted from q) has the target's law: sum over drafted x of q(x) times
    [the accepted x, or the draw from the rest]."""
    rng = np.random.default_rng(5)
    V, n = 4, 200
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    grid = (np.arange(n) + 0.5) / n
    law = np.zeros(V)
    for x in range(V):
        u = np.stack(np.meshgrid(grid, grid, indexing="ij"), -1).reshape(-1, 2)
        B = len(u)
        acc, nxt = spec.verify_chain(np.broadcast_to(np.stack([p, p]), (B, 2, V)), np.broadcast_to(q, (B, 1, V)),
                                     np.full((B, 1), x), u)
        law[x] += q[x] * np.mean(acc == 1)
        for t in range(V):
            law[t] += q[x] * np.mean((acc == 0) & (nxt == t))
    # each of the two grids is off by at most half a cell per border
    assert np.abs(law - p).max() <= V / n


def test_tree_samples_are_the_targets():
    rng = np.random.default_rng(6)
    V, n = 5, 1000
    p = rng.dirichlet(np.ones(V), 3)
    u = np.zeros((n, 3))
    u[:, 0] = (np.arange(n) + 0.5) / n
    target = np.broadcast_to(p, (n, 3, V))
    path, acc, nxt = spec.verify_tree(target, np.tile([1, 3], (n, 1)), np.full((n, 2), -1), u)
    first = np.where(acc == 0, nxt, np.where(path[:, 0] == 0, 1, 3))
    for t in range(V):
        assert abs(np.mean(first == t) - p[0, t]) <= 1.0 / n
    # after node 0 the next token is drawn from row 1, after node 1 from row 2
    assert set(nxt[path[:, 0] == 0]) == {spec.draw(p[1], 0.0)}
    assert set(nxt[path[:, 0] == 1]) == {spec.draw(p[2], 0.0)}


def test_draw_edges():
    assert spec.draw([0.0, 0.5, 0.0, 0.5], 0.0) == 1
    assert spec.draw([0.0, 0.5, 0.0, 0.5], 0.5) == 3
    assert spec.draw([0.0, 0.5, 0.0, 0.5, 0.0], 1.0) == 3
    assert spec.draw([0.0, 0.0], 0.3) == -1
    assert spec.draw([np.nan, -1.0, 2.0], 0.9) == 2


def test_pack_takes_the_nearest_values():
    import torch
    rng = np.random.default_rng(7)
    S = (rng.standard_normal((2, 3, 16, 64)) * np.exp(rng.uniform(-40, 40, (2, 3, 16, 1)))).astype(np.float32)
    S[0, 0, 0] = 0.0
    S[0, 0, 1, :4] = [448.0, 449.0, -448.0, 1e-30]
    S[0, 0, 2, 0] = np.inf
    S[0, 0, 3, 5] = np.nan
    S[0, 0, 4, :3] = [3.4e38, -3.4e38, np.inf]
    codes, scales = spec.pack(S)
    back = spec.unpack(codes, scales)
    x = S.reshape(2, 3, 16, 2, 32).astype(np.float64)
    e = 2.0 ** (scales.astype(float) - 127)[..., None]
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1, keepdims=True)
    assert np.all(top <= 448 * e) and np.all((top > 224 * e) | (e == 2.0 ** -127))
    ok = np.isfinite(x)
    err = np.abs(back.reshape(x.shape) - x)
    assert np.all(err[ok] <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * e)[ok])
    assert np.isnan(back[0, 0, 3, 5]) and back[0, 0, 2, 0] == 448 * e[0, 0, 2, 0, 0]
    # the codes are torch's cast of the scaled values
    assert np.isfinite(back[0, 0, 4]).all() and np.abs(back[0, 0, 4]).max() == 240 * 2.0 ** 120
    ok &= e < 2.0 ** 120
    want = torch.from_numpy((x / e).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes.reshape(x.shape)[ok], want[ok])
    # and packing what comes back changes no value (a block whose largest value
    # was rounded down to a power of two may take another scale)
    again = spec.unpack(*spec.pack(np.nan_to_num(back)))
    assert np.array_equal(again[~np.isnan(back)], back[~np.isnan(back)])
