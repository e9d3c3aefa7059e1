"""Tree decode at the ends of fp32's range: states that are infinite, and values
between bf16's largest number (2^128 - 2^120) and fp32's, which the tensor-core
kernels hold as two bf16 parts. Bounds as in test_gpu_spec.py."""

import numpy as np
import pytest

import causal_linear_attention_la_gb300 as la
from helpers import build_lib, to_dev, to_host
from oracle import spec
from test_gpu_spec import cuda, gamma, i32, near, on_tc, rows, state, tree

pytestmark = pytest.mark.gpu

BF16_MAX = 2.0 ** 128 - 2.0 ** 120


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build_lib()
    la.lib()
    yield
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK


def same_where_not_finite(got, want, scale, dtype, g):
    with np.errstate(invalid="ignore"):
        odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True)
    near(got[~odd], want[~odd], scale[~odd], dtype, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("T", [9, 24, 60])
def test_infinite_state(T, rule, d, dtype):
    """An infinity in the state reaches its column as the steps would have it:
    infinite of its sign, NaN where both signs meet, and no other column.

    By the delta rule the column is not finite anywhere, but which of its values
    are NaN goes by the order of the sums: the steps take k (S^T k) from a state
    row s = inf first, inf - k^2 inf = NaN, the formula of the whole path adds
    q.S = +-inf and (q.k) u = +-inf, which may have one sign."""
    B, H = 1, 2
    delta = rule == "delta"
    S, z = state(B, H, d, d, T + d, delta)
    S[0, 0, 3, 5], S[0, 0, 7, 9], S[0, 1, 0, 0], S[0, 1, d - 1, d - 1] = np.inf, -np.inf, np.inf, -np.inf
    S[0, 1, 2:4, 20] = np.inf, -np.inf
    S[0, 0, 5, 33] = np.nan
    q, k, v = rows(B, H, T, d, d, T, dtype, delta)
    parent = tree(B, T, T + 1, lean=0.3)
    alpha = np.array([0.9, 1.0], np.float32) if rule == "decay" else None
    args = [to_dev(x, dtype) for x in (q, k, v)] + [i32(parent)]
    with np.errstate(invalid="ignore"):
        if delta:
            out = la.decode_tree_delta(cuda(S), *args)
            want, scale = spec.decode_tree_delta(S, q, k, v, parent)
        else:
            out = la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha))
            want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
    if not delta:
        assert np.all(want[0, 0, :, 5] == np.inf) and np.all(want[0, 0, :, 9] == -np.inf) and np.isnan(want[0, 1, :, 20]).all()
    finite = np.isfinite(want).any(axis=(0, 2))
    assert finite.sum() == 2 * d - 6
    got = to_host(out)
    if delta:
        assert not np.isfinite(got[~np.isfinite(want)]).any()
        got[~np.isfinite(want)] = want[~np.isfinite(want)]
    same_where_not_finite(got, want, scale, dtype, gamma(d, T if delta else 1, on_tc(d, d, dtype)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [9, 24, 60])
def test_values_past_the_largest_bf16(T, d, dtype):
    """A state and a pair weight that bf16 alone would round to infinity."""
    B, H = 1, 1
    S, z = state(B, H, d, d, T + d)
    q, k, v = rows(B, H, T, d, d, T, dtype)
    parent = tree(B, T, T + 1, lean=0.3)
    parent[0, :3] = -1, 0, 0
    S[0, 0, 3, 5] = np.finfo(np.float32).max
    q[..., 3] = -1.5                                  # phi 0.22: the sum stays within fp32
    # node 1's key: phi(q_1).phi(k_1) between the two largest numbers
    q[0, 0, 1, :2] = 0.0
    k[0, 0, 1, :2] = BF16_MAX, 3 * 2.0 ** 118
    args = [to_dev(x, dtype) for x in (q, k, v)] + [i32(parent)]
    out = to_host(la.decode_tree(cuda(S), cuda(z), *args))
    want, scale = spec.decode_tree(S, z, q, k, v, parent)
    below = [i for i in range(T) if 1 in spec.path_of(parent[0], i)]
    own = [i for i in range(T) if i not in below] + [1]
    # (1 / den of node 1 is below the normal numbers: 2^-149 of 2^-128, half of it)
    assert np.isfinite(out[0, 0, own]).all()
    near(out[:, :, own], want[:, :, own], scale[:, :, own], dtype, gamma(d, 1, on_tc(d, d, dtype)) + 2.0 ** -21)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [9, 24, 40, 60])
def test_increments_past_the_largest_bf16(T, d, dtype):
    """A delta-rule increment between bf16's largest number and fp32's stays
    with the nodes below it: u_1 = v_1 - (k_1.k_0) u_0 = 2^128 - 2^120 + 3 * 2^118."""
    B, H = 1, 2
    S, _ = state(B, H, d, d, T + d, True)
    q, k, v = rows(B, H, T, d, d, T, dtype, True)
    parent = tree(B, T, T + 1, lean=0.3)
    parent[0, :4] = -1, 0, -1, 2
    S[:, 0, :, 7] = 0.0
    k[:, 0, :2] = 0.0
    k[:, 0, 0, 0], k[:, 0, 1, 0] = 1.0, -1.0
    v[0, 0, 0, 7], v[0, 0, 1, 7] = 3 * 2.0 ** 118, BF16_MAX
    args = [to_dev(x, dtype) for x in (q, k, v)] + [i32(parent)]
    out = to_host(la.decode_tree_delta(cuda(S), *args))
    want, scale = spec.decode_tree_delta(S, q, k, v, parent)
    clean = [i for i in range(T) if 0 not in spec.path_of(parent[0], i)]
    assert len(clean) > 1
    near(out[:, :, clean], want[:, :, clean], scale[:, :, clean], dtype, gamma(d, T, on_tc(d, d, dtype)))
    near(out[:, :, :2], want[:, :, :2], scale[:, :, :2], dtype, gamma(d, T, on_tc(d, d, dtype)))
