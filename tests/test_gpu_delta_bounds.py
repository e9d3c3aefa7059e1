"""The delta rule's tree decode and state advance against the bounds of
oracle/spec.py, which follow the increments themselves and not the magnitudes
along a path (test_spec_bounds.py shows what they let through and what not)."""

import numpy as np
import pytest

import causal_linear_attention_la_gb300 as la
from helpers import build_lib, to_dev, to_host
from oracle import spec
from test_spec_bounds import inputs

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build_lib()
    la.lib()
    yield
    torch.cuda.synchronize()
    assert la.la_device_status(True) == la.LA_OK


def i32(x):
    import torch
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


def check_tree(T, dk, dv, dtype, tensor_cores, correlated, count=None):
    import torch
    S, q, k, v, parent = inputs(T, dk, dv, T + dk + dv, correlated=correlated)
    for b, n in enumerate(count or []):
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = np.nan, np.inf, np.nan
    want, _ = spec.decode_tree_delta(S, q, k, v, parent, count)
    bound = HALF[dtype] * np.abs(want) + spec.decode_tree_delta_bound(S, q, k, v, parent, count, parts=tensor_cores)
    prev = la.la_set_path(la.LA_PATH_AUTO if tensor_cores else la.LA_PATH_SIMT)
    try:
        assert la.la_tree_path(dk, dv, la.LA_BF16 if dtype == "bf16" else la.LA_F32) == int(tensor_cores)
        out = to_dev(np.full(v.shape, 5.0, np.float32), dtype)
        la.decode_tree_delta(torch.from_numpy(S).cuda(), *[to_dev(x.astype(np.float32), dtype) for x in (q, k, v)], i32(parent),
                             count=None if count is None else i32(count), out=out)
    finally:
        la.la_set_path(prev)
    got = to_host(out)
    for b, n in enumerate([T] * 3 if count is None else count):
        assert np.all(got[b, :, n:] == 5.0)
        ratio = np.abs(got[b, :, :n] - want[b, :, :n]) / bound[b, :, :n]
        assert np.all(ratio <= 1.0), (b, ratio.max())


@pytest.mark.parametrize("correlated", [0.0, 2.0])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 25, 32, 33, 48, 49, 57, 64])
def test_tree_on_tensor_cores(T, dk, dv, correlated):
    check_tree(T, dk, dv, "bf16", True, correlated)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 16), (16, 128), (128, 32)])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 16, 17, 33, 64])
def test_tree_on_cuda_cores(T, dk, dv, dtype):
    check_tree(T, dk, dv, dtype, False, 2.0 * (T % 2))


@pytest.mark.parametrize("count", [[64, 17, 40], [33, 0, 64], [16, 48, 49], [1, 32, 15]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ragged_trees(count, dtype):
    for correlated in (0.0, 2.0):
        check_tree(64, 128, 128, dtype, dtype == "bf16", correlated, count)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [14, 24, 47, 60])
def test_nodes_beside_one_that_is_not_finite(T, d, dtype):
    """Nodes whose paths are clean, held to the bound of the tree that is left
    when the others are taken out."""
    import torch
    S, q, k, v, parent = inputs(T, d, d, T + d, correlated=2.0)
    S, q, k, v = (x[2:] for x in (S, q, k, v))
    parent, bad = parent[2], [2, 9]
    clean = [i for i in range(T) if not set(spec.path_of(parent, i)) & set(bad)]
    left = np.array([[clean.index(parent[i]) if parent[i] >= 0 else -1 for i in clean]])
    rest = [x[:, :, clean] for x in (q, k, v)]
    want, _ = spec.decode_tree_delta(S, *rest, left)
    # (fp32 on the CUDA cores; on the tensor cores such a tree is done again in fp32)
    bound = HALF[dtype] * np.abs(want) + spec.decode_tree_delta_bound(S, *rest, left)
    for rows in (k, v):
        for x in (np.nan, np.inf, -3e38):
            was = rows[:, :, bad].copy()
            rows[:, :, bad, 1::5] = x
            out = la.decode_tree_delta(torch.from_numpy(S).cuda(), *[to_dev(y.astype(np.float32), dtype) for y in (q, k, v)],
                                       i32(parent[None]))
            rows[:, :, bad] = was
            got = to_host(out)[:, :, clean]
            if x != -3e38 or dtype == "f32":
                assert np.all(np.abs(got - want) <= bound)
            else:                                # finite until a product overflows: may stay on the tensor cores
                parts = spec.decode_tree_delta_bound(S, *rest, left, parts=True)
                assert np.all(np.abs(got - want) <= HALF[dtype] * np.abs(want) + parts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (16, 16), (32, 128)])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 33, 100])
def test_advance(T, dk, dv, dtype):
    import torch
    S, _, k, v, _ = inputs(T, dk, dv, T + dk, correlated=2.0 * (T % 2))
    rng = np.random.default_rng(T)
    path, accepted = rng.integers(0, T, (3, T)), [T, T // 2, 0]
    kd, vd = (to_dev(x.astype(np.float32), dtype) for x in (k, v))
    for p in (None, path):
        want, _ = spec.advance_delta(S, k, v, p, accepted)
        bound = spec.advance_delta_bound(S, k, v, p, accepted)
        got = la.state_advance_delta(torch.from_numpy(S.copy()).cuda(), kd, vd, None if p is None else i32(p), i32(accepted))
        off = np.abs(to_host(got) - want)
        assert np.all(off <= bound), (off / np.maximum(bound, 1e-300)).max()
