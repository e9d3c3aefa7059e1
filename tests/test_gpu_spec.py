"""Speculative decoding on the recurrent state (tree decode, draft
verification, state advance, packed state pool): CUDA path vs the fp64 oracle.

Tolerances. A value that is a sum of m products, each off by a relative r, is
off by at most (r + m 2^-24) times the sum of its terms' magnitudes (the oracle's
``scale``), whatever the order of the fp32 sums. Per product: the feature map's
exponential (2 units in the last place) on either side, the decay's power (12
roundings) and the products themselves, below 32 roundings in all; m is dk for
the read and at most 64 for the path. The denominator is a sum of positive terms
with the same bound, hence the factor 2. A delta-rule increment rests on those
before it, so that its bound is once more for every node of the path. The result
is rounded to its type once: half a step, eps / 2 of the value.
"""

import numpy as np
import pytest

import oracle as orc
from oracle import spec
import causal_linear_attention_la_gb300 as la
from causal_linear_attention_la_gb300 import synth
from helpers import build_lib, to_dev, to_host

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


def gamma(dk, depth=1, tc=False):
    """On the tensor cores every term is off by 2^-16 of itself on top (fp32
    operands as two bf16 parts): in the pair products and again where they
    weight a value, numerator and denominator, so four times."""
    return (2 * (dk + 64 + 32) * 2.0 ** -24 + (4 * 2.0 ** -16 if tc else 0.0)) * depth


def on_tc(dk, dv, dtype):
    return la.la_tree_path(dk, dv, la.LA_BF16 if dtype == "bf16" else la.LA_F32) == 1


def near(got, want, scale, dtype, g):
    """|got - want| within half a step of the type and g times the scale."""
    bound = HALF[dtype] * np.abs(want) + g * scale
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} values out, worst "
                           f"{np.nanmax(np.abs(got - want) / np.maximum(bound, 1e-300)):.3g} times the bound")


def cuda(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def i32(x):
    return cuda(np.asarray(x, np.int32))


def state(B, H, dk, dv, seed, delta=False):
    q, k, v = synth.qkv(B, H, 24, dk, dv, seed=seed, dtype="f32")
    if delta:
        k = k / np.linalg.norm(k, axis=-1, keepdims=True)
        return np.einsum("bhtk,bhtv->bhkv", k, v).astype(np.float32), None
    _, S, z = orc.forward_recurrent(q, k, v, return_state=True)
    return S.astype(np.float32), z.astype(np.float32)


def rows(B, H, T, dk, dv, seed, dtype, delta=False):
    q, k, v = synth.qkv(B, H, T, dk, dv, seed=seed, dtype="f32")
    if delta:
        k = k / np.linalg.norm(k, axis=-1, keepdims=True)
    if dtype == "bf16":
        q, k, v = (synth.round_to_bf16(x) for x in (q, k, v))
    return q, k, v


def tree(B, T, seed, lean=0.5):
    """Random parents; lean 0: one path, 1: everything hangs off the root's side."""
    rng = np.random.default_rng(seed)
    i = np.arange(T)
    return np.minimum((rng.random((B, T)) ** lean * (i + 1)).astype(int), i) - 1


TREES = [(1, 1, 1, 16, 16), (2, 3, 2, 32, 64), (1, 2, 7, 64, 64), (2, 2, 8, 128, 128), (2, 1, 9, 128, 32), (1, 2, 16, 64, 128),
         (2, 2, 31, 128, 128), (1, 1, 32, 16, 128), (1, 3, 33, 32, 32), (2, 2, 63, 64, 64), (2, 3, 64, 128, 128),
         (1, 1, 64, 128, 16), (3, 2, 17, 16, 64), (2, 2, 3, 64, 128), (1, 2, 40, 128, 64), (2, 1, 49, 64, 128), (1, 3, 11, 128, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("B,H,T,dk,dv", TREES)
def test_tree(B, H, T, dk, dv, rule, dtype):
    import torch
    delta = rule == "delta"
    S, z = state(B, H, dk, dv, 11 * T + dk, delta)
    q, k, v = rows(B, H, T, dk, dv, 7 + T, dtype, delta)
    parent = tree(B, T, T, lean=[0.0, 0.3, 1.0][T % 3])
    alpha = np.linspace(0.6, 1.0, H).astype(np.float32) if rule == "decay" else None
    args = [to_dev(x, dtype) for x in (q, k, v)] + [i32(parent)]
    Sd = cuda(S)
    if delta:
        out = la.decode_tree_delta(Sd, *args)
        want, scale = spec.decode_tree_delta(S, q, k, v, parent)
    else:
        out = la.decode_tree(Sd, cuda(z), *args, alpha=None if alpha is None else cuda(alpha))
        want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
    assert out.dtype == args[0].dtype
    near(to_host(out), want, scale, dtype, gamma(dk, T if delta else 1, on_tc(dk, dv, dtype)))
    assert torch.equal(Sd.cpu(), torch.from_numpy(S)), "the state is only read"


@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_tree_sizes_on_tensor_cores(dk, dv, rule):
    """Both sides of every size at which the tensor-core kernels change (16, 32,
    48 and 64 nodes, halves and whole blocks of 16), as one path, as a star and
    as a random tree."""
    H = 2
    delta = rule == "delta"
    alpha = np.array([0.7, 0.95], np.float32) if rule == "decay" else None
    for T in (1, 8, 9, 15, 16, 17, 24, 25, 31, 32, 33, 41, 48, 49, 56, 57, 63, 64):
        B = 3
        S, z = state(B, H, dk, dv, T, delta)
        q, k, v = rows(B, H, T, dk, dv, T + 1, "bf16", delta)
        parent = np.stack([np.arange(T) - 1, np.full(T, -1), tree(1, T, T)[0]])
        args = [to_dev(x, "bf16") for x in (q, k, v)] + [i32(parent)]
        if delta:
            out = la.decode_tree_delta(cuda(S), *args)
            want, scale = spec.decode_tree_delta(S, q, k, v, parent)
        else:
            out = la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha))
            want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
        near(to_host(out), want, scale, "bf16", gamma(dk, T if delta else 1, True))


@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
def test_tree_sizes_on_cuda_cores(dk, dv, rule):
    """Every head size of the CUDA-core kernel, both sides of its node groups
    (4 or 8), of the delta rule's blocks (8) and of its pair tiles (16, 32)."""
    H = 2
    delta = rule == "delta"
    alpha = np.array([0.7, 0.95], np.float32) if rule == "decay" else None
    for T in (1, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64):
        B = 3
        S, z = state(B, H, dk, dv, T, delta)
        q, k, v = rows(B, H, T, dk, dv, T + 1, "f32", delta)
        parent = np.stack([np.arange(T) - 1, np.full(T, -1), tree(1, T, T)[0]])
        args = [to_dev(x, "f32") for x in (q, k, v)] + [i32(parent)]
        if delta:
            out = la.decode_tree_delta(cuda(S), *args)
            want, scale = spec.decode_tree_delta(S, q, k, v, parent)
        else:
            out = la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha))
            want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
        near(to_host(out), want, scale, "f32", gamma(dk, T if delta else 1))


@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
def test_tree_of_64_ragged(rule):
    """Trees of every size class in one call of 64 rows; rows behind them stay."""
    B, H, T, d = 10, 2, 64, 128
    delta = rule == "delta"
    count = [0, 1, 8, 16, 17, 32, 33, 48, 49, 64]
    alpha = np.array([0.5, 1.0], np.float32) if rule == "decay" else None
    S, z = state(B, H, d, d, 44, delta)
    q, k, v = rows(B, H, T, d, d, 45, "bf16", delta)
    for b, n in enumerate(count):
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = np.nan, np.inf, np.nan
    parent = tree(B, T, 46, lean=0.2)
    args = [to_dev(x, "bf16") for x in (q, k, v)] + [i32(parent)]
    out = to_dev(np.full((B, H, T, d), -3.0, np.float32), "bf16")
    if delta:
        la.decode_tree_delta(cuda(S), *args, count=i32(count), out=out)
        want, scale = spec.decode_tree_delta(S, q, k, v, parent, count)
    else:
        la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha), count=i32(count), out=out)
        want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha, count)
    got = to_host(out)
    for b, n in enumerate(count):
        assert np.all(got[b, :, n:] == -3.0)
        near(got[b, :, :n], want[b, :, :n], scale[b, :, :n], "bf16", gamma(d, T if delta else 1, True))


@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (32, 128)])
def test_tree_of_64_ragged_f32(dk, dv, rule):
    """The same on the CUDA cores, whose layout goes by the rows of the call."""
    B, H, T = 9, 2, 64
    delta = rule == "delta"
    count = [0, 1, 7, 16, 31, 33, 59, 61, 64]
    alpha = np.array([0.5, 1.0], np.float32) if rule == "decay" else None
    S, z = state(B, H, dk, dv, 47, delta)
    q, k, v = rows(B, H, T, dk, dv, 48, "f32", delta)
    for b, n in enumerate(count):
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = np.nan, np.inf, np.nan
    parent = tree(B, T, 49, lean=0.2)
    args = [to_dev(x, "f32") for x in (q, k, v)] + [i32(parent)]
    out = to_dev(np.full((B, H, T, dv), -3.0, np.float32), "f32")
    if delta:
        la.decode_tree_delta(cuda(S), *args, count=i32(count), out=out)
        want, scale = spec.decode_tree_delta(S, q, k, v, parent, count)
    else:
        la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha), count=i32(count), out=out)
        want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha, count)
    got = to_host(out)
    for b, n in enumerate(count):
        assert np.all(got[b, :, n:] == -3.0)
        near(got[b, :, :n], want[b, :, :n], scale[b, :, :n], "f32", gamma(dk, T if delta else 1))


def test_tree_repeats_bit_for_bit():
    import torch
    B, H, T, d = 40, 8, 40, 128
    S, z = (cuda(x) for x in state(B, H, d, d, 50))
    q, k, v = (to_dev(x, "bf16") for x in rows(B, H, T, d, d, 51, "bf16"))
    parent = i32(tree(B, T, 52))
    one = la.decode_tree(S, z, q, k, v, parent)
    two = la.decode_tree_delta(S, q, k, v, parent)
    for _ in range(5):
        assert torch.equal(one, la.decode_tree(S, z, q, k, v, parent))
        assert torch.equal(two, la.decode_tree_delta(S, q, k, v, parent))


@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("T", [1, 5, 16, 24, 47, 64])
def test_tree_on_cuda_cores_agrees(T, rule):
    """The CUDA-core kernel on bf16 rows of the tensor-core shapes."""
    B, H, d = 2, 2, 64
    delta = rule == "delta"
    S, z = state(B, H, d, d, T, delta)
    q, k, v = rows(B, H, T, d, d, T + 1, "bf16", delta)
    parent = tree(B, T, T + 2)
    alpha = np.linspace(0.6, 1.0, H).astype(np.float32) if rule == "decay" else None
    args = [to_dev(x, "bf16") for x in (q, k, v)] + [i32(parent)]
    prev = la.la_set_path(la.LA_PATH_SIMT)
    try:
        assert la.la_tree_path(d, d, la.LA_BF16) == 0
        if delta:
            out = la.decode_tree_delta(cuda(S), *args)
            want, scale = spec.decode_tree_delta(S, q, k, v, parent)
        else:
            out = la.decode_tree(cuda(S), cuda(z), *args, alpha=None if alpha is None else cuda(alpha))
            want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
        near(to_host(out), want, scale, "bf16", gamma(d, T if delta else 1))
    finally:
        la.la_set_path(prev)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("delta", [False, True])
def test_tree_ragged(delta, dtype):
    """Trees of 0, 1, some and all nodes, counts out of range; rows behind the
    last node keep what they hold and NaN rows behind it are not read."""
    B, H, T, d = 6, 2, 20, 128
    S, z = state(B, H, d, d, 3, delta)
    q, k, v = rows(B, H, T, d, d, 5, dtype, delta)
    parent = tree(B, T, 6)
    count = [0, 1, 13, 20, 99, -4]
    for b, n in enumerate(count):
        n = min(max(n, 0), T)
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = np.nan, np.nan, np.inf
    out = to_dev(np.full((B, H, T, d), 7.0, np.float32), dtype)
    args = [to_dev(x, dtype) for x in (q, k, v)] + [i32(parent)]
    if delta:
        la.decode_tree_delta(cuda(S), *args, count=i32(count), out=out)
        want, scale = spec.decode_tree_delta(S, q, k, v, parent, count)
    else:
        la.decode_tree(cuda(S), cuda(z), *args, count=i32(count), out=out)
        want, scale = spec.decode_tree(S, z, q, k, v, parent, count=count)
    got = to_host(out)
    for b, n in enumerate(count):
        n = min(max(n, 0), T)
        assert np.all(got[b, :, n:] == 7.0)
        near(got[b, :, :n], want[b, :, :n], scale[b, :, :n], dtype, gamma(d, T if delta else 1, on_tc(d, d, dtype)))
    # out allocated by the call: zeros behind the last node
    if not delta:
        got = to_host(la.decode_tree(cuda(S), cuda(z), *args, count=i32(count)))
        assert np.all(got[0] == 0.0) and np.all(got[2, :, 13:] == 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("T", [14, 24, 60])
def test_tree_nonfinite_rows_off_the_path(T, delta, d, dtype):
    """Infinities, NaN and the type's largest numbers in one node reach that
    node's descendants and nobody else."""
    B, H = 1, 2
    S, z = state(B, H, d, d, 8, delta)
    q, k, v = rows(B, H, T, d, d, 9, dtype, delta)
    parent = tree(B, T, 10)
    bad = [2, 9]
    clean = [i for i in range(T) if not set(spec.path_of(parent[0], i)) & set(bad)]
    soiled = [i for i in range(T) if i not in clean]
    assert len(clean) > 4 and len(soiled) > 2
    if delta:
        want, scale = spec.decode_tree_delta(S, q, k, v, parent)
    else:
        want, scale = spec.decode_tree(S, z, q, k, v, parent)
    for kv in ("v", "k", "kv"):
        for x in (np.nan, np.inf, -np.inf, 3e38, -3e38):
            k2, v2 = k.copy(), v.copy()
            if "v" in kv:
                v2[:, :, bad, ::3] = x
            if "k" in kv:
                k2[:, :, bad, 1::5] = x
            args = [to_dev(y, dtype) for y in (q, k2, v2)] + [i32(parent)]
            out = la.decode_tree_delta(cuda(S), *args) if delta else la.decode_tree(cuda(S), cuda(z), *args)
            got = to_host(out)
            near(got[:, :, clean], want[:, :, clean], scale[:, :, clean], dtype, gamma(d, T if delta else 1, on_tc(d, d, dtype)))
            if kv == "v" and np.isnan(x):
                assert np.all(np.isnan(got[:, :, soiled][..., ::3]))
                if not delta:
                    cols = np.ones(d, bool)
                    cols[::3] = False
                    near(got[..., cols], want[..., cols], scale[..., cols], dtype, gamma(d, 1, on_tc(d, d, dtype)))


def test_tree_parents_out_of_range():
    """A parent that is no earlier node counts as the committed state."""
    B, H, T, d = 2, 2, 12, 64
    S, z = state(B, H, d, d, 12)
    q, k, v = rows(B, H, T, d, d, 13, "f32")
    parent = tree(B, T, 14)
    wild = parent.copy()
    wild[0, [0, 3, 5]] = [0, 3, 2 ** 31 - 1]
    wild[1, [1, 4, 11]] = [-2 ** 31, 11, 12]
    args = [to_dev(x, "f32") for x in (q, k, v)]
    got = to_host(la.decode_tree(cuda(S), cuda(z), *args, i32(wild)))
    want, scale = spec.decode_tree(S, z, q, k, v, wild)
    near(got, want, scale, "f32", gamma(d))


@pytest.mark.parametrize("alpha", [0.0, 1e-30, 1.0, 1.25])
def test_tree_decay_extremes(alpha):
    B, H, T, d = 1, 2, 40, 64
    S, z = state(B, H, d, d, 15)
    for dtype in ("f32", "bf16"):
        q, k, v = rows(B, H, T, d, d, 16, dtype)
        parent = tree(B, T, 17, lean=0.1)
        a = np.full(H, alpha, np.float32)
        got = to_host(la.decode_tree(cuda(S), cuda(z), *[to_dev(x, dtype) for x in (q, k, v)], i32(parent), alpha=cuda(a)))
        want, scale = spec.decode_tree(S, z, q, k, v, parent, a)
        near(got, want, scale, dtype, gamma(d, 1, on_tc(d, d, dtype)))


def test_tree_of_one_path_matches_decode_steps():
    """A chain's outputs are those of la_decode_steps within both calls' bounds."""
    import torch
    B, H, T, d = 2, 4, 16, 128
    S, z = state(B, H, d, d, 18)
    q, k, v = rows(B, H, T, d, d, 19, "f32")
    args = [to_dev(x, "f32") for x in (q, k, v)]
    parent = i32(np.tile(np.arange(T) - 1, (B, 1)))
    tree_out = la.decode_tree(cuda(S), cuda(z), *args, parent)
    S2, z2 = cuda(S), cuda(z)
    steps = la.decode_steps(S2, z2, *args)
    S3, z3 = la.state_advance(cuda(S), cuda(z), args[1], args[2])
    _, scale = spec.decode_tree(S, z, q, k, v, parent.cpu().numpy())
    assert np.all(np.abs(to_host(tree_out) - to_host(steps)) <= 2 * (gamma(d) * scale + 2.0 ** -24 * np.abs(to_host(steps))))
    assert torch.equal(S2, S3) and torch.equal(z2, z3)


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def probabilities(shape, rng, dtype, sharp=2.0):
    p = softmax(sharp * rng.standard_normal(shape)).astype(np.float32)
    return synth.round_to_bf16(p) if dtype == "bf16" else p


def run_chain(p, q, x, u, count=None, dtype="f32"):
    acc, nxt = la.verify_chain(to_dev(p, dtype), to_dev(q, dtype), i32(x), cuda(u), count=None if count is None else i32(count))
    return acc.cpu().numpy(), nxt.cpu().numpy()


VOCABS = [1, 2, 31, 33, 1000, 4095, 4097, 8191, 20003, 50021, 131072, 200001]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_chain(V, dtype):
    rng = np.random.default_rng(V)
    B, T = 5, 6
    p = probabilities((B, T + 1, V), rng, dtype)
    q = probabilities((B, T, V), rng, dtype)
    q[::2] = p[::2, :T]                                  # some drafts know the target: everything stands
    x = np.array([[spec.draw(q[b, i], rng.random()) for i in range(T)] for b in range(B)])
    u = rng.random((B, T + 1)).astype(np.float32)
    for count in (None, [6, 0, 3, 77, -1]):
        acc, nxt = run_chain(p, q, x, u, count, dtype)
        want = spec.verify_chain(p, q, x, u, count)
        assert np.array_equal(acc, want[0]) and np.array_equal(nxt, want[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_verify_tree(V, dtype):
    rng = np.random.default_rng(V + 1)
    B, T = 4, 40
    p = probabilities((B, T + 1, V), rng, dtype, sharp=3.0)
    u = rng.random((B, T + 1)).astype(np.float32)
    parent = tree(B, T, V, lean=0.6)
    # the likeliest tokens of the parent's row, in turn: paths of several nodes
    order = np.argsort(-p, -1)
    seen = np.zeros((B, T + 1), int)
    x = np.zeros((B, T), int)
    for b in range(B):
        for i in range(T):
            c = parent[b, i] + 1
            x[b, i] = order[b, c, seen[b, c] % V]
            seen[b, c] += 1
    for count in (None, [40, 0, 17, 1]):
        got = la.verify_tree(to_dev(p, dtype), i32(x), i32(parent), cuda(u), count=None if count is None else i32(count))
        want = spec.verify_tree(p, x, parent, u, count)
        for g, w in zip(got, want):
            assert np.array_equal(g.cpu().numpy(), w)


def test_verify_many_draws():
    """Every border of a small vocabulary from many random numbers, against the
    64-bit cumulative sums."""
    rng = np.random.default_rng(3)
    B, V = 4096, 257
    p = np.broadcast_to(probabilities((1, 1, V), rng, "f32"), (B, 1, V))
    u = rng.random((B, 1)).astype(np.float32)
    u[:3, 0] = [0.0, 1.0 - 2.0 ** -24, 0.5]
    acc, nxt = run_chain(p, np.zeros((B, 0, V), np.float32), np.zeros((B, 0)), u)
    assert np.all(acc == 0)
    assert np.array_equal(nxt, [spec.draw(p[b, 0], u[b, 0]) for b in range(B)])


def test_verify_zero_and_nonfinite_weights():
    V, T = 5000, 2
    cases = []
    p = np.zeros((T + 1, V), np.float32)
    q = np.zeros((T, V), np.float32)
    cases.append((p, q, [1, 2], [0.5, 0.5, 0.5]))                       # nothing to draw from: -1
    p1 = p.copy(); p1[:, 4321] = 1.0
    cases.append((p1, p1[:T], [4321, 4321], [0.9, 0.9, 0.9]))           # certain everywhere
    cases.append((p1, p1[:T], [17, 4321], [0.9, 0.9, 0.9]))             # p = q, the token falls: drawn from p
    p2 = p1.copy(); p2[0, 7] = np.nan; p2[0, 9] = -3.0
    cases.append((p2, q, [7, 9], [0.1, 0.1, 0.999]))                    # NaN and negative weights count as 0
    cases.append((p1, q, [-1, V], [0.0, 0.0, 0.0]))                     # tokens outside the vocabulary fall
    cases.append((p1, p1[:T], [4321, V + 5], [0.0, 0.0, 0.3]))
    p3 = p.copy(); p3[:, [0, V - 1]] = [1e-30, 1e-30]
    cases.append((p3, q, [5, 6], [0.3, 0.3, 1.0]))                      # random numbers of 1 and more: the last one
    cases.append((p3, q, [5, 6], [0.3, 0.3, np.nan]))
    cases.append((p3, q, [5, 6], [0.3, 0.3, -1.0]))                     # below zero: the first
    P, Q, X, U = (np.stack([np.asarray(c[i], np.float32) for c in cases]) for i in range(4))
    acc, nxt = run_chain(P, Q, X, U.astype(np.float32))
    want = spec.verify_chain(P, Q, X, U)
    assert np.array_equal(acc, want[0]) and np.array_equal(nxt, want[1])
    assert nxt[0] == -1 and acc[1] == 2 and acc[2] == 0 and nxt[2] == 4321
    p4 = p1.copy(); p4[0, 3] = np.inf                                   # an infinite weight: no draw
    acc, nxt = run_chain(p4[None], q[None], [[5, 6]], np.array([[0.5, 0.5, 0.5]], np.float32))
    assert nxt[0] == -1


def test_verify_tree_twins_and_wild_entries():
    """Two children with the same token: the first is taken. Parents that are no
    earlier node count as the root; tokens outside the vocabulary never match."""
    V, T = 300, 6
    p = np.zeros((1, T + 1, V), np.float32)
    p[0, :, 42] = 1.0
    x = [[-5, 42, 42, 42, V, 42]]
    parent = [[-1, -1, -1, 1, 3, 99]]
    u = np.full((1, T + 1), 0.5, np.float32)
    got = [g.cpu().numpy() for g in la.verify_tree(cuda(p), i32(x), i32(parent), cuda(u))]
    assert list(got[0][0]) == [1, 3, -1, -1, -1, -1] and got[1][0] == 2 and got[2][0] == 42
    want = spec.verify_tree(p, x, parent, u)
    assert all(np.array_equal(g, w) for g, w in zip(got, want))


def test_verify_offsets_past_32_bits():
    """Rows that start beyond 2^31 elements."""
    import torch
    B, T, V = 2, 64, 1 << 24
    p = torch.zeros((B, T + 1, V), dtype=torch.bfloat16, device="cuda")
    assert p.numel() > 2 ** 31
    hit = [(i * 7919 * 101) % V for i in range(T + 1)]
    for i in range(T + 1):
        p[1, i, hit[i]] = 1.0
    p[0, 0, 5] = 1.0
    x = i32([[9] * T, hit[:T]])
    parent = i32(np.tile(np.arange(T) - 1, (B, 1)))
    path, acc, nxt = la.verify_tree(p, x, parent, torch.full((B, T + 1), 0.5, device="cuda"))
    assert acc.tolist() == [0, T] and nxt.tolist() == [5, hit[T]] and path[1].tolist() == list(range(T))
    acc, nxt = la.verify_chain(p, p[:, :T].contiguous(), x, torch.full((B, T + 1), 0.5, device="cuda"))
    assert acc.tolist() == [0, T] and nxt.tolist() == [5, hit[T]]


# ---------------------------------------------------------------------------
# State advance
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rule", ["plain", "decay", "delta"])
@pytest.mark.parametrize("B,H,T,dk,dv", [(5, 2, 1, 16, 16), (5, 3, 5, 32, 64), (5, 2, 16, 128, 128), (5, 1, 33, 128, 16),
                                         (5, 2, 64, 16, 128), (5, 2, 20, 64, 64), (5, 1, 100, 64, 32)])
def test_advance(B, H, T, dk, dv, rule, dtype):
    import torch
    delta = rule == "delta"
    S, z = state(B, H, dk, dv, T, delta)
    _, k, v = rows(B, H, T, dk, dv, T + 2, dtype, delta)
    rng = np.random.default_rng(T)
    path = rng.integers(0, T, (B, T))                    # repeats and any order
    path[1, T // 2:] = -1
    path[2, T // 3] = T
    accepted = [T, T, T, 0, T + 50]
    alpha = np.linspace(0.7, 1.0, H).astype(np.float32) if rule == "decay" else None
    kd, vd = to_dev(k, dtype), to_dev(v, dtype)
    for pth, acc in ((path, accepted), (None, accepted), (None, None), (path, None)):
        # (a decay-free z is a sum of at most T + 1 positive terms, rounded T times)
        kw = dict(path=None if pth is None else i32(pth), accepted=None if acc is None else i32(acc))
        g = (T + 32 + (dk if delta else 0)) * 2.0 ** -24
        if delta:
            want, scale = spec.advance_delta(S, k, v, pth, acc)
            got = la.state_advance_delta(cuda(S), kd, vd, **kw)
            other = la.state_advance_delta(cuda(S), kd, vd, S_out=torch.full_like(cuda(S), np.nan), **kw)
            # every increment of a path rests on the ones before it: the bound is per token
            near(to_host(got), want, scale, "f32", T * g)
            assert torch.equal(got, other)
        else:
            want, wz, scale = spec.advance(S, z, k, v, pth, acc, alpha)
            kw["alpha"] = None if alpha is None else cuda(alpha)
            got, gz = la.state_advance(cuda(S), cuda(z), kd, vd, **kw)
            out = torch.full_like(cuda(S), np.nan), torch.full_like(cuda(z), np.nan)
            other = la.state_advance(cuda(S), cuda(z), kd, vd, S_out=out[0], z_out=out[1], **kw)
            near(to_host(got), want, scale, "f32", g)
            near(to_host(gz), wz, wz, "f32", g)
            assert torch.equal(got, other[0]) and torch.equal(gz, other[1])


def test_advance_without_tokens():
    import torch
    S, z = (cuda(x) for x in state(2, 3, 64, 64, 1))
    empty = torch.empty((2, 3, 0, 64), device="cuda")
    out = torch.zeros_like(S), torch.zeros_like(z)
    la.state_advance(S, z, empty, empty, S_out=out[0], z_out=out[1])
    assert torch.equal(out[0], S) and torch.equal(out[1], z)
    S0 = S.clone()
    la.state_advance(S, z, empty, empty)
    la.state_advance_delta(S, empty, empty)
    assert torch.equal(S, S0)
    # a NaN state of a sequence that accepted nothing is left alone in place
    S[0] = float("nan")
    kv = torch.randn((2, 3, 4, 64), device="cuda")
    la.state_advance(S, z, kv, kv, accepted=i32([0, 4]))
    assert torch.isnan(S[0]).all() and torch.isfinite(S[1]).all()


# ---------------------------------------------------------------------------
# Packed state pool
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 16, 16), (3, 2, 32, 64), (2, 5, 16, 32), (4, 3, 128, 128), (2, 7, 64, 16)])
def test_pack_and_unpack(B, H, dk, dv):
    import torch
    rng = np.random.default_rng(dk + dv)
    S = (rng.standard_normal((B, H, dk, dv)) * np.exp(rng.uniform(-85, 85, (B, H, dk, 1)))).astype(np.float32)
    S[0, 0, 0] = 0.0
    S[0, 0, 1] = 1e-42                                    # subnormal
    S[0, 0, 2, :4] = [448.0, 449.0, -448.0, 1e-30]
    S[0, 0, 3, :3] = [np.inf, -np.inf, 2.0]
    S[0, 0, 4, 5] = np.nan
    S[0, 0, 5, :2] = [3.4e38, -3.4e38]
    S[0, 0, 6] = np.inf
    z = rng.standard_normal((B, H, dk)).astype(np.float32)
    slots = B + 3
    codes, scales, z_pool = la.state_pool(slots, H, dk, dv)
    codes.fill_(0xAB)
    scales.fill_(0xCD)
    slot = rng.permutation(slots)[:B]
    la.state_pack(cuda(S), codes, scales, i32(slot), z=cuda(z), z_pool=z_pool)
    wc, ws = spec.pack(S)
    gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
    nan = np.isnan(S)
    assert np.array_equal(gs[slot], ws)
    assert np.array_equal(np.where(nan, 0x7f, gc[slot] & np.where(nan, 0x7f, 0xff)), np.where(nan, 0x7f, wc))
    assert np.array_equal(z_pool.cpu().numpy()[slot], z)
    rest = np.setdiff1d(np.arange(slots), slot)
    assert np.all(gc[rest] == 0xAB) and np.all(gs[rest] == 0xCD)
    back, zb = torch.zeros((B, H, dk, dv), device="cuda"), torch.zeros((B, H, dk), device="cuda")
    la.state_unpack(codes, scales, i32(slot), back, z_pool=z_pool, z=zb)
    assert np.array_equal(back.cpu().numpy(), spec.unpack(gc[slot], ws), equal_nan=True)
    assert np.array_equal(zb.cpu().numpy(), z)


def test_pool_slots():
    """Sequences without a slot are left out, one slot may come back several
    times, and of several sequences packed into one slot the last one stays."""
    import torch
    B, H, d, slots = 7, 2, 32, 4
    S = torch.randn((B, H, d, d), device="cuda")
    codes, scales, _ = la.state_pool(slots, H, d, d)
    la.state_pack(S, codes, scales, i32([2, -1, 2, 0, 4, 2, 2 ** 31 - 1]))
    wc, ws = spec.pack(S.cpu().numpy())
    gc, gs = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(gc[2], wc[5]) and np.array_equal(gs[2], ws[5])
    assert np.array_equal(gc[0], wc[3]) and not gc[[1, 3]].any() and not gs[[1, 3]].any()
    back = torch.full((B, H, d, d), 5.0, device="cuda")
    la.state_unpack(codes, scales, i32([2, 2, -7, 0, 4, 1, 2]), back)
    got = back.cpu().numpy()
    want = spec.unpack(gc, gs)
    for b, s in enumerate([2, 2, None, 0, None, 1, 2]):
        assert np.all(got[b] == (5.0 if s is None else want[s]))


def test_state_offsets_past_32_bits():
    """States that start beyond 2^31 elements: tree, advance, pack and unpack of
    the last heads of a large batch."""
    import torch
    B, H, d = 1030, 128, 128
    S = torch.zeros((B, H, d, d), device="cuda")
    z = torch.ones((B, H, d), device="cuda")
    assert S.numel() > 2 ** 31
    S1, z1 = state(1, H, d, d, 77)
    S[-1], z[-1] = cuda(S1[0]), cuda(z1[0])
    q, k, v = rows(1, H, 1, d, d, 78, "bf16")
    big = [torch.zeros((B, H, 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for t, x in zip(big, (q, k, v)):
        t[-1] = to_dev(x[0], "bf16")
    out = la.decode_tree(S, z, *big, torch.full((B, 1), -1, dtype=torch.int32, device="cuda"))
    want, scale = spec.decode_tree(S1, z1, q, k, v, [[-1]])
    near(to_host(out[-1:]), want, scale, "bf16", gamma(d, 1, True))
    codes, scales, _ = la.state_pool(B, H, d, d)
    slot = torch.arange(B, dtype=torch.int32, device="cuda")
    la.state_pack(S, codes, scales, slot)
    wc, ws = spec.pack(S1)
    assert np.array_equal(codes[-1:].cpu().numpy(), wc) and np.array_equal(scales[-1:].cpu().numpy(), ws)
    la.state_advance(S, z, big[1], big[2])
    wS, wz, A = spec.advance(S1, z1, k, v)
    near(to_host(S[-1:]), wS, A, "f32", 40 * 2.0 ** -24)
    la.state_unpack(codes, scales, slot, S)
    assert np.array_equal(S[-1:].cpu().numpy(), spec.unpack(wc, ws))


# ---------------------------------------------------------------------------
# All of it together
# ---------------------------------------------------------------------------


def round_of_drafting(S, z, q, k, v, x, parent, p, u, codes, scales, z_pool, slot, alpha):
    """One turn of a server: snapshot, read the tree, verify, move the state."""
    la.state_pack(S, codes, scales, slot, z=z, z_pool=z_pool)
    out = la.decode_tree(S, z, q, k, v, parent, alpha=alpha)
    path, accepted, nxt = la.verify_tree(p, x, parent, u)
    la.state_advance(S, z, k, v, path, accepted, alpha=alpha)
    return out, path, accepted, nxt


def make_turn(seed, B=3, H=4, T=12, d=128, V=999, dtype="bf16"):
    S, z = state(B, H, d, d, seed)
    q, k, v = rows(B, H, T, d, d, seed + 1, dtype)
    rng = np.random.default_rng(seed)
    parent = tree(B, T, seed)
    p = probabilities((B, T + 1, V), rng, "f32", sharp=3.0)
    u = rng.random((B, T + 1)).astype(np.float32)
    x = rng.integers(0, V, (B, T))
    for b in range(B):
        at = -1
        for i in range(T):                               # plant an accepted path
            if parent[b, i] == at and rng.random() < 0.7:
                x[b, i] = spec.draw(p[b, at + 1], u[b, at + 1])
                at = i
    alpha = np.linspace(0.8, 1.0, H).astype(np.float32)
    host = (S, z, q, k, v, x, parent, p, u, alpha)
    slot = rng.permutation(B + 2)[:B]
    dev = [cuda(S), cuda(z)] + [to_dev(y, dtype) for y in (q, k, v)] + [i32(x), i32(parent), cuda(p), cuda(u)]
    return host, dev + list(la.state_pool(B + 2, H, d, d)) + [i32(slot), cuda(alpha)]


def test_a_turn():
    host, dev = make_turn(21)
    S, z, q, k, v, x, parent, p, u, alpha = host
    out, path, accepted, nxt = round_of_drafting(*dev)
    wp, wa, wn = spec.verify_tree(p, x, parent, u)
    assert wa.max() >= 2
    assert np.array_equal(path.cpu().numpy(), wp) and np.array_equal(accepted.cpu().numpy(), wa)
    assert np.array_equal(nxt.cpu().numpy(), wn)
    want, scale = spec.decode_tree(S, z, q, k, v, parent, alpha)
    near(to_host(out), want, scale, "bf16", gamma(128, 1, True))
    wS, wz, A = spec.advance(S, z, k, v, wp, wa, alpha)
    near(to_host(dev[0]), wS, A, "f32", 64 * 2.0 ** -24)
    near(to_host(dev[1]), wz, wz, "f32", 64 * 2.0 ** -24)
    # the accepted tokens' outputs are those of stepping through them
    for b in range(3):
        n = wa[b]
        if n:
            at = wp[b, :n]
            S2, z2, steps = orc.decode_steps_decay(S[b], z[b], q[b][:, at], k[b][:, at], v[b][:, at], alpha=alpha)
            near(to_host(out)[b][:, at], steps, scale[b][:, at], "bf16", gamma(128, 1, True))
    # and the snapshot brings the first state back, to its 8 bits
    back, zb = dev[0].clone(), dev[1].clone()
    la.state_unpack(dev[9], dev[10], dev[12], back, z_pool=dev[11], z=zb)
    assert np.array_equal(back.cpu().numpy(), spec.unpack(*spec.pack(S))) and np.array_equal(zb.cpu().numpy(), z)


def test_a_turn_captured_and_replayed():
    """Captured once, replayed on new inputs: bit for bit the eager calls. Two
    graphs share nothing but what the caller gives them."""
    import torch
    turns = [make_turn(31), make_turn(32)]
    eager = []
    for _, dev in turns:
        mine = [t.clone() for t in dev]
        eager.append([t.clone() for t in round_of_drafting(*mine)] + mine)
    static = [[t.clone() for t in turns[0][1]] for _ in range(2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for dev in static:
        with torch.cuda.stream(side):
            round_of_drafting(*dev)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = round_of_drafting(*dev)
        graphs.append(g)
        outs.append(out)
    for order in ((0, 1), (1, 0)):
        for i, t in enumerate(order):
            for a, b in zip(static[i], turns[t][1]):
                a.copy_(b)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for i, t in enumerate(order):
            for a, b in zip(list(outs[i]) + static[i], eager[t]):
                assert torch.equal(a, b)


def test_turns_on_two_streams():
    """Two turns at once on streams of their own, results as one after the other."""
    import torch
    turns = [make_turn(41, B=5, V=20011), make_turn(42, B=5, V=20011)]
    serial = []
    for _, dev in turns:
        mine = [t.clone() for t in dev]
        serial.append([t.clone() for t in round_of_drafting(*mine)] + mine)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in turns]
    for _ in range(5):
        both = [[t.clone() for t in dev] for _, dev in turns]
        got = []
        for s, dev in zip(streams, both):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(round_of_drafting(*dev))
        torch.cuda.synchronize()
        for g, dev, want in zip(got, both, serial):
            for a, b in zip(list(g) + dev, want):
                assert torch.equal(a, b)


def test_python_checks_on_the_gpu():
    import torch
    S, z = torch.zeros((2, 3, 32, 32), device="cuda"), torch.zeros((2, 3, 32), device="cuda")
    q = torch.zeros((2, 3, 4, 32), device="cuda")
    parent = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    for bad in (dict(k=q[:, :, :3].contiguous()), dict(z=z[:1].contiguous()), dict(parent=parent[:, :2].contiguous()),
                dict(q=q.transpose(1, 2)), dict(v=q.cpu()), dict(count=torch.ones(3, dtype=torch.int32, device="cuda")),
                dict(alpha=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            la.decode_tree(**{**dict(S=S, z=z, q=q, k=q, v=q, parent=parent), **bad})
    for bad in (dict(parent=parent.long()), dict(v=q.bfloat16()), dict(q=q.half(), k=q.half(), v=q.half()),
                dict(S=S.double())):
        with pytest.raises(TypeError):
            la.decode_tree(**{**dict(S=S, z=z, q=q, k=q, v=q, parent=parent), **bad})
    wide = torch.zeros((2, 3, 65, 32), device="cuda")
    with pytest.raises(la.LaError) as e:
        la.decode_tree(S, z, wide, wide, wide, torch.full((2, 65), -1, dtype=torch.int32, device="cuda"))
    assert e.value.status == la.LA_ERR_UNSUPPORTED
    p = torch.full((2, 5, 9), 1 / 9, device="cuda")
    u = torch.zeros((2, 5), device="cuda")
    with pytest.raises(ValueError):
        la.verify_chain(p, p, parent, u)
    with pytest.raises(ValueError):
        la.verify_tree(p, parent, parent[:, :3].contiguous(), u)
    with pytest.raises(TypeError):
        la.verify_tree(p, parent, parent, u.double())
    with pytest.raises(ValueError):
        la.state_advance(S, z, q, q, S_out=S.clone())
    codes, scales, z_pool = la.state_pool(3, 3, 32, 32)
    slot = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        la.state_pack(S, codes, scales, slot, z=z)
    with pytest.raises(ValueError):
        la.state_pack(S, codes, scales[:, :2].contiguous(), slot)
    with pytest.raises(ValueError):
        la.state_unpack(codes, scales, slot[:1].contiguous(), S)
