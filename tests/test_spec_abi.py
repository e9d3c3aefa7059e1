"""Host-only checks of the speculative-decoding entry points: refusals come
before any device work, empty problems are accepted, and the Python layer
checks what it is given."""

import pytest
import torch

import causal_linear_attention_la_gb300 as la
from helpers import build_lib

INVALID, UNSUPPORTED, OK = la.LA_ERR_INVALID_ARG, la.LA_ERR_UNSUPPORTED, la.LA_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib()
    return la.lib()


TREE = dict(S=1024, z=1024, q=1024, k=1024, v=1024, parent=1024, count=None, out=2048, B=2, H=3, T=4, dk=64, dv=64,
            alpha=None, eps=1e-6, dtype=la.LA_BF16, stream=None)


def test_tree_refusals(lib):
    f = lambda **kw: la.la_decode_tree(**{**TREE, **kw})  # noqa: E731
    for name in ("S", "z", "q", "k", "v", "parent", "out"):
        assert f(**{name: None}) == INVALID, name
        assert b"la_decode_tree" in lib.la_last_error() and b"non-NULL" in lib.la_last_error()
    for name in ("S", "z", "q", "k", "v", "out"):
        assert f(**{name: 1032}) == INVALID, name
    for name in ("parent", "count", "alpha"):
        assert f(**{name: 1026}) == INVALID, name
    assert f(T=la.LA_TREE_MAX + 1) == UNSUPPORTED
    assert f(T=-1) == INVALID and f(B=-1) == INVALID and f(H=-2) == INVALID
    assert f(dk=48) == UNSUPPORTED and f(dv=256) == UNSUPPORTED and f(dtype=2) == UNSUPPORTED
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(eps=float("inf")) == INVALID
    assert f(B=1 << 20, H=1 << 20) == INVALID
    assert f(B=0) == OK and f(H=0) == OK and f(T=0, q=None) == OK


def test_tree_delta_refusals():
    d = {k: v for k, v in TREE.items() if k not in ("z", "alpha", "eps")}
    f = lambda **kw: la.la_decode_tree_delta(**{**d, **kw})  # noqa: E731
    for name in ("S", "q", "k", "v", "parent", "out"):
        assert f(**{name: None}) == INVALID, name
    assert f(q=1028) == INVALID and f(parent=3) == INVALID
    assert f(T=65) == UNSUPPORTED and f(dk=24) == UNSUPPORTED
    assert f(B=0) == OK and f(T=0) == OK


def test_tree_path():
    assert la.la_tree_path(128, 128, la.LA_BF16) == 1 and la.la_tree_path(64, 128, la.LA_BF16) == 1
    assert la.la_tree_path(128, 128, la.LA_F32) == 0 and la.la_tree_path(32, 64, la.LA_BF16) == 0
    assert la.la_tree_path(48, 64, la.LA_BF16) == -1 and la.la_tree_path(64, 64, 7) == -1
    prev = la.la_set_path(la.LA_PATH_SIMT)
    try:
        assert la.la_tree_path(128, 128, la.LA_BF16) == 0
    finally:
        la.la_set_path(prev)


def test_verify_refusals(lib):
    c = dict(target=1024, draft=1024, tokens=1024, count=None, uniform=1024, accepted=2048, next=2048, B=2, T=3, V=100,
             dtype=la.LA_F32, stream=None)
    f = lambda **kw: la.la_verify_chain(**{**c, **kw})  # noqa: E731
    for name in ("target", "draft", "tokens", "uniform", "accepted", "next"):
        assert f(**{name: None}) == INVALID, name
        assert b"la_verify_chain" in lib.la_last_error()
    assert f(target=1028) == INVALID and f(draft=1032) == INVALID
    for name in ("tokens", "count", "uniform", "accepted", "next"):
        assert f(**{name: 1026}) == INVALID, name
    assert f(V=0) == INVALID and f(V=(1 << 30) + 1) == INVALID and f(T=-1) == INVALID and f(B=-1) == INVALID
    assert f(T=65) == UNSUPPORTED and f(dtype=5) == UNSUPPORTED and f(B=(1 << 27) + 1) == INVALID
    assert f(B=0, target=None) == OK
    t = dict(target=1024, tokens=1024, parent=1024, count=None, uniform=1024, path=2048, accepted=2048, next=2048, B=2, T=3,
             V=100, dtype=la.LA_F32, stream=None)
    g = lambda **kw: la.la_verify_tree(**{**t, **kw})  # noqa: E731
    for name in ("target", "tokens", "parent", "uniform", "path", "accepted", "next"):
        assert g(**{name: None}) == INVALID, name
    for name in ("tokens", "parent", "count", "uniform", "path", "accepted", "next"):
        assert g(**{name: 1025}) == INVALID, name
    assert g(target=1030) == INVALID and g(T=65) == UNSUPPORTED and g(V=-4) == INVALID
    assert g(B=0, target=None) == OK


def test_advance_refusals(lib):
    c = dict(S=1024, z=1024, k=1024, v=1024, path=None, accepted=None, S_out=4096, z_out=4096, B=2, H=3, T=4, dk=64, dv=64,
             alpha=None, dtype=la.LA_BF16, stream=None)
    f = lambda **kw: la.la_state_advance(**{**c, **kw})  # noqa: E731
    for name in ("S", "z", "k", "v", "S_out", "z_out"):
        assert f(**{name: None}) == INVALID, name
        assert b"la_state_advance" in lib.la_last_error()
        assert f(**{name: 1032}) == INVALID, name
    for name in ("path", "accepted", "alpha"):
        assert f(**{name: 1026}) == INVALID, name
    assert f(S_out=1024) == INVALID and b"in place" in lib.la_last_error()      # S in place, z not
    assert f(T=-1) == INVALID and f(dk=20) == UNSUPPORTED and f(dtype=9) == UNSUPPORTED
    assert f(B=0) == OK and f(H=0, S=None) == OK
    assert f(T=0, k=None, v=None, S_out=1024, z_out=1024) == OK                 # nothing to do in place
    d = {k: v for k, v in c.items() if k not in ("z", "z_out", "alpha")}
    g = lambda **kw: la.la_state_advance_delta(**{**d, **kw})  # noqa: E731
    for name in ("S", "k", "v", "S_out"):
        assert g(**{name: None}) == INVALID, name
    assert g(k=1025) == INVALID and g(T=-3) == INVALID and g(dv=8) == UNSUPPORTED
    assert g(B=0) == OK and g(T=0, k=None, v=None, S_out=1024) == OK


def test_pool_refusals(lib):
    c = dict(S=1024, z=1024, codes=1024, scales=1024, z_pool=1024, slot=1024, B=2, H=3, dk=64, dv=64, slots=5, stream=None)
    for f0, who in ((la.la_state_pack, b"la_state_pack"), (la.la_state_unpack, b"la_state_unpack")):
        f = lambda **kw: f0(**{**c, **kw})  # noqa: E731
        for name in ("S", "codes", "scales", "slot"):
            assert f(**{name: None}) == INVALID, name
            assert who in lib.la_last_error()
        for name in ("S", "z", "codes", "z_pool"):
            assert f(**{name: 1032}) == INVALID, name
        assert f(z=None) == INVALID and f(z_pool=None) == INVALID and f(slot=1026) == INVALID
        assert f(slots=-1) == INVALID and f(B=-1) == INVALID and f(dk=12) == UNSUPPORTED and f(dv=256) == UNSUPPORTED
        assert f(H=1 << 17, dk=128, dv=128) == INVALID and b"too large" in lib.la_last_error()
        assert f(B=0) == OK and f(slots=0) == OK


def test_python_layer_checks():
    S, z = torch.zeros(2, 3, 16, 16), torch.zeros(2, 3, 16)
    q = torch.zeros(2, 3, 4, 16)
    parent = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        la.decode_tree(S, z, q, q, q, parent)
    with pytest.raises(ValueError, match="CUDA"):
        la.decode_tree_delta(S, q, q, q, parent)
    with pytest.raises(ValueError, match="CUDA"):
        la.state_advance(S, z, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        la.state_advance_delta(S, q, q)
    p = torch.zeros(2, 5, 7)
    with pytest.raises(ValueError, match="CUDA"):
        la.verify_chain(p, p[:, :4], parent, torch.zeros(2, 5))
    with pytest.raises(ValueError, match="CUDA"):
        la.verify_tree(p, parent, parent, torch.zeros(2, 5))
    codes, scales, z_pool = la.state_pool(4, 3, 16, 16, device="cpu")
    assert codes.shape == (4, 3, 16, 16) and scales.shape == (4, 3, 16, 1) and z_pool.shape == (4, 3, 16)
    assert la.state_pool(1, 2, 32, 128, device="cpu")[1].shape == (1, 2, 32, 4)
    slot = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        la.state_pack(S, codes, scales, slot)
    with pytest.raises(ValueError, match="CUDA"):
        la.state_unpack(codes, scales, slot, S)


def test_python_shape_checks():
    """The checks that stand between a wrong shape and the kernels."""
    t = torch.zeros(2, 3)
    la._need_like(-1, ("a", t, torch.float32, (2, 3)), ("b", None, torch.int32, (9,)))
    with pytest.raises(ValueError, match="a must have shape"):
        la._need_like(-1, ("a", t, torch.float32, (3, 2)))
    with pytest.raises(TypeError, match="float64"):
        la._need_like(-1, ("a", t, torch.float64, (2, 3)))
    with pytest.raises(ValueError, match="contiguous"):
        la._need_like(-1, ("a", t.t(), torch.float32, (3, 2)))
    with pytest.raises(ValueError, match="on cuda:0"):
        la._need_like(0, ("a", t, torch.float32, (2, 3)))


def test_pack_refuses_more_sequences_than_it_can_look_through(lib):
    """Each CTA reads the slots of all later sequences: B^2 / 2 reads."""
    c = dict(S=1024, z=None, codes=1024, scales=1024, z_pool=None, slot=1024, H=1, dk=16, dv=16, slots=0, stream=None)
    assert la.la_state_pack(B=1 << 20, **c) == OK                 # (no slots: nothing is launched)
    assert la.la_state_pack(B=(1 << 20) + 1, **c) == UNSUPPORTED and b"at most 1048576" in lib.la_last_error()
    assert la.la_state_unpack(B=(1 << 20) + 1, **c) == OK
