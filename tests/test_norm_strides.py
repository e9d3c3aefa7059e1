"""Strides of the rows that the gradient of the norm with rotation writes: refused, before
any device work, where one row would begin inside another."""

import ctypes

import pytest

import causal_linear_attention_la_gb300 as la
from helpers import build_lib


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib()
    return la.lib()


def strides(*s):
    return (ctypes.c_longlong * 3)(*s)


def call(B, N, Hq, dq_stride, dtype=la.LA_BF16, d=32):
    return la.la_qk_norm_rotate_backward(1024, None, None, None, None, None, 2048, None, 4096, None, None, None, B, N, Hq, 0, d, 0,
                                         strides(N * Hq * d, Hq * d, d), None, strides(*dq_stride), None, la.LA_NORM_L2, 0, 1e-6,
                                         dtype, None, 0, None)


@pytest.mark.parametrize("dtype", [la.LA_BF16, la.LA_F32])
@pytest.mark.parametrize("bad", [(1024, 128, 16), (1024, 24, 32), (8, 128, 32), (16, 16, 16)])
def test_rows_inside_each_other(lib, bad, dtype):
    assert call(2, 5, 4, bad, dtype) == la.LA_ERR_INVALID_ARG
    assert b"below d" in lib.la_last_error()


def test_a_stride_that_is_never_taken_may_be_anything(lib):
    """One token of one head: neither its stride nor the batch's is taken (rows that cannot be
    read end the call before a launch: misaligned)."""
    assert la.la_qk_norm_rotate_backward(1032, None, None, None, None, None, 2048, None, 4096, None, None, None, 1, 1, 1, 0, 32, 0,
                                         strides(0, 0, 0), None, strides(0, 0, 0), None, la.LA_NORM_L2, 0, 1e-6, la.LA_BF16, None, 0,
                                         None) == la.LA_ERR_INVALID_ARG
    assert b"16-byte aligned" in lib.la_last_error()
