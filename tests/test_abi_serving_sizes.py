"""Sizes that do not fit 32 bits: refused, not wrapped.  On the host, before any CUDA
call."""
import ctypes

import pytest
import torch

import tensor_transformer_linear_column_b200 as tp
from tensor_transformer_linear_column_b200 import build_lib
from test_abi_serving import APP, APP8, APP_GOOD, BIG, _call


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return tp.load()


@pytest.mark.parametrize("heads", [dict(nq=BIG, nkv=1, t=1), dict(nq=BIG - 1, nkv=1, t=1),
                                   dict(nq=BIG - 7, nkv=10, t=1)])
def test_heads_of_a_token_that_leave_32_bits(lib, heads):
    assert heads["nq"] % heads["nkv"] == 0
    for rows in (None, 0x10000):
        args = dict(APP_GOOD, rows=rows, **{k: heads[k] for k in heads})
        assert _call(lib, "tp_kv_append", APP, args) == tp.TP_ERR_SHAPE
        assert _call(lib, "tp_kv8_append", APP8, dict(args, ks=0x10000, vs=0x10000)) == tp.TP_ERR_SHAPE
