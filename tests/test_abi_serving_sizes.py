"""Sizes that do not fit 32 bits: refused, not wrapped.  On the host, before any CUDA
call."""
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


BEYOND = 2 ** 32  # as a C int: 0


@pytest.mark.parametrize("parents", [[BEYOND - 1, 0], [-1, BEYOND], [-1, -BEYOND], [2 ** 31]])
def test_parents_beyond_32_bits(parents):
    with pytest.raises(ValueError, match="32 bits"):
        tp.tp_tree_mask(parents)


def test_lengths_beyond_32_bits():
    qkv = torch.zeros(4, 12 * 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 20, 128, dtype=torch.bfloat16)
    k8, s = torch.zeros(2, 20, 128, dtype=torch.uint8), torch.zeros(2, 20)
    heads = (8, 2, 128, 1)
    for past in (BEYOND + 4, -BEYOND + 4, 2 ** 31):
        for call in (lambda: tp.tp_kv_append(qkv, k, k, past, *heads),
                     lambda: tp.tp_kv8_append(qkv, k8, s, k8, s, past, *heads),
                     lambda: tp.tp_kv8_read(k8, s, k8, s, past, 4, 1),
                     lambda: tp.tp_kv8_read(k8, s, k8, s, 4, past, 1),
                     lambda: tp.tp_qk_norm_rope(qkv, past, *heads),
                     lambda: tp.tp_qk_norm_rope_backward(qkv, qkv, past, *heads),
                     lambda: tp.tp_attn_tree_workspace_bytes(4, past, 8, 2, 128),
                     lambda: tp.tp_attn_decode_kv8_workspace_bytes(4, past, 8, 2, 128),
                     lambda: tp.tp_attn_tree_workspace_bytes_upto(4, past, 8, 2, 128)):
            with pytest.raises(ValueError, match="32 bits"):
                call()


@pytest.mark.gpu
def test_attention_and_read_beyond_32_bits_on_the_gpu():
    qkv = torch.zeros(4, 12 * 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 20, 128, dtype=torch.bfloat16, device="cuda")
    k8, s = torch.zeros(2, 20, 128, dtype=torch.uint8, device="cuda"), torch.zeros(2, 20, device="cuda")
    for call in (lambda: tp.tp_attn_tree(qkv, k, k, BEYOND + 4, 8, 2, 128, 1),
                 lambda: tp.tp_attn_decode_kv8(qkv, k8, s, k8, s, BEYOND + 4, 8, 2, 128, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    # a range past the cache is refused without memory for it
    with pytest.raises(tp.TPError) as e:
        tp.tp_kv8_read(k8, s, k8, s, 5, 2 ** 31 - 6, 1)
    assert e.value.status == tp.TP_ERR_SHAPE
