"""One workspace for a cache that grows: what a length needs may be less than what a
shorter one does, and tp_attn_tree_workspace_bytes_upto covers them all."""
import pytest
import torch

import tensor_transformer_linear_column_b200 as tp

HEADS = [(64, 8), (8, 2), (28, 4), (16, 1), (40, 40), (64, 64), (9, 3), (512, 256), (2048, 1024)]


@pytest.mark.parametrize("nq,nkv", HEADS)
@pytest.mark.parametrize("T", [1, 4, 8, 21, 64, 65, 128])
def test_covers_every_shorter_cache(T, nq, nkv):
    both, eight = tp.tp_attn_tree_workspace_bytes, tp.tp_attn_decode_kv8_workspace_bytes
    upto = tp.tp_attn_tree_workspace_bytes_upto
    most = 0
    for past in [1, *range(65, 40000, 128), 40001, 65536, 1 << 20, (1 << 20) + 1, 2 ** 31 - 129]:
        most = max(most, both(T, past, nq, nkv, 128), eight(T, past, nq, nkv, 128))
        assert upto(T, past, nq, nkv, 128) >= most, past


def test_the_size_of_a_final_length_does_not_cover_the_way_there():
    # 4 tokens of 64 / 8 heads, 8 bits: more at 4736 than at 8192
    eight = tp.tp_attn_decode_kv8_workspace_bytes
    assert eight(4, 4736, 64, 8, 128) > eight(4, 8192, 64, 8, 128)
    assert tp.tp_attn_tree_workspace_bytes_upto(4, 8192, 64, 8, 128) >= eight(4, 4736, 64, 8, 128)


def test_arguments_out_of_range_and_the_size_stays_small():
    upto = tp.tp_attn_tree_workspace_bytes_upto
    for bad in ((129, 5, 8, 2, 128), (0, 5, 8, 2, 128), (4, -1, 8, 2, 128), (4, 5, 9, 2, 128),
                (4, 5, 34, 2, 128), (4, 5, 8, 2, 64), (4, 0, 8, 2, 128)):
        assert upto(*bad) == 0
    for T in (1, 4, 64, 128):
        assert 0 < upto(T, 1 << 20, 64, 8, 128) < 128 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("T", [4, 64])
def test_one_buffer_for_a_growing_cache(T, eight):
    nq, nkv, d, last = 64, 8, 128, 8192
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(T, (nq + 2 * nkv) * d, generator=g).to(torch.bfloat16).cuda()
    kv = [torch.randn(nkv, last + T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    call = tp.tp_attn_decode_kv8 if eight else tp.tp_attn_tree
    if eight:
        rows = torch.cat([torch.zeros(last + T, nq * d, dtype=torch.bfloat16, device="cuda"),
                          *[m.transpose(0, 1).reshape(last + T, -1) for m in kv]], 1)
        cache = [torch.zeros(nkv, last + T, d, dtype=torch.uint8, device="cuda"),
                 torch.zeros(nkv, last + T, device="cuda")] * 2
        cache = [m.clone() for m in cache]
        tp.tp_kv8_append(rows, *cache, 0, nq, nkv, d, 1)
    else:
        cache = kv
    ws = torch.empty(tp.tp_attn_tree_workspace_bytes_upto(T, last, nq, nkv, d), dtype=torch.uint8,
                     device="cuda")
    for past in (1, 1000, 2200, 4736, 4737, 8064, 8192):
        a, b = [m.clone() for m in cache], [m.clone() for m in cache]
        assert torch.equal(call(qkv, *a, past, nq, nkv, d, 1, workspace=ws),
                           call(qkv, *b, past, nq, nkv, d, 1))
