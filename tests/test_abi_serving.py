"""Argument checks of the norm / rotation, cache and tree-attention calls, on the
host: fake pointers that are never dereferenced, each call refused before any
CUDA call."""
import ctypes

import pytest
import torch

import tensor_transformer_linear_column_b200 as tp
from tensor_transformer_linear_column_b200 import build_lib

GOOD = 0x10000
ODD = 0x10008 + 1
BIG = 2 ** 31 - 1
N, A, S, D, W, U = (tp.TP_ERR_NULL, tp.TP_ERR_ALIGN, tp.TP_ERR_SHAPE, tp.TP_ERR_TP_DEGREE,
                    tp.TP_ERR_WORKSPACE, tp.TP_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return tp.load()


def _call(lib, name, order, good, **change):
    args = dict(good, **change)
    assert set(change) <= set(order)
    return getattr(lib, name)(*[args[k] for k in order], None)


QK = "qkv gq gk fr pos T past nq nkv d rot layout eps t out".split()
QK_GOOD = dict(qkv=GOOD, gq=GOOD, gk=GOOD, fr=GOOD, pos=None, T=4, past=0, nq=8, nkv=2, d=128,
               rot=128, layout=0, eps=1e-5, t=1, out=GOOD)
QK_BAD = [
    (N, dict(qkv=None)), (N, dict(gq=None)), (N, dict(gk=None)), (N, dict(fr=None)),
    (A, dict(qkv=ODD)), (A, dict(gq=ODD)), (A, dict(fr=ODD)), (A, dict(pos=ODD)),
    (S, dict(T=0)), (S, dict(past=-1)), (S, dict(nq=0)), (S, dict(nkv=0)), (S, dict(nq=7)),
    (S, dict(d=0)), (S, dict(d=120)), (S, dict(d=272)), (S, dict(rot=-16)), (S, dict(rot=8)),
    (S, dict(rot=144)), (S, dict(eps=-1.0)), (S, dict(eps=float("nan"))),
    (S, dict(past=BIG)), (S, dict(nq=1 << 30, nkv=1 << 29)), (S, dict(nq=4092, nkv=4)),
    (U, dict(layout=2)), (U, dict(layout=-1)), (D, dict(t=0)), (D, dict(t=4)), (D, dict(t=3)),
]


@pytest.mark.parametrize("status,change", QK_BAD + [(N, dict(out=None)), (A, dict(out=ODD))])
def test_qk_norm_rope(lib, status, change):
    assert _call(lib, "tp_qk_norm_rope", QK, QK_GOOD, **change) == status


BACK = "qkv gq gk fr pos dout T past nq nkv d rot layout eps t dqkv dgq dgk ws bytes".split()
BACK_GOOD = dict({k: v for k, v in QK_GOOD.items() if k != "out"}, dout=GOOD, dqkv=GOOD, dgq=GOOD,
                 dgk=GOOD, ws=GOOD, bytes=1 << 30)


@pytest.mark.parametrize("status,change", QK_BAD + [
    (N, dict(dout=None)), (N, dict(dqkv=None)), (N, dict(dgq=None)), (N, dict(dgk=None)),
    (A, dict(dout=ODD)), (A, dict(dqkv=ODD)), (A, dict(dgq=ODD)), (A, dict(dgk=ODD)),
    (A, dict(ws=ODD)), (W, dict(ws=None)), (W, dict(bytes=0)),
    (W, dict(bytes=296 * 2 * 128 * 4 - 1)),
])
def test_qk_norm_rope_backward(lib, status, change):
    assert _call(lib, "tp_qk_norm_rope_backward", BACK, BACK_GOOD, **change) == status


def test_qk_backward_workspace():
    f = tp.tp_qk_norm_rope_backward_workspace_bytes
    assert f(4, 128) == 296 * 2 * 128 * 4
    assert f(1, 16) == f(10 ** 6, 16) == 296 * 2 * 16 * 4  # whatever T is
    assert f(0, 128) == f(4, 120) == f(4, 0) == f(4, 272) == 0


APP = "qkv rows k v T n past max_len nq nkv d t".split()
APP_GOOD = dict(qkv=GOOD, rows=None, k=GOOD, v=GOOD, T=4, n=4, past=10, max_len=14, nq=8, nkv=2,
                d=128, t=2)
APP8 = "qkv rows k ks v vs T n past max_len nq nkv d t".split()
APP_BAD = [
    (N, dict(qkv=None)), (N, dict(k=None)), (N, dict(v=None)), (A, dict(qkv=ODD)),
    (A, dict(rows=ODD)), (A, dict(k=ODD)), (A, dict(v=ODD)), (S, dict(T=0, n=1)), (S, dict(n=0)),
    (S, dict(n=5, max_len=99)), (S, dict(past=-1)), (S, dict(past=11)), (S, dict(past=BIG)),
    (S, dict(max_len=13)), (S, dict(max_len=BIG)), (S, dict(max_len=0)), (S, dict(nq=9)),
    (S, dict(nkv=0)), (S, dict(d=100)), (S, dict(d=512)), (S, dict(rows=GOOD, n=5)),
    (S, dict(nq=1 << 16, nkv=1 << 16)), (D, dict(t=0)), (D, dict(t=4)),
]


@pytest.mark.parametrize("status,change", APP_BAD)
def test_kv_append(lib, status, change):
    assert _call(lib, "tp_kv_append", APP, APP_GOOD, **change) == status
    assert _call(lib, "tp_kv8_append", APP8, dict(APP_GOOD, ks=GOOD, vs=GOOD), **change) == status


@pytest.mark.parametrize("status,change", [(N, dict(ks=None)), (N, dict(vs=None)), (A, dict(ks=ODD)),
                                           (A, dict(vs=ODD))])
def test_kv8_append_scales(lib, status, change):
    assert _call(lib, "tp_kv8_append", APP8, dict(APP_GOOD, ks=GOOD, vs=GOOD), **change) == status


READ = "k ks v vs start count max_len nkv d t ko vo out_len".split()
READ_GOOD = dict(k=GOOD, ks=GOOD, v=GOOD, vs=GOOD, start=2, count=5, max_len=7, nkv=4, d=128, t=2,
                 ko=GOOD, vo=GOOD, out_len=7)


@pytest.mark.parametrize("status,change", [
    *[(N, {k: None}) for k in ("k", "ks", "v", "vs", "ko", "vo")],
    *[(A, {k: ODD}) for k in ("k", "ks", "v", "vs", "ko", "vo")],
    (S, dict(start=-1)), (S, dict(start=3)), (S, dict(start=BIG)), (S, dict(count=0)),
    (S, dict(count=BIG)), (S, dict(max_len=6)), (S, dict(out_len=6)), (S, dict(out_len=0)),
    (S, dict(nkv=0)), (S, dict(d=8)), (S, dict(d=130)), (D, dict(t=0)), (D, dict(t=3)),
])
def test_kv8_read(lib, status, change):
    assert _call(lib, "tp_kv8_read", READ, READ_GOOD, **change) == status


TREE = "qkv k v mask T past max_len nq nkv d t ctx ws bytes".split()
TREE8 = "qkv k ks v vs mask T past max_len nq nkv d t ctx ws bytes".split()
TREE_GOOD = dict(qkv=GOOD, k=GOOD, v=GOOD, mask=None, T=4, past=100, max_len=104, nq=8, nkv=2,
                 d=128, t=2, ctx=GOOD, ws=GOOD, bytes=1 << 30)


@pytest.mark.parametrize("status,change", [
    *[(N, {k: None}) for k in ("qkv", "k", "v", "ctx")],
    *[(A, {k: ODD}) for k in ("qkv", "k", "v", "ctx", "mask", "ws")],
    (S, dict(T=0)), (S, dict(past=-1)), (S, dict(past=101)), (S, dict(past=BIG)),
    (S, dict(max_len=103)), (S, dict(max_len=BIG)), (S, dict(nq=9)), (S, dict(nkv=0)),
    (S, dict(nq=0)), (S, dict(d=0)), (U, dict(d=64)), (U, dict(T=129, max_len=300)),
    (U, dict(nq=34)), (D, dict(t=0)), (D, dict(t=4)), (W, dict(ws=None)), (W, dict(bytes=100)),
])
def test_tree_attention(lib, status, change):
    assert _call(lib, "tp_attn_tree", TREE, TREE_GOOD, **change) == status
    good8 = dict(TREE_GOOD, ks=GOOD, vs=GOOD)
    assert _call(lib, "tp_attn_decode_kv8", TREE8, good8, **change) == status


@pytest.mark.parametrize("status,change", [(N, dict(ks=None)), (N, dict(vs=None)), (A, dict(ks=ODD)),
                                           (A, dict(vs=ODD))])
def test_tree_attention_scales(lib, status, change):
    good8 = dict(TREE_GOOD, ks=GOOD, vs=GOOD)
    assert _call(lib, "tp_attn_decode_kv8", TREE8, good8, **change) == status


def test_tree_workspace():
    f = tp.tp_attn_tree_workspace_bytes
    assert f(4, 0, 8, 2, 128) == 0
    assert f(1, 1, 8, 2, 128) > 0
    # a row is 128 sums, a maximum and a sum of weights; rows fill tiles of 16 to 128
    assert f(1, 1, 8, 2, 128) == 2 * 16 * 128 * 4 + 256
    for bad in ((129, 5, 8, 2, 128), (0, 5, 8, 2, 128), (4, -1, 8, 2, 128), (4, 5, 9, 2, 128),
                (4, 5, 34, 2, 128), (4, 5, 8, 2, 64)):
        assert f(*bad) == 0
    # the partials of a call stay small next to the cache that it reads
    for T in (1, 4, 64, 128):
        for past in (1000, 65536, 1 << 20):
            assert f(T, past, 64, 8, 128) < 128 << 20


def test_8_bit_workspace():
    both, own = tp.tp_attn_tree_workspace_bytes, tp.tp_attn_decode_kv8_workspace_bytes
    for T in (1, 4, 8, 9, 33, 128):
        for past in (0, 1, 128, 1000, 2048, 2049, 65536):
            for nq, nkv in ((8, 2), (64, 8), (28, 4), (16, 1), (64, 64)):
                assert 0 <= own(T, past, nq, nkv, 128) <= both(T, past, nq, nkv, 128)
    assert own(1, 1000, 64, 8, 128) == 0 and own(1, 65536, 64, 8, 128) > 0
    assert own(129, 5, 8, 2, 128) == 0 and own(4, 5, 8, 2, 64) == 0


def test_tree_mask_pointers(lib):
    p = (ctypes.c_int32 * 2)(-1, 0)
    m = (ctypes.c_uint64 * 2)()
    assert lib.tp_tree_mask(None, 2, ctypes.addressof(m)) == N
    assert lib.tp_tree_mask(ctypes.addressof(p), 2, None) == N
    assert lib.tp_tree_mask(ctypes.addressof(p), 0, ctypes.addressof(m)) == S
    assert lib.tp_tree_mask(ctypes.addressof(p), 2, ctypes.addressof(m)) == tp.TP_OK
    assert list(m) == [1, 3]


def test_binding_rejects_host_tensors_and_wrong_shapes():
    qkv = torch.zeros(4, 12 * 128, dtype=torch.bfloat16)
    k = torch.zeros(2, 20, 128, dtype=torch.bfloat16)
    k8, s = torch.zeros(2, 20, 128, dtype=torch.uint8), torch.zeros(2, 20)
    heads = (8, 2, 128, 1)
    for call in (lambda: tp.tp_qk_norm_rope(qkv, 0, *heads),
                 lambda: tp.tp_qk_norm_rope_backward(qkv, qkv, 0, *heads),
                 lambda: tp.tp_kv_append(qkv, k, k, 0, *heads),
                 lambda: tp.tp_kv8_append(qkv, k8, s, k8, s, 0, *heads),
                 lambda: tp.tp_kv8_read(k8, s, k8, s, 0, 4, 1),
                 lambda: tp.tp_attn_tree(qkv, k, k, 4, *heads),
                 lambda: tp.tp_attn_decode_kv8(qkv, k8, s, k8, s, 4, *heads),
                 # shapes are looked at before the device
                 lambda: tp.tp_kv_append(qkv, k, k, 0, 8, 4, 128, 1),
                 lambda: tp.tp_attn_tree(qkv, k[:, :, :64], k[:, :, :64], 4, *heads),
                 lambda: tp.tp_attn_tree(qkv[:, :-1], k, k, 4, *heads)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_rejects_wrong_tensors_on_the_gpu():
    qkv = torch.zeros(4, 12 * 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 20, 128, dtype=torch.bfloat16, device="cuda")
    k8, s = torch.zeros(2, 20, 128, dtype=torch.uint8, device="cuda"), torch.zeros(2, 20, device="cuda")
    mask = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    fr = torch.ones(64, device="cuda")
    heads = (8, 2, 128, 1)
    bad = [
        lambda: tp.tp_attn_tree(qkv, k, k, 4, *heads, tree_mask=mask.int()),
        lambda: tp.tp_attn_tree(qkv, k, k, 4, *heads, tree_mask=mask[:3]),
        lambda: tp.tp_attn_tree(qkv, k, k, 4, *heads, tree_mask=mask.cpu()),
        lambda: tp.tp_attn_tree(qkv, k.transpose(0, 1).contiguous().transpose(0, 1), k, 4, *heads),
        lambda: tp.tp_attn_tree(qkv, k, k, 4, *heads, ctx=qkv),
        lambda: tp.tp_attn_decode_kv8(qkv, k, s, k, s, 4, *heads),
        lambda: tp.tp_attn_decode_kv8(qkv, k8, s.double(), k8, s, 4, *heads),
        lambda: tp.tp_attn_decode_kv8(qkv, k8, s[:, :19], k8, s, 4, *heads),
        lambda: tp.tp_kv_append(qkv, k, k, 0, *heads, rows=mask),
        lambda: tp.tp_kv_append(qkv, k, k, 0, *heads, rows=torch.zeros(2, 2, dtype=torch.int32,
                                                                       device="cuda")),
        lambda: tp.tp_kv8_read(k8, s, k8, s, 0, 4, 1, k_out=k8),
        lambda: tp.tp_kv8_read(k8, s, k8, s, 0, 4, 1, k_out=k, v_out=k[:, :19].contiguous()),
        lambda: tp.tp_qk_norm_rope(qkv, 0, *heads, gamma_q=gamma, gamma_k=gamma[:64]),
        lambda: tp.tp_qk_norm_rope(qkv, 0, *heads, inv_freq=fr.half()),
        lambda: tp.tp_qk_norm_rope(qkv, 0, *heads, inv_freq=fr, positions=mask[:, 0]),
        lambda: tp.tp_qk_norm_rope(qkv, 0, *heads, inv_freq=fr, out=qkv[:3]),
        lambda: tp.tp_qk_norm_rope(qkv.float(), 0, *heads, inv_freq=fr),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was not refused")
    refused = [
        (tp.TP_ERR_NULL, lambda: tp.tp_qk_norm_rope(qkv, 0, *heads, gamma_q=gamma)),
        (tp.TP_ERR_SHAPE, lambda: tp.tp_attn_tree(qkv, k, k, 17, *heads)),
        (tp.TP_ERR_SHAPE, lambda: tp.tp_kv_append(qkv, k, k, 17, *heads)),
        (tp.TP_ERR_SHAPE, lambda: tp.tp_kv8_read(k8, s, k8, s, 0, 21, 1)),
        (tp.TP_ERR_SHAPE, lambda: tp.tp_kv8_read(k8, s, k8, s, 0, 0, 1)),
        (tp.TP_ERR_WORKSPACE, lambda: tp.tp_attn_tree(
            qkv, k, k, 4, *heads, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))),
    ]
    for status, call in refused:
        with pytest.raises(tp.TPError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
