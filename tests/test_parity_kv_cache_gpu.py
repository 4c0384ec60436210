"""GPU parity of the cache calls against the fp64 oracle: codes, scales and
bf16 values are defined by single roundings of fp32 quotients and products, so
every bit has to agree; rows outside the written range keep theirs."""
import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp

pytestmark = pytest.mark.gpu


def _qkv(T, nq, nkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, nq + 2 * nkv, d, generator=g)
    x *= torch.exp(2 * torch.randn(T, nq + 2 * nkv, 1, generator=g))
    return x.to(torch.bfloat16).reshape(T, -1)


def _caches(nkv, n, d):
    """8-bit caches whose untouched rows would show."""
    return (torch.full((nkv, n, d), 0x55, dtype=torch.uint8), torch.full((nkv, n), 7.5),
            torch.full((nkv, n, d), 0x2a, dtype=torch.uint8), torch.full((nkv, n), -3.0))


SHAPES = [(1, 64, 8, 128, 0), (37, 8, 2, 128, 100), (5, 9, 3, 80, 3), (130, 4, 4, 16, 1),
          (3, 2, 1, 256, 12), (64, 6, 2, 96, 0), (2, 32, 32, 64, 5)]


def _new(x, nq, nkv, d, which):
    T = x.shape[0]
    at = nq + which * nkv
    return x.reshape(T, -1, d)[:, at:at + nkv].transpose(0, 1)  # [nkv, T, d]


@pytest.mark.parametrize("T,nq,nkv,d,past", SHAPES)
@pytest.mark.parametrize("pick", [False, True])
def test_append8_and_read(T, nq, nkv, d, past, pick):
    x = _qkv(T, nq, nkv, d, T + d)
    x.view(T, -1, d)[0, nq] = 0  # a key of zeros
    rows = torch.tensor([(3 * j + 1) % T for j in range(T // 2 + 1)], dtype=torch.int32) if pick \
        else None
    n = T if rows is None else len(rows)
    host = _caches(nkv, past + n + 4, d)
    dev = [c.cuda() for c in host]
    tp.tp_kv8_append(x.cuda(), *dev, past, nq, nkv, d, 1, rows=None if rows is None else rows.cuda())
    torch.cuda.synchronize()
    for which in (0, 1):
        src = _new(x, nq, nkv, d, which)
        if rows is not None:
            src = src[:, rows.long()]
        codes, scale = oracle.kv8_quantize(src)
        want_c, want_s = host[2 * which].clone(), host[2 * which + 1].clone()
        want_c[:, past:past + n] = torch.from_numpy(codes)
        want_s[:, past:past + n] = torch.from_numpy(scale)
        assert torch.equal(dev[2 * which].cpu(), want_c)
        assert torch.equal(dev[2 * which + 1].cpu(), want_s)
    # read back a range that starts and ends inside
    start, count = past, n
    if n > 2:
        start, count = past + 1, n - 2
    k = torch.full((nkv, past + n + 9, d), 5.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 6.0)
    tp.tp_kv8_read(*dev, start, count, 1, k_out=k, v_out=v)
    for which, (got, fill) in enumerate(((k, 5.0), (v, 6.0))):
        want = torch.full_like(got.cpu(), fill)
        val = torch.from_numpy(oracle.E4M3_TABLE[dev[2 * which].cpu().numpy()]).float() * \
            dev[2 * which + 1].cpu()[..., None]
        want[:, start:start + count] = val[:, start:start + count].to(torch.bfloat16)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("T,nq,nkv,d,past", SHAPES)
def test_append_bf16(T, nq, nkv, d, past):
    x = _qkv(T, nq, nkv, d, T + d)
    for rows in (None, torch.tensor([T - 1] * 2 + [0], dtype=torch.int32)):
        n = T if rows is None else 3
        k = torch.full((nkv, past + n + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, 6.0)
        tp.tp_kv_append(x.cuda(), k, v, past, nq, nkv, d, 1,
                        rows=None if rows is None else rows.cuda())
        for which, (got, fill) in enumerate(((k, 5.0), (v, 6.0))):
            want = torch.full_like(got.cpu(), fill)
            src = _new(x, nq, nkv, d, which)
            want[:, past:past + n] = src if rows is None else src[:, rows.long()]
            assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("eight", [False, True])
def test_row_indices_outside_qkv_leave_their_rows(eight):
    nq, nkv, d, T = 4, 2, 64, 5
    x = _qkv(T, nq, nkv, d, 1)
    rows = torch.tensor([4, -1, 0, 5, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32)
    keep = [1, 3, 4, 5]
    if eight:
        host = _caches(nkv, 20, d)
    else:
        host = (torch.full((nkv, 20, d), 5.0, dtype=torch.bfloat16),
                torch.full((nkv, 20, d), 6.0, dtype=torch.bfloat16))
    dev = [c.cuda() for c in host]
    call = tp.tp_kv8_append if eight else tp.tp_kv_append
    call(x.cuda(), *dev, 8, nq, nkv, d, 2, rows=rows.cuda())
    torch.cuda.synchronize()
    for a, b in zip(dev, host):
        for j in keep + list(range(-8, 0)) + list(range(7, 12)):
            assert torch.equal(a[:, 8 + j].cpu(), b[:, 8 + j])
        assert not torch.equal(a[:, 8].cpu(), b[:, 8])


def test_append8_of_values_that_are_not_finite_or_extreme():
    nq, nkv, d = 1, 1, 64
    x = torch.randn(6, 3 * d).to(torch.bfloat16)
    x[0, d] = float("nan")              # a NaN element: the rest as without it
    x[1, d + 5] = float("inf")          # an infinity: the row reads back as NaN
    x[2, d:2 * d] = 1e-38               # a scale far below 2^-126
    x[3, d:2 * d] = torch.tensor([3e38, -3e38]).repeat(32)
    x[4, d:2 * d] = float("nan")        # nothing but NaN
    x[5, d:2 * d] = -0.0
    dev = [c.cuda() for c in _caches(nkv, 6, d)]
    tp.tp_kv8_append(x.cuda(), *dev, 0, nq, nkv, d, 1)
    codes, scale = oracle.kv8_quantize(_new(x, nq, nkv, d, 0))
    assert torch.equal(dev[1].cpu(), torch.from_numpy(scale))
    got = dev[0].cpu().numpy()
    nan = (codes & 0x7f) == 0x7f
    assert (((got & 0x7f) == 0x7f) == nan).all() and (got[~nan] == codes[~nan]).all()
    k, _ = tp.tp_kv8_read(*dev, 0, 6, 1)
    assert torch.isnan(k[0, 1]).all() and torch.isnan(k[0, 0, 0]) and torch.isfinite(k[0, 0, 1:]).all()
    assert torch.isfinite(k[0, 2:4]).all() and (k[0, 5] == 0).all()
    # half a step of E4M3 (2^-4 of the value) and of bf16
    want = x[3, d:2 * d].double()
    assert ((k[0, 3].cpu().double() - want).abs() <= (2.0 ** -4 + 2.0 ** -8) * want.abs()).all()


def test_offsets_past_32_bits():
    # a cache of over 2^32 bytes per tensor: rows near its end
    nq, nkv, d, n = 2, 2, 256, 1 << 23
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    x = _qkv(3, nq, nkv, d, 5)
    k8 = torch.zeros(nkv, n, d, dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    ks, vs = (torch.zeros(nkv, n, device="cuda") for _ in range(2))
    past = n - 3
    tp.tp_kv8_append(x.cuda(), k8, ks, v8, vs, past, nq, nkv, d, 1)
    for which, (c, s) in enumerate(((k8, ks), (v8, vs))):
        codes, scale = oracle.kv8_quantize(_new(x, nq, nkv, d, which))
        assert torch.equal(c[:, past:].cpu(), torch.from_numpy(codes))
        assert torch.equal(s[:, past:].cpu(), torch.from_numpy(scale))
        assert not c[:, past - 1].any() and not c[0, :5].any()
    k = torch.zeros(nkv, n, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    tp.tp_kv8_read(k8, ks, v8, vs, past, 3, 2, k_out=k, v_out=v)
    codes, scale = oracle.kv8_quantize(_new(x, nq, nkv, d, 1))
    want = torch.from_numpy(oracle.E4M3_TABLE[codes]).float() * torch.from_numpy(scale)[..., None]
    assert torch.equal(v[:, past:].cpu(), want.to(torch.bfloat16))
    assert not v[:, past - 1].any()


def test_in_a_graph_and_on_another_stream():
    nq, nkv, d, T = 8, 2, 128, 9
    x = _qkv(T, nq, nkv, d, 2).cuda()
    a = [c.cuda() for c in _caches(nkv, 40, d)]
    b = [c.clone() for c in a]
    c = [t.clone() for t in a]
    tp.tp_kv8_append(x, *a, 20, nq, nkv, d, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tp.tp_kv8_append(x, *b, 20, nq, nkv, d, 1, stream=side)
    k, v = tp.tp_kv8_read(*b, 20, T, 1, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.tp_kv8_append(x, *c, 20, nq, nkv, d, 1)
        k2, v2 = tp.tp_kv8_read(*c, 20, T, 1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(a, b, c))
    assert torch.equal(k[:, 20:], k2[:, 20:]) and torch.equal(v[:, 20:], v2[:, 20:])
