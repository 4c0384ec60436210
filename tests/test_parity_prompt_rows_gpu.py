"""The forms that long prompts take: norms and rotation where a block reuses its
ring's slots (from its fifth token on, and their barriers' second phase), and
cache rows where a lane group takes four.  Bounds as in
tests/test_parity_qk_norm_gpu.py; cache rows are exact."""
import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp
from test_parity_kv_cache_gpu import _caches, _new, _qkv
from test_parity_qk_norm_gpu import _case, _close, _gpu

pytestmark = pytest.mark.gpu

# 296 blocks at most walk the tokens: 14 each, 5 each, and 9 each with two segments a token
LONG = [(4000, 2, 1, 48, 48), (1400, 8, 2, 128, 64), (1330, 130, 2, 112, 16), (2700, 3, 1, 16, 0)]


def _head_max(z, T, d):
    return np.abs(z).reshape(T, -1, d).max(-1, keepdims=True).repeat(d, -1).reshape(T, -1)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,nq,nkv,d,rot", LONG)
@pytest.mark.parametrize("norm", [True, False])
def test_forward(T, nq, nkv, d, rot, layout, norm):
    x, _, gq, gk, fr, pos, at = _case(T, nq, nkv, d, rot, norm, far=1 << 20, seed=T)
    ref = oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, fr, at, layout)
    z = oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, None, at, layout)
    args = dict(gamma_q=_gpu(gq), gamma_k=_gpu(gk), inv_freq=_gpu(fr), positions=_gpu(pos),
                layout=layout)
    xg = x.cuda()
    y = tp.tp_qk_norm_rope(xg, 0, nq, nkv, d, 1, **args)
    torch.cuda.synchronize()
    assert torch.equal(xg.cpu(), x)
    _close(y, ref, _head_max(z, T, d), 2.0 ** -17, (T, layout, norm))
    assert torch.equal(y[:, (nq + nkv) * d:].cpu(), x[:, (nq + nkv) * d:])
    tp.tp_qk_norm_rope(xg, 0, nq, nkv, d, 1, out=xg, **args)
    assert torch.equal(xg, y)
    assert tp.tp_device_error_check() == tp.TP_OK


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,nq,nkv,d,rot", LONG)
@pytest.mark.parametrize("norm", [True, False])
def test_backward(T, nq, nkv, d, rot, layout, norm):
    x, dy, gq, gk, fr, pos, at = _case(T, nq, nkv, d, rot, norm, far=1 << 20, seed=T + 1)
    ref = oracle.qk_norm_rope_backward(x, dy, nq, nkv, d, gq, gk, fr, at, layout)
    args = dict(gamma_q=_gpu(gq), gamma_k=_gpu(gk), inv_freq=_gpu(fr), positions=_gpu(pos),
                layout=layout)
    dyg = dy.cuda()
    got = tp.tp_qk_norm_rope_backward(x.cuda(), dyg, 0, nq, nkv, d, 1, **args)
    _close(got["dqkv"], ref["dqkv"], _head_max(ref["mag"], T, d), 2.0 ** -17, (T, layout, norm))
    if norm:
        _close(got["dgamma_q"], ref["dgamma_q"], ref["mag_q"], 2.0 ** -13, (T, layout))
        _close(got["dgamma_k"], ref["dgamma_k"], ref["mag_k"], 2.0 ** -13, (T, layout))
    again = tp.tp_qk_norm_rope_backward(x.cuda(), dyg, 0, nq, nkv, d, 1, dqkv=dyg, **args)
    for k in got:
        assert got[k] is None and again[k] is None or torch.equal(got[k], again[k]), k
    assert tp.tp_device_error_check() == tp.TP_OK


# more than 16 x 148 x (256 / lanes of a row) rows, by a bit that ends inside a block
FOUR = [(16, 19000, 8), (32, 9500, 8), (64, 4800, 8), (48, 4800, 8), (80, 4800, 4), (128, 1300, 16),
        (256, 2000, 5)]


@pytest.mark.parametrize("d,n,nkv", FOUR)
@pytest.mark.parametrize("pick", [False, True])
@pytest.mark.parametrize("eight", [False, True])
def test_many_cache_rows(d, n, nkv, pick, eight):
    nq, past = nkv, 3
    lanes = 1 << (d // 8 - 1).bit_length()
    assert n * 2 * nkv > 16 * 148 * (256 // lanes)
    T = n // 2 + 1 if pick else n
    x = _qkv(T, nq, nkv, d, d)
    rows = None
    if pick:
        rows = torch.randint(0, T, (n,), generator=torch.Generator().manual_seed(d)).int()
    if eight:
        host = _caches(nkv, past + n + 2, d)
    else:
        host = (torch.full((nkv, past + n + 2, d), 5.0, dtype=torch.bfloat16),
                torch.full((nkv, past + n + 2, d), 6.0, dtype=torch.bfloat16))
    dev = [c.cuda() for c in host]
    call = tp.tp_kv8_append if eight else tp.tp_kv_append
    call(x.cuda(), *dev, past, nq, nkv, d, 1, rows=None if rows is None else rows.cuda())
    torch.cuda.synchronize()
    for which in (0, 1):
        src = _new(x, nq, nkv, d, which)
        if pick:
            src = src[:, rows.long()]
        parts = [torch.from_numpy(a) for a in oracle.kv8_quantize(src)] if eight else [src]
        for i, part in enumerate(parts):
            at = len(parts) * which + i
            want = host[at].clone()
            want[:, past:past + n] = part
            assert torch.equal(dev[at].cpu(), want)
