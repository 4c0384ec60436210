"""GPU parity of tp_qk_norm_rope and its gradient against the fp64 oracle.

Bounds (element by element, not fitted): the result is rounded once to bf16,
2^-8 of its value at most (finfo(bf16).eps / 2).  Before that everything is
fp32: the mean of d <= 256 squares, a reciprocal root, three products and a
turn of two terms, each with relative errors of a few 2^-24, and sine and cosine
of an angle held to 2^-22: under 2^-17 of the magnitudes that are added.  A
gain's gradient is a sum in fp32 over tokens and heads in runs of a few hundred
terms: under 2^-13 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8


def _case(T, nq, nkv, d, rot, norm=True, far=0, past=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = nq + 2 * nkv
    size = torch.exp(0.5 * torch.randn(1, n, 1, generator=g))
    x = (torch.randn(T, n, d, generator=g) * size).to(torch.bfloat16).reshape(T, -1)
    dy = torch.randn(T, n * d, generator=g).to(torch.bfloat16)
    gq = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None
    gk = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) if norm else None
    fr = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))).float() \
        if rot else None
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32) if far else None
    at = pos.tolist() if far else list(range(past, past + T))
    return x, dy, gq, gk, fr, pos, at


def _gpu(t):
    return None if t is None else t.cuda()


def _close(got, ref, mag, rel, what):
    y = got.double().cpu().numpy()
    assert np.isfinite(y).all(), what
    err = np.abs(y - ref)
    bound = HALF_STEP * np.abs(ref) * (1 + 2.0 ** -6) + rel * mag + 1e-37
    assert (err <= bound).all(), f"{what}: {np.max(err / bound):.3f} of the bound"


SHAPES = [
    # T, nq, nkv, d, rot
    (1, 64, 8, 128, 128), (5, 64, 8, 128, 64), (3, 9, 3, 80, 32), (2, 4, 4, 16, 16),
    (7, 6, 2, 96, 96), (4, 3, 1, 256, 256), (300, 8, 2, 128, 128), (1, 1, 1, 64, 0),
    (2, 130, 2, 112, 16), (601, 2, 1, 48, 48), (3, 4000, 40, 16, 16), (2, 1998, 999, 256, 32),
]


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,nq,nkv,d,rot", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_forward(T, nq, nkv, d, rot, layout, norm):
    x, _, gq, gk, fr, pos, at = _case(T, nq, nkv, d, rot, norm, past=1000, seed=T + d)
    ref = oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, fr, at, layout)
    z = oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, None, at, layout)
    mag = np.abs(z).reshape(T, -1, d).max(-1, keepdims=True).repeat(d, -1).reshape(T, -1)
    args = dict(gamma_q=_gpu(gq), gamma_k=_gpu(gk), inv_freq=_gpu(fr), layout=layout)
    xg = x.cuda()
    y = tp.tp_qk_norm_rope(xg, 1000, nq, nkv, d, 1, **args)
    torch.cuda.synchronize()
    assert torch.equal(xg.cpu(), x)
    _close(y, ref, mag, 2.0 ** -17, (T, nq, nkv, d, rot, layout, norm))
    v = (nq + nkv) * d
    assert torch.equal(y[:, v:].cpu(), x[:, v:])
    # in place: the same bits
    tp.tp_qk_norm_rope(xg, 1000, nq, nkv, d, 1, out=xg, **args)
    assert torch.equal(xg, y)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_far_and_unordered_positions(layout):
    x, _, gq, gk, fr, pos, at = _case(65, 8, 2, 128, 128, far=1 << 30, seed=3)
    pos[:3] = torch.tensor([0, 2 ** 31 - 1, 1])
    at = pos.tolist()
    ref = oracle.qk_norm_rope(x, 8, 2, 128, gq, gk, fr, at, layout)
    z = oracle.qk_norm_rope(x, 8, 2, 128, gq, gk, None, at, layout)
    mag = np.abs(z).reshape(65, -1, 128).max(-1, keepdims=True).repeat(128, -1).reshape(65, -1)
    y = tp.tp_qk_norm_rope(x.cuda(), 0, 8, 2, 128, 2, _gpu(gq), _gpu(gk), _gpu(fr), _gpu(pos),
                           layout)
    _close(y, ref, mag, 2.0 ** -17, layout)


def test_a_row_of_zeros_and_extreme_rows():
    x, _, gq, gk, fr, _, at = _case(4, 4, 2, 128, 128, seed=4)
    x[0] = 0
    x[1] *= 1e-15   # squares near 1e-30: far below eps
    x[2, :128] = 3e18
    ref = oracle.qk_norm_rope(x, 4, 2, 128, gq, gk, fr, at)
    z = oracle.qk_norm_rope(x, 4, 2, 128, gq, gk, None, at)
    mag = np.abs(z).reshape(4, -1, 128).max(-1, keepdims=True).repeat(128, -1).reshape(4, -1)
    y = tp.tp_qk_norm_rope(x.cuda(), 0, 4, 2, 128, 1, _gpu(gq), _gpu(gk), _gpu(fr))
    _close(y, ref, mag, 2.0 ** -17, "zeros")
    assert (y[0] == 0).all()


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e19, 3e37])
def test_heads_whose_squares_leave_fp32(size):
    # without eps a head's scale cancels in the norm and divides its gradient
    x, dy, gq, gk, fr, _, at = _case(3, 4, 2, 64, 64, seed=14)
    x = (x.double() * size / x.double().abs().max()).to(torch.bfloat16)
    ref = oracle.qk_norm_rope(x, 4, 2, 64, gq, gk, fr, at, eps=0.0)
    y = tp.tp_qk_norm_rope(x.cuda(), 0, 4, 2, 64, 1, _gpu(gq), _gpu(gk), _gpu(fr), eps=0.0)
    z = oracle.qk_norm_rope(x, 4, 2, 64, gq, gk, None, at, eps=0.0)
    mag = np.abs(z).reshape(3, -1, 64).max(-1, keepdims=True).repeat(64, -1).reshape(3, -1)
    _close(y, ref, mag, 2.0 ** -17, size)
    dy = (dy.double() * min(size, 1.0)).to(torch.bfloat16)  # the gradient stays in range
    ref = oracle.qk_norm_rope_backward(x, dy, 4, 2, 64, gq, gk, fr, at, eps=0.0)
    got = tp.tp_qk_norm_rope_backward(x.cuda(), dy.cuda(), 0, 4, 2, 64, 1, _gpu(gq), _gpu(gk),
                                      _gpu(fr), eps=0.0)
    mag = ref["mag"].reshape(3, -1, 64).max(-1, keepdims=True).repeat(64, -1).reshape(3, -1)
    if size <= 1e19:  # above that the gradient itself leaves bf16's normal range
        _close(got["dqkv"], ref["dqkv"], mag, 2.0 ** -17, size)
    _close(got["dgamma_q"], ref["dgamma_q"], ref["mag_q"], 2.0 ** -13, size)


def test_a_nan_stays_in_its_head():
    x, _, gq, gk, fr, _, at = _case(2, 4, 2, 64, 64, seed=5)
    clean = tp.tp_qk_norm_rope(x.cuda(), 0, 4, 2, 64, 1, _gpu(gq), _gpu(gk), _gpu(fr))
    x[1, 70] = float("nan")  # head 1 of token 1
    y = tp.tp_qk_norm_rope(x.cuda(), 0, 4, 2, 64, 1, _gpu(gq), _gpu(gk), _gpu(fr))
    assert torch.isnan(y[1, 64:128]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1, 64:128] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("T,nq,nkv,d,rot", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_backward(T, nq, nkv, d, rot, layout, norm):
    x, dy, gq, gk, fr, _, at = _case(T, nq, nkv, d, rot, norm, past=77, seed=2 * T + d)
    ref = oracle.qk_norm_rope_backward(x, dy, nq, nkv, d, gq, gk, fr, at, layout)
    args = dict(gamma_q=_gpu(gq), gamma_k=_gpu(gk), inv_freq=_gpu(fr), layout=layout)
    dyg = dy.cuda()
    got = tp.tp_qk_norm_rope_backward(x.cuda(), dyg, 77, nq, nkv, d, 1, **args)
    torch.cuda.synchronize()
    what = (T, nq, nkv, d, rot, layout, norm)
    mag = ref["mag"].reshape(T, -1, d).max(-1, keepdims=True).repeat(d, -1).reshape(T, -1)
    _close(got["dqkv"], ref["dqkv"], mag, 2.0 ** -17, what)
    if norm:
        _close(got["dgamma_q"], ref["dgamma_q"], ref["mag_q"], 2.0 ** -13, what)
        _close(got["dgamma_k"], ref["dgamma_k"], ref["mag_k"], 2.0 ** -13, what)
    else:
        assert got["dgamma_q"] is None and got["dgamma_k"] is None
    # bit-identical again, and into dout itself
    again = tp.tp_qk_norm_rope_backward(x.cuda(), dyg, 77, nq, nkv, d, 1, dqkv=dyg, **args)
    for k in got:
        assert got[k] is None and again[k] is None or torch.equal(got[k], again[k]), k
    assert again["dqkv"] is dyg


def test_backward_against_differences():
    # <dx, u> against the central difference of the oracle's forward along u,
    # and the same for both gains: bf16 gradients of about 3000 elements, each
    # off by at most 2^-8 of itself
    T, nq, nkv, d, rot = 3, 5, 1, 96, 64
    x, dy, gq, gk, fr, _, at = _case(T, nq, nkv, d, rot, past=9, seed=8)
    got = tp.tp_qk_norm_rope_backward(x.cuda(), dy.cuda(), 9, nq, nkv, d, 1, _gpu(gq), _gpu(gk),
                                      _gpu(fr))
    rng = np.random.default_rng(0)
    xf, dyf = x.double().numpy(), dy.double().numpy()
    base = [xf, gq.double().numpy(), gk.double().numpy()]
    grads = [got["dqkv"], got["dgamma_q"], got["dgamma_k"]]
    for which in range(3):
        u = rng.standard_normal(base[which].shape)
        h = 1e-5

        def f(s):
            a = list(base)
            a[which] = a[which] + s * h * u
            return float((oracle.qk_norm_rope(a[0], nq, nkv, d, a[1], a[2], fr, at) * dyf).sum())

        diff = (f(1) - f(-1)) / (2 * h)
        g = grads[which].double().cpu().numpy()
        assert abs((g * u).sum() - diff) <= HALF_STEP * np.abs(g * u).sum() + 1e-5 * abs(diff)


def test_chained_with_the_projection_in_a_graph_and_on_another_stream():
    nq, nkv, d, T, H = 8, 2, 128, 6, 256
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((nq + 2 * nkv) * d, H, generator=g) * 0.05).to(torch.bfloat16).cuda()
    wo = (torch.randn(H, nq * d, generator=g) * 0.05).to(torch.bfloat16).cuda()
    ctx = torch.zeros(T, nq * d, dtype=torch.bfloat16, device="cuda")
    _, dy, gq, gk, fr, _, _ = _case(T, nq, nkv, d, 128, seed=2)
    args = (_gpu(gq), _gpu(gk), _gpu(fr))
    qkv, _ = tp.tp_attn_proj_forward(x, w, None, ctx, wo, None, nq, nkv, d, 2)
    y = tp.tp_qk_norm_rope(qkv, 40, nq, nkv, d, 2, *args)
    back = tp.tp_qk_norm_rope_backward(qkv, _gpu(dy), 40, nq, nkv, d, 2, *args)
    dyg = _gpu(dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = tp.tp_qk_norm_rope(qkv, 40, nq, nkv, d, 2, *args, stream=side)
    b2 = tp.tp_qk_norm_rope_backward(qkv, dyg, 40, nq, nkv, d, 2, *args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(back["dgamma_q"], b2["dgamma_q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q3, _ = tp.tp_attn_proj_forward(x, w, None, ctx, wo, None, nq, nkv, d, 2)
        tp.tp_qk_norm_rope(q3, 40, nq, nkv, d, 2, *args, out=q3)
        b3 = tp.tp_qk_norm_rope_backward(qkv, dyg, 40, nq, nkv, d, 2, *args)
    for _ in range(3):
        q3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q3, y)
        assert all(torch.equal(b3[k], back[k]) for k in back)
