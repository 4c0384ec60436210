"""Pins of oracle/tp_serving.py (CPU): pure-Python brute force, central
differences, and the older oracles where they overlap."""
import math

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp


def _x(T, n, d, seed):
    return np.random.default_rng(seed).standard_normal((T, n * d))


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_norm_and_rotation_by_brute_force(layout):
    T, nq, nkv, d, rot = 3, 2, 1, 8, 4
    x = _x(T, 4, d, 0)
    gq, gk = np.linspace(0.5, 2, d), np.linspace(-1, 1, d)
    fr = np.array([1.0, 0.25], dtype=np.float32)
    pos = [0, 7, 100000]
    got = oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, fr, pos, layout, 1e-5)
    for i in range(T):
        for h in range(4):
            v = [float(a) for a in x[i, h * d:(h + 1) * d]]
            if h < nq + nkv:
                r = 1 / math.sqrt(math.fsum(a * a for a in v) / d + 1e-5)
                g = gq if h < nq else gk
                v = [a * r * float(b) for a, b in zip(v, g)]
                for p in range(rot // 2):
                    a, b = (p, p + rot // 2) if layout == "half" else (2 * p, 2 * p + 1)
                    th = pos[i] * float(fr[p])
                    v[a], v[b] = (v[a] * math.cos(th) - v[b] * math.sin(th),
                                  v[a] * math.sin(th) + v[b] * math.cos(th))
            assert np.allclose(got[i, h * d:(h + 1) * d], v, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("norm", [True, False])
def test_gradient_against_central_differences(layout, norm):
    T, nq, nkv, d, rot = 2, 3, 1, 16, 16
    x, dy = _x(T, 5, d, 1), _x(T, 5, d, 2)
    rng = np.random.default_rng(3)
    gq, gk = (rng.standard_normal(d), rng.standard_normal(d)) if norm else (None, None)
    fr, pos = (0.5 ** np.arange(8)).astype(np.float32), [3, 900]
    g = oracle.qk_norm_rope_backward(x, dy, nq, nkv, d, gq, gk, fr, pos, layout)

    def f(x, gq, gk):
        return float((oracle.qk_norm_rope(x, nq, nkv, d, gq, gk, fr, pos, layout) * dy).sum())

    h = 1e-6
    for e in [(0, 0), (0, 17), (1, 40), (1, 63), (1, 79)]:
        a, b = x.copy(), x.copy()
        a[e] += h
        b[e] -= h
        assert abs((f(a, gq, gk) - f(b, gq, gk)) / (2 * h) - g["dqkv"][e]) < 1e-6
    if norm:
        for j in (0, 5, 15):
            u = np.zeros(d)
            u[j] = h
            assert abs((f(x, gq + u, gk) - f(x, gq - u, gk)) / (2 * h) - g["dgamma_q"][j]) < 1e-6
            assert abs((f(x, gq, gk + u) - f(x, gq, gk - u)) / (2 * h) - g["dgamma_k"][j]) < 1e-6


def test_the_norm_is_the_rms_norm_of_the_older_oracle():
    x = _x(4, 3, 64, 4)
    gamma = np.random.default_rng(5).standard_normal(64)
    got = oracle.qk_norm_rope(x, 1, 1, 64, gamma, gamma, None, [0] * 4, eps=oracle.RMS_EPS)
    for h in (0, 1):
        want = oracle.rms_norm(x[:, h * 64:(h + 1) * 64], gamma, oracle.RMS_EPS)
        assert np.allclose(got[:, h * 64:(h + 1) * 64], want, rtol=1e-12)
    assert np.array_equal(got[:, 128:], x[:, 128:])


def test_codes_are_torchs_and_rows_keep_their_largest():
    g = torch.Generator().manual_seed(0)
    y = torch.randn(20000, generator=g) * torch.exp(4 * torch.randn(20000, generator=g))
    y[:4] = torch.tensor([0.0, -0.0, 448.0, 1e30])
    want = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_codes(y.numpy()), want)
    x = torch.randn(7, 64, generator=g).to(torch.bfloat16)
    x[2] = 0
    codes, scale = oracle.kv8_quantize(x)
    assert scale.dtype == np.float32 and scale[2] == 0 and not codes[2].any()
    val = oracle.kv8_values(codes, scale)
    xf = x.double().numpy()
    at = np.abs(xf).argmax(-1)
    rows = np.arange(7)
    assert np.allclose(val[rows, at], xf[rows, at], rtol=2e-7)
    # half a step of E4M3, or of its subnormals at the row's scale
    assert (np.abs(val - xf) <= np.abs(xf) * 2.0 ** -4 + 2.0 ** -10 * scale[:, None] * 1.001).all()


def test_masked_attention_is_the_causal_core_without_a_mask():
    nq, nkv, d, past, T = 4, 2, 16, 5, 3
    rng = np.random.default_rng(6)
    qkv = rng.standard_normal((T, (nq + 2 * nkv) * d))
    ck, cv = rng.standard_normal((2, nkv, past, d))
    want, grown = oracle.attn_core(qkv, nq, nkv, d, 1, [(ck, cv)])
    ctx, mag = oracle.attn_masked(qkv[:, :nq * d], grown[0][0], grown[0][1],
                                  oracle.tree_visible(T, None), nq, nkv, d)
    assert np.allclose(ctx, want, rtol=1e-12, atol=1e-14) and (mag >= np.abs(ctx) - 1e-12).all()


def test_masked_attention_of_a_tree_is_each_path_on_its_own():
    nq, nkv, d, past = 2, 1, 8, 4
    parents = [-1, 0, 0, 2, 1]
    T = len(parents)
    words = tp.tp_tree_mask(parents)
    rng = np.random.default_rng(7)
    qkv = rng.standard_normal((T, (nq + 2 * nkv) * d))
    k = rng.standard_normal((nkv, past + T, d))
    v = rng.standard_normal((nkv, past + T, d))
    k[:, past:] = qkv[:, nq * d:(nq + 1) * d]
    v[:, past:] = qkv[:, (nq + 1) * d:]
    ctx, _ = oracle.attn_masked(qkv[:, :nq * d], k, v, oracle.tree_visible(T, words.numpy()), nq,
                                nkv, d)
    for i in range(T):
        path, at = [], i
        while at >= 0:
            path.insert(0, at)
            at = parents[at]
        line, _ = oracle.attn_core(qkv[path], nq, nkv, d, 1, [(k[:, :past], v[:, :past])])
        assert np.allclose(ctx[i], line[-1], rtol=1e-12, atol=1e-14)


def test_a_row_that_sees_nothing_is_zero():
    q = np.ones((2, 8))
    ctx, mag = oracle.attn_masked(q, np.ones((1, 2, 8)), np.ones((1, 2, 8)),
                                  np.array([[False, False], [True, False]]), 1, 1, 8)
    assert not ctx[0].any() and not mag[0].any() and (ctx[1] == 1).all()


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128])
def test_tree_words(T):
    rng = np.random.default_rng(T)
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, T)]
    words = tp.tp_tree_mask(parents)
    assert words.dtype == torch.int64 and tuple(words.shape) == (T, (T + 63) // 64)
    seen = oracle.tree_visible(T, words.numpy())
    for i in range(T):
        anc, at = set(), i
        while at >= 0:
            anc.add(at)
            at = parents[at]
        assert set(np.flatnonzero(seen[i])) == anc


@pytest.mark.parametrize("parents", [[], [0], [-1, 1], [-1, -2], [-1, 5], [-1] * 129])
def test_tree_words_refuse_what_is_no_tree(parents):
    with pytest.raises(tp.TPError) as e:
        tp.tp_tree_mask(parents)
    assert e.value.status == tp.TP_ERR_SHAPE
