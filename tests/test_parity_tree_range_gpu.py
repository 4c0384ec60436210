"""tp_attn_tree and tp_attn_decode_kv8 over the range of scores and values that
the interface names, against the fp64 oracle.

Bounds are those of tests/test_parity_tree_gpu.py, |error| <= 2^-8 |ref| +
(2^-8 + 2^-9) A with A = sum_j p_j |v_j|, and hold for a row where its scores
leave no doubt about its weights.  With B = sum |q k| / sqrt(d) of a key, its score
is off by at most 2^-17 B (fp32 sums), over an 8-bit cache by 2^-17 sum_i
max|q| |k_i| / sqrt(d) more (the queries' two E4M3 terms).  With e the largest of
that over the keys that a row sees, a row is
  sharp    if e <= 2^-10: its weights are off by under 2^-9 of themselves
  decided  if the best key leads the second by more than 2 e + 100: it takes
           all the weight but e^-100, whatever the errors
and else not looked at, but for being finite.
"""
import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_linear_column_b200 as tp
from test_parity_tree_gpu import D, EIGHT, Case

pytestmark = pytest.mark.gpu

# 8 query heads over 2: 8, 32 and 64 rows a head (the narrow kernels), 80 (split), 200 (shared)
WIDTHS = pytest.mark.parametrize("T", [2, 8, 16, 20, 50])


def _full(c):
    """Keys and values [nkv, past + T, d] in fp64, as the case's call sees them."""
    T, past, nq, nkv = c.T, c.past, c.nq, c.nkv
    new = c.qkv.reshape(T, -1, D)
    out = []
    for w in (0, 1):
        x = new[:, nq + w * nkv:nq + (w + 1) * nkv].transpose(0, 1)
        if c.eight:
            old = oracle.kv8_values(c.cache[2 * w][:, :past].numpy(),
                                    c.cache[2 * w + 1][:, :past].numpy())
            x = oracle.kv8_values(*oracle.kv8_quantize(x))
        else:
            old, x = c.cache[w][:, :past].double().numpy(), x.double().numpy()
        out.append(np.concatenate([old, x], 1))
    return out


def _look_at(c):
    """[T, nq] truth values: rows that are sharp, and rows that are decided."""
    k, _ = _full(c)
    T, past, nq, nkv = c.T, c.past, c.nq, c.nkv
    q = c.qkv[:, :nq * D].double().numpy().reshape(T, nq, D)
    seen = np.concatenate([np.ones((T, past), bool), oracle.tree_visible(T, c.words)], 1)
    sharp, decided = np.zeros((T, nq), bool), np.zeros((T, nq), bool)
    for h in range(nq):
        kg = k[h // (nq // nkv)]
        s = q[:, h] @ kg.T / np.sqrt(D)
        e = 2.0 ** -17 * (np.abs(q[:, h]) @ np.abs(kg).T) / np.sqrt(D)
        if c.eight:
            e += 2.0 ** -17 * np.abs(q[:, h]).max(1, keepdims=True) * np.abs(kg).sum(1) / np.sqrt(D)
        worst = np.where(seen, e, 0).max(1)
        top = np.sort(np.where(seen, s, -np.inf), 1)
        sharp[:, h] = worst <= 2.0 ** -10
        decided[:, h] = top[:, -1] - top[:, -2] > 2 * worst + 100
    return sharp, decided


def _check(c, least=0.9, room=0.0):
    """The rows that can be looked at, `least` of them all, and that all are finite."""
    ctx, dev = c.run()
    torch.cuda.synchronize()
    assert tp.tp_device_error_check() == tp.TP_OK
    sharp, decided = _look_at(c)
    look = sharp | decided
    assert look.mean() >= least, look.mean()
    ref, mag = c.reference()
    y = ctx.double().cpu().numpy()
    assert np.isfinite(y).all()
    err = np.abs(y - ref).reshape(c.T, c.nq, D)
    bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * mag).reshape(c.T, c.nq, D) + room
    worst = np.where(look[..., None], err / np.maximum(bound, 1e-300), 0)
    assert (worst <= 1).all(), (worst.max(), (worst.max(-1) > 1).mean())
    c.check_cache(dev)


def _scaled(c, size, keys=None):
    """Queries times `size`, keys times `size` or a factor for each."""
    x = c.qkv.reshape(c.T, -1, D).float()
    x[:, :c.nq] *= size
    x[:, c.nq:c.nq + c.nkv] *= size if keys is None else keys[-1]
    c.qkv = x.to(torch.bfloat16).reshape(c.T, -1)
    g = torch.Generator().manual_seed(c.T + 1)
    n = c.past + c.T + 3
    k = torch.randn(c.nkv, n, D, generator=g) * (size if keys is None else keys[None, :n, None])
    v = torch.randn(c.nkv, n, D, generator=g) * torch.exp(torch.randn(c.nkv, n, 1, generator=g))
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    return c


@EIGHT
@WIDTHS
@pytest.mark.parametrize("log2", [10, 12, 15, 18, 23, 30, 44])
def test_large_scores(eight, T, log2):
    # q . k of 2^(2 log2) and a few bits more, in no way powers of two
    _check(_scaled(Case(eight, T, 900, 8, 2, "tree", seed=log2), 2.0 ** log2))


@EIGHT
@WIDTHS
@pytest.mark.parametrize("log2", [11, 18, 40])
def test_large_scores_below_zero(eight, T, log2):
    # the best key is the least negative one
    c = _scaled(Case(eight, T, 700, 8, 2, "tree", seed=log2), 2.0 ** log2)
    x = c.qkv.reshape(T, -1, D).float()
    x[:, :8] = x[:, :8].abs()
    x[:, 8:10] = -x[:, 8:10].abs()
    c.qkv = x.to(torch.bfloat16).reshape(T, -1)
    for m in c.cache[:1]:
        if eight:
            m |= 0x80
        else:
            m[:, :c.past] = -m[:, :c.past].abs()
    _check(c)


@EIGHT
@WIDTHS
@pytest.mark.parametrize("log2", [18, 32])
def test_rows_of_ordinary_and_of_large_scores_side_by_side(eight, T, log2):
    # every third head of every second token is large: both kinds in each warp
    c = Case(eight, T, 1100, 8, 2, "any", seed=log2)
    x = c.qkv.reshape(T, -1, D).float()
    x[::2, 0:8:3] *= 2.0 ** log2
    c.qkv = x.to(torch.bfloat16).reshape(T, -1)
    _check(c)


@EIGHT
@WIDTHS
@pytest.mark.parametrize("last", [26, 60])
def test_scores_that_grow_into_the_large_along_the_cache(eight, T, last):
    n = 1500 + T + 3
    _check(_scaled(Case(eight, T, 1500, 8, 2, "causal", seed=last), 1.0,
                   2.0 ** torch.linspace(-4, last, n).round()))


@pytest.mark.parametrize("T", [20, 50])
@pytest.mark.parametrize("log2", [0, 15, 18, 40])
def test_value_scales_far_apart_under_large_scores(T, log2):
    # 8 bits, more than 64 rows: the product of weight and value scale is what is
    # held to 2^-11 of itself, whatever the other keys' scales are.  (Of ordinary
    # scores, the keys of weight 2^-27 and less are worth no more than the rest: no
    # bound is promised relative to them, and none is needed.)
    c = _scaled(Case(True, T, 800, 8, 2, "causal", seed=log2), 2.0 ** log2)
    g = torch.Generator().manual_seed(3)
    far = 2.0 ** torch.randint(-35, 36, (2, 803 + T, 1), generator=g)
    if log2 == 0:
        far = 2.0 ** torch.randint(-3, 4, (2, 803 + T, 1), generator=g)
    v = (1 + torch.rand(2, 803 + T, D, generator=g)) * far
    c.cache[2], c.cache[3] = (torch.from_numpy(a) for a in oracle.kv8_quantize(v.to(torch.bfloat16)))
    c.cache[2][:, 800:], c.cache[3][:, 800:] = 0x7f, float("nan")
    _check(c)


@EIGHT
@WIDTHS
@pytest.mark.parametrize("size", [1e-20, 1e-22, 1e-24, 1e20, 1e24])
def test_values_that_are_all_small_or_all_large(eight, T, size):
    # of one head; the other's are ordinary.  2^-80 is 8.3e-25, 2^80 1.2e24
    c = Case(eight, T, 700, 8, 2, "tree", seed=6)
    g = torch.Generator().manual_seed(7)
    k = torch.randn(2, 703 + T, D, generator=g)
    v = 1 + 0.1 * torch.randn(2, 703 + T, D, generator=g)
    v[0] *= size * 0.8
    x = c.qkv.reshape(T, -1, D).float()
    x[:, 10] *= size * 0.25
    c.qkv = x.to(torch.bfloat16).reshape(T, -1)
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    c.check((T, size))


@pytest.mark.parametrize("first", [7.0, 7.37, 7.71])
@pytest.mark.parametrize("high", [450.0, 894.0])
def test_many_small_weights_under_one_large_in_8_bits(high, first):
    # Up to 64 rows over 8 bits: a weight times its value scale is held to 2^-9 + 2^-11
    # of itself (three terms of three bits, of an fp16 number) plus 2^-22 of C for a
    # largest weight of 1 (where the terms end), C the power of two at or above the
    # chunk's largest scale -- here just below and twice that scale.  127 keys of one
    # weight: their errors have one sign and add up.
    nq, past = 16, 128
    c = Case(True, 1, past, nq, 1, "any", seed=1)
    c.words = torch.zeros(1, 1, dtype=torch.int64)  # the cached keys alone
    q = torch.zeros(nq + 2, D)
    log2 = first + 0.83 * torch.arange(nq)          # the weights: 2^-7 .. 2^-20
    q[:nq, 0] = log2 * np.sqrt(D) / np.log2(np.e)
    c.qkv = q.to(torch.bfloat16).reshape(1, -1)
    k = torch.zeros(1, past + 4, D)
    k[:, :past - 1, 0] = -1.0
    v = torch.full((1, past + 4, D), high)
    v[:, past - 1, 1:] = 0                           # the large one is seen in element 0 alone
    c.set_cache(k.to(torch.bfloat16), v.to(torch.bfloat16))
    _, scale = c.cache[2:]
    top = float(scale[:, :past].max())
    power = 2.0 ** np.ceil(np.log2(top))
    ref, _ = c.reference()
    y = c.run()[0].double().cpu().numpy().reshape(nq, D)[:, 1:]
    ref = ref.reshape(nq, D)[:, 1:]
    total = ref[:, :1] / high                        # the small weights over the sum of all
    small = total / (past - 1) / (1 - total)         # one of them, the large one being 1
    each = ((2.0 ** -9 + 2.0 ** -11) * small * top + 2.0 ** -22 * power) * 448
    # and 2^-17 of the weights for their scores and exponentials, 2^-8 for the result
    bound = 2.0 ** -8 * ref + (1 - total) * (past - 1) * each + 2.0 ** -17 * ref
    assert (np.abs(y - ref) <= bound * (1 + 2.0 ** -7)).all(), np.max(np.abs(y - ref) / bound)
