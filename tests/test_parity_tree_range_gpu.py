"""tp_attn_tree and tp_attn_decode_kv8 over the range of scores and values that
the interface names, against the fp64 oracle.

Bounds are those of tests/test_parity_tree_gpu.py, |error| <= 2^-8 |ref| +
(2^-8 + 2^-9) A with A = sum_j p_j |v_j|.
"""
import pytest
import torch

from test_parity_tree_gpu import D, EIGHT, Case

pytestmark = pytest.mark.gpu

# 8 query heads over 2: 8, 32 and 64 rows a head (the narrow kernels), 80 (split), 200 (shared)
WIDTHS = pytest.mark.parametrize("T", [2, 8, 16, 20, 50])


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
