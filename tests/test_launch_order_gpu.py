"""Calls that follow each other without a wait in between, where the first writes
what the second takes as a parameter: a kernel that starts before its predecessor
ends must read it only afterwards, and not through the path for data that stays as
it is for a kernel's whole life."""
import pytest
import torch

import tensor_transformer_linear_column_b200 as tp

pytestmark = pytest.mark.gpu

OPTIONS = [0, tp.TP_OPT_PDL, tp.TP_OPT_PDL | tp.TP_OPT_STATIC_WEIGHTS]


@pytest.fixture(params=OPTIONS)
def options(request):
    prev = tp.tp_get_launch_options()
    tp.tp_set_launch_options(request.param)
    yield request.param
    tp.tp_set_launch_options(prev)


@pytest.mark.parametrize("backward", [False, True])
def test_frequencies_that_the_kernel_before_writes(options, backward):
    # tp_kv8_append writes fp32 scales; read as frequencies they change from call to call
    nq, nkv, d, T = 8, 2, 128, 600
    half = d // 2
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, (nq + 2 * nkv) * d, generator=g).to(torch.bfloat16).cuda()
    rows = [(2.0 ** (i % 5) * torch.rand(half, 3 * 16, generator=g)).to(torch.bfloat16).cuda()
            for i in range(12)]
    k, v = (torch.zeros(1, half, 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    freq, other = (torch.zeros(1, half, device="cuda") for _ in range(2))

    def step(r):
        tp.tp_kv8_append(r, k, freq, v, other, 0, 1, 1, 16, 1)
        if backward:
            return tp.tp_qk_norm_rope_backward(x, x, 7, nq, nkv, d, 1, inv_freq=freq[0])["dqkv"]
        return tp.tp_qk_norm_rope(x, 7, nq, nkv, d, 1, inv_freq=freq[0])

    want = []
    for r in rows:
        want.append(step(r))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    for _ in range(5):
        got = [step(r) for r in rows]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [64, 128])
def test_queries_that_the_kernel_before_writes(options, T):
    # norms and rotation in place, then the attention that has many rows and no mask
    nq, nkv, d, past = 16, 2, 128, 130
    g = torch.Generator().manual_seed(T)
    xs = [torch.randn(T, (nq + 2 * nkv) * d, generator=g).to(torch.bfloat16).cuda()
          for _ in range(6)]
    fr = (10000.0 ** (-torch.arange(64) / 64.0)).float().cuda()
    k0, v0 = (torch.randn(nkv, past + T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    buf = torch.empty_like(xs[0])

    def run(wait):
        out, k, v = [], k0.clone(), v0.clone()
        torch.cuda.synchronize()
        for x in xs:
            tp.tp_qk_norm_rope(x, past, nq, nkv, d, 1, inv_freq=fr, out=buf)
            if wait:
                torch.cuda.synchronize()
            out.append(tp.tp_attn_tree(buf, k, v, past, nq, nkv, d, 1))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out

    want = run(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
