"""In a process of its own: after a call of another kind, the norm, rotation and
attention kernels are first used, and with that loaded, inside a graph capture, and
give what they give eagerly."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
import tensor_transformer_linear_column_b200 as tp
x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
w = torch.ones(512, 256, dtype=torch.bfloat16, device="cuda")
assert (tp.tp_colpar_gemm_gelu(x, w, None, 1) == 256).all()
g = torch.Generator().manual_seed(0)
nq, nkv, d, past = 16, 2, 128, 300
fr = (10000.0 ** (-torch.arange(64) / 64.0)).float().cuda()
ops = []
for T in (1, 3, 7, 12, 40, 100):  # each width of the attention kernels, and the merge of many rows
    qkv = torch.randn(T, (nq + 2 * nkv) * d, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(nkv, past + T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k8, v8 = (torch.randint(0, 120, (nkv, past + T, d), generator=g).to(torch.uint8).cuda() for _ in range(2))
    ks, vs = (torch.rand(nkv, past + T, generator=g).cuda() for _ in range(2))
    ops.append(lambda a=(qkv, k, v): tp.tp_attn_tree(*a, past, nq, nkv, d, 1))
    ops.append(lambda a=(qkv, k8, ks, v8, vs): tp.tp_attn_decode_kv8(*a, past, nq, nkv, d, 1))
    ops.append(lambda q=qkv: tp.tp_qk_norm_rope(q, past, nq, nkv, d, 1, inv_freq=fr))
    ops.append(lambda q=qkv: tp.tp_qk_norm_rope_backward(q, q, past, nq, nkv, d, 1, inv_freq=fr)["dqkv"])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = [op() for op in ops]
graph.replay()
torch.cuda.synchronize()
want = [op() for op in ops]
torch.cuda.synchronize()
assert tp.tp_device_error_check() == tp.TP_OK
assert all(torch.isfinite(a).all() and torch.equal(a, b) for a, b in zip(outs, want))
print("same")
"""


def test_first_use_in_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", SCRIPT], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and res.stdout.strip() == "same", res.stdout + res.stderr
