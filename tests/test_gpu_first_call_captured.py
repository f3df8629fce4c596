"""The first call of a process may be a captured one: what a call asks the runtime
(shared-memory limits, cluster sizes) is asked while a graph is recorded."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
import fp8_block_scaled_10_b200 as fp8bs
g = torch.Generator(device="cuda").manual_seed(1)
codes = [torch.randint(0, 256, (192, 256), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
scales = [torch.rand(192, 4, generator=g, device="cuda") * 0.01 for _ in range(2)]
grads = [torch.randn(1000, generator=g, device="cuda") for _ in range(3)]
outs = [torch.empty_like(v) for v in grads]
xs = [torch.randn(m, 512, generator=g, device="cuda").bfloat16() for m in (1, 16, 32)]
def run():
    r = [fp8bs.int4_linear(x, codes[0], scales[0]) for x in xs]
    r += [fp8bs.int4_linear_gated(x, codes[0], scales[0], codes[1], scales[1]) for x in xs]
    q, s = fp8bs.weight_quant(torch.ones(128, 512, device="cuda"))
    r.append(fp8bs.fp8_gated_ffn(xs[0], q, s, q, s, q[:, :128].contiguous(), s[:, :1].contiguous()))
    return r + fp8bs.clip_grads(grads, 1.0, out=outs)[0]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, run())), "the replay and a plain call differ"
assert fp8bs.device_error() == 0
print("ok")
"""


def test_first_calls_in_a_capture():
    out = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert out.returncode == 0 and out.stdout.strip().endswith("ok"), out.stdout + out.stderr[-2000:]
