"""The gradient norm's launches on the CPU (tests/clip_schedule_check.cu), and
norms over more tensors than one table holds on the GPU."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

import fp8_block_scaled_10_b200 as fp8bs

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.mark.skipif(not (os.path.exists(NVCC) or shutil.which("nvcc")), reason="nvcc not found")
def test_every_launch_has_its_ctas_and_its_slots(tmp_path):
    exe = tmp_path / "clip_schedule_check"
    cmd = [NVCC, "-std=c++17", "-O2", "-gencode", "arch=compute_100a,code=sm_100a",
           "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "fp8_block_scaled_10_b200", "csrc"),
           os.path.join(HERE, "clip_schedule_check.cu"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout + out.stderr


MARK = 0x5A


def _pieces(sizes, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.randn(sum(sizes), generator=g, device="cuda")
    return flat, list(flat.split(sizes))


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [
    [3 + i % 50 for i in range(1500)],
    [2_000_001 if i % 400 == 7 else 17 for i in range(1700)],   # a few large among many small
    [1 + i % 5 for i in range(130)] + [400_000] * 3,            # a later launch with more CTAs
    [400_000] * 3 + [0, 1, 0] * 2000,
    [33] * 45_000,
], ids=lambda s: "%dx%d" % (len(s), sum(s)))
def test_many_tensors(sizes):
    flat, grads = _pieces(sizes, len(sizes))
    ref = math.sqrt(float(flat.double().square().sum()))
    n = len(grads)
    L, p = fp8bs.lib(), fp8bs._ptr
    nws = int(L.fp8bs_grad_norm_workspace_size(n))
    ws = torch.full((nws + 4096,), MARK, dtype=torch.uint8, device="cuda")
    norm = torch.zeros((), device="cuda")
    ptrs = (ctypes.c_void_p * n)(*[g.data_ptr() if g.numel() else 0 for g in grads])
    numel = (ctypes.c_int64 * n)(*sizes)
    types = (ctypes.c_int * n)(*[fp8bs.DTYPE_F32] * n)
    for _ in range(2):   # the second call must not add to what the first one left
        fp8bs._check(L.fp8bs_grad_norm(ptrs, numel, types, n, p(norm), p(ws), nws, fp8bs._stream(flat.device)))
        # the sum is in 64 bits: one rounding of the norm to fp32, half a step
        assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    assert bool((ws[nws:] == MARK).all())
    assert torch.equal(fp8bs.grad_norm(grads), norm)
    keep = flat.double()
    out, before = fp8bs.clip_grads(grads, 0.5 * ref)
    assert torch.equal(before, norm)
    want = keep * (0.5 * ref / (ref + 1e-6))
    # factor and product rounded to fp32, the reference's norm to 2^-23
    assert ((flat.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()
    assert fp8bs.device_error() == 0


@pytest.mark.gpu
def test_captured_norm_of_many_tensors():
    flat, grads = _pieces([1 + i % 90 for i in range(1300)], 3)
    fp8bs.grad_norm(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fp8bs.grad_norm(grads)
    for scale in (1.0, 3.0, 0.5):
        flat.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, fp8bs.grad_norm(grads))
