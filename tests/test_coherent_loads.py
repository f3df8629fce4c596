"""Kernels here start while their producer may still write (programmatic
dependent launch), so nothing that another kernel writes may be read through the
non-coherent path.  The sources are checked on the CPU; on the GPU, producer and
consumer run back to back over the same buffers with alternating data."""
import glob
import os
import re

import pytest
import torch

import fp8_block_scaled_10_b200 as fp8bs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_block_scaled_10_b200", "csrc")


def _code(path):
    """The file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_kernel_asks_for_the_non_coherent_path(path):
    assert not re.findall(r"__ldg\s*\(|ld\.global\.nc", _code(path))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(g, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * 60).to(torch.float8_e4m3fn)


def _weight(g, N, K):
    s = (torch.rand(-(-N // 128), K // 128, generator=g, device="cuda") + 0.5) * 0.04 / K ** 0.5
    return _codes(g, N, K), s


def _bits(t):
    return t.view(torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(77, 576, 7168), (1, 2048, 7168), (8, 512, 4096)])
def test_split_partials_of_alternating_calls_in_one_workspace(M, N, K):
    g = _gen(M)
    w = (*_weight(g, N, K), *_weight(g, N, K))
    acts = [(_codes(g, M, K), torch.rand(M, K // 128, generator=g, device="cuda") * 0.01 + 0.005)
            for _ in range(2)]
    nws = int(fp8bs.lib().fp8bs_gemm_gated_workspace_size(M, N, K))
    assert nws > 0, "the shape is meant to split K"
    ws = torch.empty(nws, dtype=torch.uint8, device="cuda")
    want = [fp8bs.fp8_gemm_gated(*a, *w) for a in acts]
    torch.cuda.synchronize()
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(100)]
    p = fp8bs._ptr
    for i, h in enumerate(outs):
        fp8bs._check(fp8bs.lib().fp8bs_fp8_gemm_gated(*[p(t) for t in (*acts[i % 2], *w)], M, N, K, p(h), None,
                                                      p(ws), nws, fp8bs._stream(h.device)))
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(h), _bits(want[i % 2])) for i, h in enumerate(outs))
    # the dense GEMM's split of the same depth, its partials in one workspace
    nws = fp8bs.gemm_workspace_size(M, N, K)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device="cuda")
    want = [fp8bs.fp8_gemm(*a, *w[:2]) for a in acts]
    torch.cuda.synchronize()
    for i, h in enumerate(outs):
        fp8bs._check(fp8bs.lib().fp8bs_fp8_gemm(*[p(t) for t in (*acts[i % 2], *w[:2])], M, N, K, p(h), p(ws), nws,
                                                fp8bs._stream(h.device)))
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(h), _bits(want[i % 2])) for i, h in enumerate(outs))
    assert fp8bs.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 12, 32])
def test_chains_over_the_same_buffers(M):
    """act_quant -> GEMM -> 4-bit gate -> 4-bit linear, every intermediate in one
    buffer that the next pass overwrites."""
    g = _gen(50 + M)
    K, N, F = 1024, 1024, 512
    w, ws_ = _weight(g, N, K)
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(2)]
    dense = [torch.randn(n, k, generator=g, device="cuda") * 0.05 for n, k in ((F, N), (F, N), (K, F))]
    gate, up, down = [fp8bs.weight_quant_int4(d, 64) for d in dense]
    want = []
    for x in xs:
        y = fp8bs.fp8_linear(x, w, ws_)
        want.append(fp8bs.int4_linear(fp8bs.int4_linear_gated(y, *gate, *up), *down))
        torch.cuda.synchronize()
    L, p = fp8bs.lib(), fp8bs._ptr
    st = fp8bs._stream(xs[0].device)
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, K // 128, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    nws = fp8bs.gemm_workspace_size(M, N, K)
    ws = torch.empty(max(nws, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(100)]
    for i, o in enumerate(outs):
        for status in (
                L.fp8bs_act_quant(p(xs[i % 2]), 0, M, K, 128, 0, p(q), p(s), st),
                L.fp8bs_fp8_gemm(p(q), p(s), p(w), p(ws_), M, N, K, p(y), p(ws), nws, st),
                L.fp8bs_int4_linear_gated(p(y), M, *[p(t) for t in (*gate, *up)], F, N, 64, p(h), 0, st),
                L.fp8bs_int4_linear(p(h), M, p(down[0]), p(down[1]), K, F, 64, p(o), 0, st)):
            fp8bs._check(status)
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(o), _bits(want[i % 2])) for i, o in enumerate(outs))
    assert fp8bs.device_error() == 0
