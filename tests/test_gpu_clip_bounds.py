"""Clipping at the ends of its bound: infinite norms and infinite bounds."""
import math

import pytest
import torch

import fp8_block_scaled_10_b200 as fp8bs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bound", [0.0, 1.0, 1e300, math.inf])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_infinite_norm_scales_by_zero_whatever_the_bound(bound, dtype):
    grads = [torch.full((300,), 2.0, device="cuda", dtype=dtype), torch.ones(5, device="cuda")]
    grads[0][7] = -math.inf
    outs = [torch.full_like(g, 9.0) for g in grads]
    _, norm = fp8bs.clip_grads(grads, bound, out=outs)
    fp8bs.clip_grads(grads, bound)
    assert float(norm) == math.inf
    for got in (outs, grads):
        others = torch.arange(300, device="cuda") != 7
        assert got[0][7].isnan()                       # inf * 0
        assert (got[0][others] == 0).all() and (got[1] == 0).all()


def test_an_infinite_bound_clips_nothing_and_measures():
    g = torch.Generator(device="cuda").manual_seed(1)
    grads = [torch.randn(1000, generator=g, device="cuda"), torch.randn(33, generator=g, device="cuda").bfloat16()]
    keep = [v.clone() for v in grads]
    _, norm = fp8bs.clip_grads(grads, math.inf)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep)) and torch.equal(norm, fp8bs.grad_norm(keep))
    grads[0][3] = math.nan
    out, norm = fp8bs.clip_grads(grads, math.inf)
    assert norm.isnan() and all(o.isnan().all() for o in out)
