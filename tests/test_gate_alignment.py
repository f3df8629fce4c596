"""The gate's backward pass takes tensors that are aligned to their elements alone:
rows cut from a tensor of odd width, views that start anywhere."""
import ctypes

import pytest
import torch

import fp8_block_scaled_10_b200 as fp8bs
from fp8_block_scaled_10_b200 import build as fbuild


def test_two_byte_alignment_passes_the_argument_checks():
    """(Here without a GPU the call then stops at the device.)"""
    fbuild.build()
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    L, at = fp8bs.lib(), lambda k: ctypes.c_void_p(4096 + k)   # noqa: E731
    for N in (7, 8):
        for args in ((2, 0, 0, 0), (0, 6, 0, 0), (0, 0, 14, 0), (0, 0, 0, 10)):
            gu, dh, dgu, h = map(at, args)
            assert L.fp8bs_gated_backward(gu, dh, 4, N, dgu, h, None) not in (fp8bs.OK, fp8bs.ERR_INVALID_ARG)
        for args in ((1, 0, 0, 0), (0, 3, 0, 0), (0, 0, 5, 0), (0, 0, 0, 9)):
            gu, dh, dgu, h = map(at, args)
            assert L.fp8bs_gated_backward(gu, dh, 4, N, dgu, h, None) == fp8bs.ERR_INVALID_ARG


def _inputs(M, N, shift_gu, shift_dh):
    """gu [M, 2N] and dh [M, N] that start the given number of elements into their storage."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    gu = (torch.randn(M * 2 * N + 8, generator=g, device="cuda") * 2).bfloat16()
    dh = (torch.randn(M * N + 8, generator=g, device="cuda") * 1e-2).bfloat16()
    return (gu[shift_gu:shift_gu + 2 * M * N].view(M, 2 * N), dh[shift_dh:shift_dh + M * N].view(M, N))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(5, 7), (33, 256), (200, 1001), (9, 2048), (3, 4104)])
@pytest.mark.parametrize("shift_gu,shift_dh", [(1, 0), (0, 1), (3, 5), (4, 4), (7, 2)])
def test_shifted_views_give_the_same_bits(M, N, shift_gu, shift_dh):
    gu, dh = _inputs(M, N, shift_gu, shift_dh)
    got = fp8bs.gated_backward(gu, dh, return_h=True)
    want = fp8bs.gated_backward(gu.clone(), dh.clone(), return_h=True)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    assert torch.equal(fp8bs.gated_backward(gu, dh), got[0])


@pytest.mark.gpu
def test_rows_cut_from_an_odd_width():
    gu, dh = _inputs(40, 577, 0, 0)
    whole = fp8bs.gated_backward(gu, dh)
    assert torch.equal(fp8bs.gated_backward(gu[3:20], dh[3:20]), whole[3:20])
    assert fp8bs.device_error() == 0
