"""The gate's accuracy over its whole range, from pre-activations that are exact
(one product by a power of two), against 64 bits.  The bounds are the header's:
2^-20 relative for the 4-bit pair, whose output may be fp32; (1.25 |g| + 10) 2^-24 and
nothing below -87.3 for the calls with bf16 outputs."""
import pytest
import torch

import fp8_block_scaled_10_b200 as fp8bs

pytestmark = pytest.mark.gpu

BF16_HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from fp8_block_scaled_10_b200 import build
    build.build()
    yield
    assert fp8bs.device_error() == 0


def _gates():
    """bf16 values from -175 to 60, dense where something changes."""
    v = torch.cat([torch.linspace(-175, -80, 96), torch.linspace(-90, -78, 64), torch.linspace(-80, 8, 160),
                   torch.tensor([-1e-3, -1e-30, -0.0, 0.0, 1e-30, 1e-3, 17.0, 60.0])])
    return v.bfloat16().cuda()


def _silu(g):
    return g / (1 + torch.exp(-g))


def _check(y, ref, tol, what):
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(nan=1e9).max()))


def _codes_at(channel, rows):
    """Packed codes of a [rows, 128] weight that is 1 at one channel and 0 elsewhere
    (nibble 8 is 0): the word, nibble and byte of the layout in include/fp8bs.h."""
    q = torch.full((rows, 64), 0x88, dtype=torch.uint8)
    j, t, e = channel // 32, channel % 32 // 8, channel % 8
    p = e // 2 + 4 * (e % 2)
    q[:, 16 * t + 4 * j + p // 2] += 1 << (4 * (p % 2))
    return q.cuda()


@pytest.mark.parametrize("up", [1.0, -3.0, 1000.0, 1e30, 1e-20])
@pytest.mark.parametrize("tokens", [8, 16, 400])
def test_int4_gate_from_far_below_to_far_above(tokens, up):
    g = _gates()
    x = torch.zeros(g.numel(), 128, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = g
    x[:, 37] = up
    u = x[:, 37].double()
    ref = (_silu(g.double()) * u)[:, None].expand(-1, 12)
    scale = torch.ones(12, 1, device="cuda")
    pair = (_codes_at(0, 12), scale, _codes_at(37, 12), scale)
    for dtype in (torch.float32, torch.bfloat16):
        got = torch.cat([fp8bs.int4_linear_gated(part, *pair, out_dtype=dtype) for part in x.split(tokens)])
        # subnormal results: half a step of the format, and of fp32 before the last product
        tol = 2.0 ** -20 * ref.abs() + 2.0 ** -148
        if dtype is torch.bfloat16:
            tol = BF16_HALF * (ref.abs() + tol) + tol + 2.0 ** -134
        _check(got, ref, tol, str(dtype))


def test_int4_gate_passes_nan_and_infinity():
    x = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([float("nan"), 200.0, -200.0, -1000.0])
    x[:, 1] = torch.tensor([1.0, 2.0, 3.0, 1e30])
    scale = torch.ones(4, 1, device="cuda")
    h = fp8bs.int4_linear_gated(x, _codes_at(0, 4), scale, _codes_at(1, 4), scale, out_dtype=torch.float32)
    assert h[0].isnan().all() and (h[1] == 400.0).all() and (h[2:] == 0).all()


@pytest.mark.parametrize("K", [128, 7168])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_fp8_gate_keeps_its_stated_bound(K, sign):
    """K = 7168 splits K: the gate of the reduction; 128: the GEMM's own."""
    g = torch.cat([torch.linspace(0.01, 30, 40), torch.linspace(30, 89, 60)]).cuda()   # |g|
    M, N = g.numel(), 128
    one = torch.zeros(max(M, N), K, device="cuda")
    one[:, 0] = 1
    one = one.to(torch.float8_e4m3fn)
    a_s = torch.ones(M, K // 128, device="cuda")
    a_s[:, 0] = g
    ws = torch.ones(1, K // 128, device="cuda")
    gate = (sign * one[:N].float()).to(torch.float8_e4m3fn)
    h, gu = fp8bs.fp8_gemm_gated(one[:M], a_s, gate, ws, one[:N], 4 * ws, return_gu=True)
    gd = sign * g.double()[:, None].expand(M, N)
    assert torch.equal(gu[:, :N], gd.bfloat16())
    ref = _silu(gd) * 4 * g.double()[:, None]
    rel = (1.25 * gd.abs() + 10) * 2.0 ** -24
    tol = BF16_HALF * (1 + rel) * ref.abs() + rel * ref.abs() + torch.where(gd < -87.3, ref.abs(), 0.0)
    _check(h, ref, tol, "h")


@pytest.mark.parametrize("N", [400, 401])
def test_gate_backward_keeps_its_stated_bound(N):
    g = _gates()
    g = torch.cat([g, g, g])[:N][None].expand(3, N)
    u = torch.tensor([[1.0], [-40.0], [1e-3]], device="cuda").expand(3, N)
    gu = torch.cat([g, u.bfloat16()], 1).contiguous()
    dh = torch.tensor([[1.0], [0.01], [-7.0]], device="cuda").bfloat16().expand(3, N).contiguous()
    dgu, h = fp8bs.gated_backward(gu, dh, return_h=True)
    gd, ud, d = gu[:, :N].double(), gu[:, N:].double(), dh.double()
    p = 1 / (1 + torch.exp(-gd))
    rel = (1.25 * gd.abs() + 10) * 2.0 ** -24
    shut = lambda ref: torch.where(gd < -87.3, ref.abs(), 0.0)   # noqa: E731
    for what, got, ref, err in (("du", dgu[:, N:], d * gd * p, rel * (d * gd * p).abs()),
                                ("h", h, gd * p * ud, rel * (gd * p * ud).abs()),
                                # 1 + g (1 - p): p's error enters |g| + 1 fold
                                ("dg", dgu[:, :N], d * ud * p * (1 + gd * (1 - p)),
                                 rel * (d * ud).abs() * p * (2 + 2 * gd.abs()))):
        _check(got, ref, BF16_HALF * (ref.abs() + err) + err + shut(ref) + 2.0 ** -133, what)
