"""Slopes of the activations as computed, before any rounding to bf16: the slope of
one token is dbias itself (dy = 1).  And values for bf16 outputs, seen through a
residual that takes their leading bits away.

Bounds, from the documented errors of the functions (ulp = at most 2^-23 of a value):
SiLU for bf16 gradients: exp(-z) within (2 + 1.173 |z|) ulp, the divide 2 ulp, the sum
below it 2^-24, so s within D = ((1 - s) (2 + 1.173 |z|) + 2.5) 2^-23; s + z s (1 - s)
moves by s D (1 + |z| |1 - 2 s|), and three roundings add 3 2^-24 of the terms: below (3
+ |z|) 2^-22 s (1 + |z|).  For fp32 gradients the exponential has 2 ulp whatever z.
GELU: the exponent -z^2 / 2 is off by at most 2.5 2^-24 of itself, the exponential 2^-22,
the tail's fit 2^-21, five roundings 2^-24 each: below (4 + z^2 / 2) 2^-22 (Phi + |z| phi);
for fp32 gradients erfc within 4 ulp of its rounded argument, which moves it by 1.5 z^2
2^-24: the same.  Slopes below 2^-118 may be 0 for bf16 gradients, and numbers below
2^-126 have a fixed step."""
import math

import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def points(zdt):
    if zdt == BF16:     # every bf16 value up to 100
        z = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(BF16)
        return z[z.abs() <= 100][None].contiguous()
    z = torch.cat([torch.linspace(-100, 100, 1 << 20, device="cuda"), torch.linspace(-15, 15, 1 << 20, device="cuda")])
    return z[None].contiguous()


def slopes(z, act, dt):
    dy, db = torch.ones(z.shape, dtype=dt, device="cuda"), torch.empty(z.shape[1], device="cuda")
    ws = torch.zeros(B.bitlinear_epilogue_backward_workspace_bytes(*z.shape), dtype=torch.uint8, device="cuda")
    B.bitlinear_epilogue_backward(dy, z, act, None, db, ws)
    return db.double()


LOW = {BF16: 2.0 ** -118, F32: 2.0 ** -140}


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("zdt", [BF16, F32])
def test_silu(zdt, dt):
    z = points(zdt)
    d = z[0].double()
    s, c = torch.sigmoid(d), torch.sigmoid(-d)
    error = (slopes(z, B.BL_ACT_SILU, dt) - (s + d * s * c)).abs()
    assert (error <= (3 + d.abs()) * 2.0 ** -22 * s * (1 + d.abs()) + LOW[dt]).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("zdt", [BF16, F32])
def test_gelu(zdt, dt):
    z = points(zdt)
    d = z[0].double()
    cdf = torch.where(d < 0, 0.5 * torch.special.erfc(-d / math.sqrt(2)), 1 - 0.5 * torch.special.erfc(d / math.sqrt(2)))
    term = d * torch.exp(-d * d / 2) / math.sqrt(2 * math.pi)
    error = (slopes(z, B.BL_ACT_GELU, dt) - (cdf + term)).abs()
    assert (error <= (4 + d * d / 2) * 2.0 ** -22 * (cdf + term.abs()) + LOW[dt]).all()


@pytest.mark.parametrize("act", [B.BL_ACT_SILU, B.BL_ACT_GELU])
def test_not_a_number_stays(act):
    z = torch.full((1, 8), float("nan"), dtype=BF16, device="cuda")
    assert slopes(z, act, BF16).isnan().all() and slopes(z.float(), act, F32).isnan().all()


def test_far_values():
    """Where the exponential has gone to 0 the slope is 0 or 1."""
    z = torch.tensor([[-3e38, -1e20, -500.0, 500.0, 1e20, 3e38, -200.0, 200.0]], device="cuda")
    want = (z[0] > 0).double()
    for act in (B.BL_ACT_SILU, B.BL_ACT_GELU):
        for dt in (BF16, F32):
            got = slopes(z, act, dt)
            assert torch.equal(got, want), (act, dt, got)


@pytest.mark.parametrize("act", [B.BL_ACT_SILU, B.BL_ACT_GELU])
def test_values_before_the_rounding(act):
    """Weights of 0 leave act(bias) + residual.  With minus the bf16 value of act as the residual the sum is at most a
    half step, 2^-8 of act, and its own rounding 2^-8 of that."""
    z = points(F32)[0]
    N, K = z.numel(), 64
    d = z.double()
    a = d * torch.sigmoid(d) if act == B.BL_ACT_SILU else 0.5 * d * torch.special.erfc(-d / math.sqrt(2))
    res = -a.to(BF16)[None].contiguous()
    y = torch.empty(1, N, dtype=BF16, device="cuda")
    ws = torch.zeros(B.bitlinear_forward_epilogue_workspace_bytes(1, N, K, B.BL_PACK_I2, B.BL_I8), dtype=torch.uint8,
                     device="cuda")
    B.bitlinear_forward_epilogue(torch.full((N, 16), 0x55, dtype=torch.uint8, device="cuda"), B.BL_PACK_I2,
                                 torch.ones(1, device="cuda"), N, K, torch.ones(1, K, dtype=torch.int8, device="cuda"),
                                 torch.ones(1, device="cuda"), y, ws, bias=z.contiguous(), act=act, residual=res)
    error = (y[0].double() - res[0].double() - a).abs()
    rel = 2.0 ** -17 if act == B.BL_ACT_SILU else (4 + d * d / 2) * 2.0 ** -22
    assert (error <= (rel + 2.0 ** -16 + 2.0 ** -24) * a.abs() + 2.0 ** -118).all()
