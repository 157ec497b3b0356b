"""dW of gradients near the lower end of fp32's range.  A row of dz is scaled by a
power of two before its product, and the power's inverse times gamma / 127 may lie
below 2^-126 where the results do not.

Tolerance: 2^-16 sum |terms| as for every dW (one run, of at most 32 additions), 4
roundings of the result, and a result or a product dz s below 2^-126 is rounded to
a multiple of 2^-149."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("exponent", [-60, -100, -106, -112, -118, -124])
@pytest.mark.parametrize("gamma", [0.02, 1.0, 3.0e-4])
def test_dw(exponent, gamma):
    M, N, K = 200, 72, 130
    gen = torch.Generator(device="cuda").manual_seed(-exponent)
    dz = (torch.randn(M, N, generator=gen, device="cuda", dtype=torch.float64) * 2.0 ** exponent).to(torch.bfloat16)
    xq = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    scale = 0.5 + 3 * torch.rand(M, generator=gen, device="cuda")
    g = torch.tensor([gamma], device="cuda")
    dw = torch.full((N, K), float("nan"), device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dw_bf16(dz, xq, scale, g, dw, ws)
    x = xq.double() * scale.double()[:, None] / 127
    want, mag = g.double() * (dz.double().t() @ x), g.double() * (dz.double().abs().t() @ x.abs())
    low = 2.0 ** -149 * (1 + g.double() * xq.double().abs().sum(0) / 127)
    bad = ~((dw.double() - want).abs() <= 2.0 ** -16 * mag + 4 * U * want.abs() + low)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, the worst by " \
                          f"{float(((dw.double() - want).abs() / mag).nan_to_num(0).max()):.3g} of its terms"
