"""dW of rows of dz whose entries differ by more than two fp16 parts hold.

Tolerance: 2^-16 sum |terms| and 4 roundings of the result, as for every dW, and
2^-38 of the row's largest dz s for each entry: the row is scaled so that its largest
is at 2^13 or above, where the second part's half step is 2^-25."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
M, N, K = 300, 72, 136


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def inputs(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dz = torch.randn(M, N, generator=gen, device="cuda")
    xq = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    return dz, xq, 0.5 + torch.rand(M, generator=gen, device="cuda"), torch.tensor([0.02], device="cuda")


def dw_of(dz, xq, scale, gamma):
    dw = torch.empty(N, K, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dw_bf16(dz, xq, scale, gamma, dw, ws)
    assert B.bitlinear_device_status(ws) == B.BL_OK
    return dw


@pytest.mark.parametrize("below", [10, 20, 30, 36, 50])
def test_one_large_token(below):
    """Token 7 is 2^below times the others, and its codes are 0: the others alone make the result."""
    dz, xq, scale, gamma = inputs(below)
    dz[7] *= 2.0 ** below
    dz = dz.to(torch.bfloat16)
    xq[7] = 0
    x = xq.double() * scale.double()[:, None] / 127
    want, mag = gamma.double() * (dz.double().t() @ x), gamma.double() * (dz.double().abs().t() @ x.abs())
    largest = (dz.double().abs() * scale.double()[:, None]).amax(0)[:, None]
    lost = 2.0 ** -38 * largest * gamma.double() * xq.double().abs().sum(0) / 127
    assert ((dw_of(dz, xq, scale, gamma).double() - want).abs() <= 2.0 ** -16 * mag + 4 * U * want.abs() + lost).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3e38])
def test_not_finite_in_one_row(value):
    """(3e38 times its token's scale is beyond fp32.)"""
    dz, xq, scale, gamma = inputs(3)
    dz = dz.to(torch.bfloat16)
    scale[11] = 1.4
    want = dw_of(dz, xq, scale, gamma)
    dz[11, 5] = value
    got = dw_of(dz, xq, scale, gamma)
    rest = torch.arange(N, device="cuda") != 5
    assert got[5].isnan().all() and torch.equal(got[rest], want[rest])
