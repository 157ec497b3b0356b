"""The error of the gradient products over contractions of many runs: below
(2^-17 + (17 + R) 2^-24) sum |terms| for R runs of 512 rows (dx) or 256 tokens (dW).

Every term is positive, so that the sum of magnitudes is the result itself.  With
dW's terms the same for every token each run has the same sum, and adding it to the
registers loses the same share every time while the total keeps its binade: the
loss grows with the number of runs as the bound says it may (over 4096 runs the worst
of these measured above 2^-16)."""
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


def bound(runs):
    return 2.0 ** -17 + (17 + runs) * 2.0 ** -24


# the product from packed words (up to 32 tokens) and the one in tensor memory; a cut contraction and whole ones
@pytest.mark.parametrize("M,N,K", [(3, 131072, 64), (32, 131072, 640), (40, 131072, 64), (300, 70000, 2048)])
def test_dx(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M)
    packed = torch.full((N, (K + 63) // 64 * 16), 0xAA, dtype=torch.uint8, device="cuda")   # codes of +1
    dz = (0.5 + torch.rand(M, N, generator=gen, device="cuda")).to(torch.bfloat16)
    gamma = torch.tensor([0.02], device="cuda")
    dx = torch.empty(M, K, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, B.BL_PACK_I2), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dx_bf16(packed, B.BL_PACK_I2, gamma, N, K, dz, dx, ws)
    assert B.bitlinear_device_status(ws) == B.BL_OK
    want = gamma.double() * dz.double().sum(1, keepdim=True)
    assert ((dx.double() - want).abs() <= (bound(-(-N // 512)) + 4 * U) * want).all()


@pytest.mark.parametrize("M", [40000, 1 << 20])
def test_dw(M):
    N = K = 64
    gen = torch.Generator(device="cuda").manual_seed(M)
    row = (0.5 + torch.rand(N, generator=gen, device="cuda")).to(torch.bfloat16)
    col = torch.randint(1, 128, (K,), generator=gen, device="cuda", dtype=torch.int8)
    dz, xq = row.expand(M, N).contiguous(), col.expand(M, K).contiguous()
    scale, gamma = torch.full((M,), 0.7, device="cuda"), torch.tensor([0.02], device="cuda")
    dw = torch.empty(N, K, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dw_bf16(dz, xq, scale, gamma, dw, ws)
    assert B.bitlinear_device_status(ws) == B.BL_OK
    want = gamma.double() * M * row.double()[:, None] * (scale[0].double() * col.double() / 127)
    assert ((dw.double() - want).abs() <= (bound(-(-M // 256)) + 4 * U) * want).all()
