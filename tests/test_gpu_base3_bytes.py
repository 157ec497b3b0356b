"""Every base-3 byte value at every position of a 16-byte segment, through each
kernel that takes such words apart: bytes 0..242 are five digits, 243..255 (which
no encoder writes) five weights of 0.  Outputs are compared bit for bit: integer
sums, and small integers in fp32."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

N, K = 256, 400  # 80 bytes a row: five segments


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def packed():
    """Byte b of row n is n + 37 b mod 256: each value meets each position."""
    n, b = torch.arange(N, device="cuda")[:, None], torch.arange(80, device="cuda")[None]
    return ((n + 37 * b) % 256).to(torch.uint8)


def weights(p):
    v = torch.where(p < 243, p.long(), 121)
    return torch.stack([v // 3 ** i % 3 - 1 for i in range(5)], dim=2).reshape(N, -1)[:, :K].double()


def tokens(M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    return torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)


# one token (decode), a few, the one-SM product and the two-SM product
@pytest.mark.parametrize("M", [1, 3, 5, 16, 128, 300])
def test_plain_forward(M):
    p, xq = packed(), tokens(M)
    y = torch.empty(M, N, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.bitlinear_forward_workspace_bytes(M, N, K, B.BL_PACK_T5, B.BL_I8), dtype=torch.uint8, device="cuda")
    one = torch.ones(M, device="cuda")
    B.bitlinear_forward(p, B.BL_PACK_T5, one[:1], N, K, xq, one, y, ws)
    assert B.bitlinear_device_status(ws) == B.BL_OK
    assert torch.equal(y.double(), xq.double() @ weights(p).t())


# the decode kernel's size aside: a few tokens, and the product on expanded weights
@pytest.mark.parametrize("M", [1, 5, 16, 64, 65, 300])
def test_epilogue_forward(M):
    p, xq = packed(), tokens(M)
    y = torch.empty(M, N, device="cuda")
    ws = torch.zeros(B.bitlinear_forward_epilogue_workspace_bytes(M, N, K, B.BL_PACK_T5, B.BL_I8), dtype=torch.uint8,
                     device="cuda")
    scale = torch.full((M,), 127.0, device="cuda")  # (1 * 127) / 127: a factor of 1
    B.bitlinear_forward_epilogue(p, B.BL_PACK_T5, scale[:1] / 127, N, K, xq, scale, y, ws)
    assert torch.equal(y.double(), xq.double() @ weights(p).t())


# from packed words, and through the bf16 copy of the weights
@pytest.mark.parametrize("M", [1, 32, 33, 300])
def test_dx(M):
    p = packed()
    gen = torch.Generator(device="cuda").manual_seed(M)
    dz = torch.randint(-8, 9, (M, N), generator=gen, device="cuda").to(torch.bfloat16)
    dx = torch.empty(M, K, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, B.BL_PACK_T5), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dx_bf16(p, B.BL_PACK_T5, torch.ones(1, device="cuda"), N, K, dz, dx, ws)
    assert torch.equal(dx.double(), dz.double() @ weights(p))
