"""The bounded waits of the tensor-core products run out: their TMA threads are
switched off and the limit is about a millisecond."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

TIMEOUT, INT8, GRAD = 1, 0x100, 0x200      # bits of the workspace's first word


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def test_each_product_reports_and_the_next_call_is_right():
    ws = torch.zeros(256 + 8192, dtype=torch.uint8, device="cuda")
    B.bitlinear_selftest_wait_timeout(ws)
    assert int(ws[:4].view(torch.int32)) == TIMEOUT | INT8 | GRAD
    assert not ws[256:].any()
    assert B.bitlinear_device_status(ws) == B.BL_ERR_DEVICE_TIMEOUT
    assert B.bitlinear_device_status(ws) == B.BL_OK
    # both products again, with their producers: integers, exact
    M, N, K = 300, 512, 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    packed = torch.full((N, K // 4), 0xAA, dtype=torch.uint8, device="cuda")        # codes of +1
    one = torch.ones(M, device="cuda")
    y = torch.empty(M, N, device="cuda")
    ws = torch.zeros(max(B.bitlinear_forward_epilogue_workspace_bytes(M, N, K, B.BL_PACK_I2, B.BL_I8),
                         B.bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, B.BL_PACK_I2),
                         B.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K)), dtype=torch.uint8, device="cuda")
    B.bitlinear_forward_epilogue(packed, B.BL_PACK_I2, one[:1], N, K, xq, 127 * one, y, ws)
    assert torch.equal(y.double(), xq.double().sum(1, keepdim=True).expand(M, N))
    dz = torch.randint(-8, 9, (M, N), generator=gen, device="cuda").to(torch.bfloat16)
    dx, dw = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda")
    B.bitlinear_backward_dx_bf16(packed, B.BL_PACK_I2, one[:1], N, K, dz, dx, ws)
    assert torch.equal(dx.double(), dz.double().sum(1, keepdim=True).expand(M, K))
    B.bitlinear_backward_dw_bf16(dz, xq, one, 127 * one[:1], dw, ws)
    assert torch.equal(dw.double(), dz.double().t() @ xq.double())
    assert B.bitlinear_device_status(ws) == B.BL_OK
