"""The residual sum h = res_scale r + branch_scale gate u of the norms around a
block, where its two products meet: both are rounded to fp32 before the sum, so
products that cancel leave 0, and equal scales treat b and r alike."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# columns: eight per thread, one per thread, and rows longer than the registers of either
COLUMNS = [512, 3200, 313, 1001, 17408, 16001]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def tokens(M, K, dt, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, generator=gen, device="cuda") * 2).to(dt)


@pytest.mark.parametrize("pre", [B.BL_NORM_RMS, B.BL_NORM_LAYER])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", COLUMNS)
def test_cancelling_products_leave_zero(K, dt, pre):
    """r = -b under equal scales: h, y and the codes are 0 (one product with its rounding inside the sum leaves some
    2^-25 of itself, which the next norm blows up)."""
    b = tokens(5, K, dt, K)
    h, y = torch.empty_like(b), torch.empty_like(b)
    xq, scale = torch.full((5, K), 7, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    B.bitlinear_residual_norm(b, -b, h, res_scale=0.9, branch_scale=0.9, pre=pre, pre_eps=1e-6, y=y, xq=xq, scale=scale)
    assert not h.any() and not y.any() and not xq.any()
    assert (scale == 1e-6).all()


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("K", COLUMNS)
def test_equal_to_the_formula_in_fp32(K, dt, biased):
    """Without a norm before the sum every step is one fp32 operation of the formula: the same bits (0.9 and 0.6 give
    bf16 inputs many sums halfway between two bf16 values).  A bias of 0 is no other value."""
    b, r = tokens(7, K, dt, K + 1), tokens(7, K, dt, K + 2)
    h = torch.empty_like(r)
    zero = torch.zeros(K, device="cuda") if biased else None
    B.bitlinear_residual_norm(b, r, h, post_b=zero, res_scale=0.9, branch_scale=0.6)
    rs, bs = (torch.tensor(s, dtype=F32, device="cuda") for s in (0.9, 0.6))
    assert torch.equal(h, (rs * r.float() + bs * b.float()).to(dt))


@pytest.mark.parametrize("K", COLUMNS)
def test_equal_scales_treat_both_alike(K):
    b, r = tokens(3, K, F32, K + 3), tokens(3, K, F32, K + 4)
    h1, h2 = torch.empty_like(r), torch.empty_like(r)
    B.bitlinear_residual_norm(b, r, h1, res_scale=0.7, branch_scale=0.7)
    B.bitlinear_residual_norm(r, b, h2, res_scale=0.7, branch_scale=0.7)
    assert torch.equal(h1, h2)
