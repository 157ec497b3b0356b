"""Which kernel serves the product with an epilogue, told by the workspace it asks
for, and its results bit for bit: z and the two ReLUs are fp32 operations of exact
sums, so torch's are the same.

  decode   one token where the format's decode kernel takes the shape (base 3 from 8.4
           million weights on), two to four tokens of 2-bit layers of 2^24, 2^26 and
           2^28 weights: the header alone
  few      up to 64 tokens, from packed weights: their codes in pieces, and sums
  many     more tokens, or fewer where it is estimated to be faster: int8 copies"""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

pytestmark = pytest.mark.gpu

I2, T5, B1 = B.BL_PACK_I2, B.BL_PACK_T5, B.BL_PACK_B1
F32, BF16 = torch.float32, torch.bfloat16
HEADER = 256
PIECES = {I2: 4, T5: 5, B1: 8}      # of 16 codes in a packed segment


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def few_bytes(M, K, fmt):
    tokens = next(n for n in (8, 16, 32, 64) if M <= n)
    chunks = (B.bitlinear_packed_row_bytes(K, fmt) // 16 + 3) // 4
    return HEADER + chunks * PIECES[fmt] * tokens * 64 + 4 * tokens


def weights(N, K, fmt, gen):
    """Packed rows and their codes."""
    per, base, shift = {I2: (4, 4, 1), T5: (5, 3, 1), B1: (8, 2, 0)}[fmt]
    rb = B.bitlinear_packed_row_bytes(K, fmt)
    top = 3 if fmt != B1 else 2
    packed = torch.empty(N, rb, dtype=torch.uint8, device="cuda")
    codes = torch.empty(N, K, dtype=F32, device="cuda")
    for n0 in range(0, N, 4096):
        n1 = min(N, n0 + 4096)
        d = torch.randint(0, top, (n1 - n0, rb * per), generator=gen, device="cuda", dtype=torch.uint8)
        d[:, K:] = shift
        power = torch.tensor([base ** i for i in range(per)], device="cuda", dtype=torch.uint8)
        packed[n0:n1] = (d.view(n1 - n0, rb, per) * power).sum(-1, dtype=torch.int32).to(torch.uint8)
        codes[n0:n1] = d[:, :K].float() * (2 if fmt == B1 else 1) - 1
    return packed, codes


CASES = [("decode", 1, 640, 512, I2), ("decode", 1, 8640, 3200, I2), ("decode", 1, 8640, 3200, T5),
         ("decode", 1, 2624, 3216, T5), ("decode", 1, 1000, 1024, B1), ("decode", 2, 8640, 3200, I2),
         ("decode", 3, 8640, 8192, I2), ("decode", 4, 28672, 9408, I2),
         ("few", 1, 512, 512, T5), ("few", 1, 40, 1011, B1), ("few", 2, 3200, 3200, I2), ("few", 3, 8640, 3200, I2),
         ("few", 4, 8640, 3200, T5), ("few", 16, 8640, 3200, I2), ("few", 33, 333, 777, B1), ("few", 64, 1024, 1024, T5),
         ("many", 64, 8640, 3200, I2), ("many", 65, 264, 520, T5), ("many", 130, 1011, 777, B1), ("many", 300, 1024, 640, I2)]


@pytest.mark.parametrize("path,M,N,K,fmt", CASES)
@pytest.mark.parametrize("ydt", [BF16, F32])
def test_path_and_bits(path, M, N, K, fmt, ydt):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    packed, codes = weights(N, K, fmt, gen)
    x = torch.randn(M, K, generator=gen, device="cuda").to(BF16)
    bias = torch.randn(N, generator=gen, device="cuda")
    res = torch.randn(M, N, generator=gen, device="cuda").to(ydt)
    gamma = torch.tensor([0.0173], device="cuda")
    need = B.bitlinear_forward_epilogue_workspace_bytes(M, N, K, fmt, B.BL_BF16)
    few = few_bytes(M, K, fmt) if M <= 64 else 0
    assert path == ("decode" if need == HEADER else "few" if need == few else "many"), need
    xq, s_ref = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    B.bitlinear_quantize_acts(x, xq, s_ref)
    factor = gamma * s_ref / torch.full_like(s_ref, 127)      # (torch multiplies by the inverse of a number)
    z_ref = (xq.float() @ codes.t()) * factor[:, None] + bias  # sums below 2^24: exact
    y, z, s = torch.empty(M, N, dtype=ydt, device="cuda"), torch.empty(M, N, dtype=ydt, device="cuda"), torch.empty(M, device="cuda")
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for act in (B.BL_ACT_RELU2, B.BL_ACT_NONE):
        B.bitlinear_forward_epilogue(packed, fmt, gamma, N, K, x, s, y, ws, bias=bias, act=act, residual=res, preact=z)
        a = z_ref.clamp_min(0).square() if act == B.BL_ACT_RELU2 else z_ref
        assert torch.equal(s, s_ref) and torch.equal(z, z_ref.to(ydt)) and torch.equal(y, (a + res.float()).to(ydt))
    assert B.bitlinear_device_status(ws) == B.BL_OK
