"""The gradient products on the tensor cores against fp64 products of the same
inputs.

Tolerance: the products of bf16 dz and the codes are exact; dW's two fp16 parts
keep 22 bits of fl(dz s) (error below 2^-22 and 2^-24 of a term).  A run adds 32
partial products (K = 16 MMAs) in fp32, each addition losing less than 2^-22 of
the magnitudes added so far, and at most 32 runs add in fp32 registers: below
2^-16 sum |terms| in all.  alpha takes
three roundings; a bf16 output half a step, 2^-8."""
import numpy as np
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B
from bitlinear_b1_fwd_b200 import synth
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
I2, T5, B1 = B.BL_PACK_I2, B.BL_PACK_T5, B.BL_PACK_B1
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


class Case:
    def __init__(self, orc, M, N, K, fmt, seed, spread=False):
        self.M, self.N, self.K, self.fmt = M, N, K, fmt
        W = synth.normal_f32(seed, (N, K), 0.02)
        if fmt == B1:
            _, g, codes = orc.binarize_weights(W)
        else:
            g = orc.gamma(W)
            codes = orc.ternarize(W, g, 1e-5)
        self.codes = torch.from_numpy(codes.astype(np.float64)).cuda()
        self.packed = dev(orc.pack(codes, fmt))
        self.gamma = torch.tensor([float(g)], device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dz = torch.randn(M, N, generator=gen, device="cuda") * 1e-3
        if spread:      # rows of very different size, a row and a column of zeros, tiny entries
            dz *= 2.0 ** torch.randint(-60, 60, (1, N), generator=gen, device="cuda").float()
            dz *= 2.0 ** torch.randint(-6, 1, (M, N), generator=gen, device="cuda").float()
            dz[:, N // 2] = 0
            dz[M // 2] = 0
        self.dz = dz.to(BF16)
        x = torch.randn(M, K, generator=gen, device="cuda") * (0.1 + 3 * torch.rand(M, 1, generator=gen, device="cuda"))
        xq, s = orc.act_quant(host(x))
        self.xq, self.scale = dev(xq), dev(s)

    def dx(self, dt=F32, ws=None, out=None, stream=None):
        out = torch.full((self.M, self.K), float("nan"), dtype=dt, device="cuda") if out is None else out
        if ws is None:
            ws = torch.zeros(B.bitlinear_backward_dx_bf16_workspace_bytes(self.M, self.N, self.K, self.fmt),
                             dtype=torch.uint8, device="cuda")
        B.bitlinear_backward_dx_bf16(self.packed, self.fmt, self.gamma, self.N, self.K, self.dz, out, ws, stream=stream)
        assert stream is not None or torch.cuda.is_current_stream_capturing() or B.bitlinear_device_status(ws) == B.BL_OK
        return out

    def dw(self, ws=None, out=None, stream=None):
        out = torch.full((self.N, self.K), float("nan"), device="cuda") if out is None else out
        if ws is None:
            ws = torch.zeros(B.bitlinear_backward_dw_bf16_workspace_bytes(self.M, self.N, self.K), dtype=torch.uint8,
                             device="cuda")
        B.bitlinear_backward_dw_bf16(self.dz, self.xq, self.scale, self.gamma, out, ws, stream=stream)
        assert stream is not None or torch.cuda.is_current_stream_capturing() or B.bitlinear_device_status(ws) == B.BL_OK
        return out

    def check_dx(self, got):
        g, d = self.gamma.double(), self.dz.double()
        want, mag = g * (d @ self.codes), g * (d.abs() @ self.codes.abs())
        h = 0.0 if got.dtype == F32 else torch.finfo(got.dtype).eps / 2
        self._check(got, want, 2.0 ** -16 * mag + (h + 4 * U) * want.abs() + 1e-38)

    def check_dw(self, got):
        g, d = self.gamma.double(), self.dz.double()
        x = self.xq.double() * self.scale.double()[:, None] / 127
        want, mag = g * (d.t() @ x), g * (d.abs().t() @ x.abs())
        self._check(got, want, 2.0 ** -16 * mag + 4 * U * want.abs() + 1e-38)

    @staticmethod
    def _check(got, want, tol):
        bad = ~((got.double() - want).abs() <= tol)
        assert not bad.any(), f"{int(bad.sum())} off, first {bad.nonzero()[:4].tolist()}, worst " \
                              f"{float(((got.double() - want).abs() / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


# tokens from one, sizes on and off the 256 tile and the 64-element stage, odd widths (padded copies), one row or
# column, contractions shorter than a stage and longer than several runs
SHAPES = [(256, 256, 256, I2), (1, 64, 64, I2), (1, 1, 1, I2), (2, 77, 33, T5), (16, 264, 520, I2), (33, 100, 1000, B1),
          (128, 1031, 256, I2), (130, 640, 512, T5), (257, 513, 259, I2), (600, 1280, 136, B1), (1100, 72, 320, I2),
          (64, 3200, 640, I2), (300, 8, 2056, I2)]


@pytest.mark.parametrize("M,N,K,fmt", SHAPES)
def test_products(orc, M, N, K, fmt):
    c = Case(orc, M, N, K, fmt, 1200 + M)
    for dt in (F32, BF16):
        c.check_dx(c.dx(dt))
    c.check_dw(c.dw())
    # the same bits again
    assert torch.equal(c.dx(), c.dx()) and torch.equal(c.dw(), c.dw())


# up to 32 tokens take packed weights: row counts on and off the step of 16, columns on and off the block of 128,
# one range of rows and several, more rows than one warp adds up, every format; 33 tokens do not
@pytest.mark.parametrize("M,N,K,fmt", [(1, 15, 129, I2), (8, 16, 128, I2), (16, 4097, 96, I2), (17, 333, 1000, T5),
                                       (32, 9000, 40, I2), (31, 8640, 320, B1), (5, 40000, 130, I2), (32, 100, 5000, T5),
                                       (33, 100, 500, T5)])
def test_dx_of_a_few_tokens(orc, M, N, K, fmt):
    c = Case(orc, M, N, K, fmt, 1300 + M)
    f, b = c.dx(F32), c.dx(BF16)
    c.check_dx(f)
    c.check_dx(b)
    assert torch.equal(c.dx(F32), f) and torch.equal(f.to(BF16), b)


@pytest.mark.parametrize("M,N,K", [(200, 300, 264), (70, 129, 64)])
def test_gradients_of_very_different_size(orc, M, N, K):
    """Each output row of dW has its own power of two: rows 2^-60 .. 2^60 apart keep their precision."""
    c = Case(orc, M, N, K, I2, 1250 + M, spread=True)
    c.check_dx(c.dx())
    dw = c.dw()
    c.check_dw(dw)
    assert (dw[N // 2] == 0).all()


def test_agrees_with_the_fp64_backward(orc):
    c = Case(orc, 6, 320, 256, I2, 1260)
    dx = torch.empty(6, 256, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dx_workspace_bytes(6, 320, 256, I2), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dx(c.packed, I2, c.gamma, 320, 256, c.dz, dx, ws)
    dw = torch.empty(320, 256, device="cuda")
    B.bitlinear_backward_dw(c.dz, c.xq, c.scale, c.gamma, dw)
    c.check_dx(dx)
    c.check_dw(dw)
    assert torch.allclose(c.dx(), dx, rtol=2.0 ** -16, atol=2.0 ** -16 * float(dx.abs().max()))
    assert torch.allclose(c.dw(), dw, rtol=2.0 ** -16, atol=2.0 ** -16 * float(dw.abs().max()))


def test_precision_of_long_contractions(orc):
    """Random signs over 4096 tokens and 4096 rows: the 2-norm error stays at fp32's level (each run loses less
    than 2^-22 of itself per addition, with signs that mostly cancel: a few 2^-23 in all, and 1e-6 is 8 x 2^-23)."""
    c = Case(orc, 4096, 4096, 256, I2, 1270)
    want = c.gamma.double() * (c.dz.double() @ c.codes)
    assert float((c.dx().double() - want).norm() / want.norm()) < 1e-6
    x = c.xq.double() * c.scale.double()[:, None] / 127
    want = c.gamma.double() * (c.dz.double().t() @ x)
    assert float((c.dw().double() - want).norm() / want.norm()) < 1e-6


def test_empty_batch(orc):
    c = Case(orc, 1, 40, 48, I2, 1280)
    dw = torch.full((40, 48), 5.0, device="cuda")
    ws = torch.zeros(B.bitlinear_backward_dw_bf16_workspace_bytes(0, 40, 48), dtype=torch.uint8, device="cuda")
    B.bitlinear_backward_dw_bf16(c.dz[:0], c.xq[:0], c.scale[:0], c.gamma, dw, ws)
    assert (dw == 0).all()
    B.bitlinear_backward_dx_bf16(c.packed, I2, c.gamma, 40, 48, c.dz[:0], torch.empty(0, 48, device="cuda"), ws)


def test_guards_streams_and_graphs(orc):
    for M, N, K, fmt in ((17, 33, 77, T5), (140, 264, 520, I2)):
        c = Case(orc, M, N, K, fmt, 1290)
        want_dx, want_dw = c.dx(), c.dw()
        for which, need, shape, want in (
                ("dx", B.bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, fmt), (M, K), want_dx),
                ("dw", B.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K), (N, K), want_dw)):
            n = 4 * shape[0] * shape[1]
            buf = torch.full((2, 8192 + -(-max(need, n) // 256) * 256), 0xA5, dtype=torch.uint8, device="cuda")
            ws, out = buf[0, 4096:4096 + need], buf[1, 4096:4096 + n].view(F32).view(shape)
            ws[:256] = 0
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            (c.dx(ws=ws, out=out, stream=side) if which == "dx" else c.dw(ws=ws, out=out, stream=side))
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            for i, k in ((0, need), (1, n)):
                assert (buf[i, :4096] == 0xA5).all() and (buf[i, 4096 + k:] == 0xA5).all()
            graphs, outs = [], []
            for _ in range(2):      # two graphs share the workspace, replayed in turn on one stream
                g, o = torch.cuda.CUDAGraph(), torch.empty_like(want)
                with torch.cuda.graph(g):
                    c.dx(ws=ws, out=o) if which == "dx" else c.dw(ws=ws, out=o)
                graphs.append(g)
                outs.append(o)
            for _ in range(2):
                for g in graphs:
                    g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(o, want) for o in outs)
            assert B.bitlinear_device_status(ws) == B.BL_OK
