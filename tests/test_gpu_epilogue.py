"""The product with bias, activation and residual in its epilogue, and the
gradients through that epilogue, against the formulas in fp64.

Tolerances (u = 2^-24): acc is exact, c_m = (gamma s)/127 and acc c_m take
three roundings and the bias one more, so z is off by at most 3u |acc c| + u
|z|; the activation multiplies that by its slope (at most 1.2, or 2 |z| for
relu^2) and adds its own error: 8u |a| for the elementary functions, and for
GELU the argument of erfc (two roundings, each moving erfc by up to a factor
1 + z^2 u); the residual adds one rounding.  A value stored in bf16 is off by
half a step more, 2^-8 of its size."""
import math

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
ACTS = [B.BL_ACT_NONE, B.BL_ACT_RELU, B.BL_ACT_RELU2, B.BL_ACT_SILU, B.BL_ACT_GELU]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def half_step(t):
    return 0.0 if t == F32 else torch.finfo(t).eps / 2


def act64(z, act):
    """The activation and its derivative in fp64."""
    if act == B.BL_ACT_RELU:
        return z.clamp_min(0), (z > 0).double()
    if act == B.BL_ACT_RELU2:
        return z.clamp_min(0) ** 2, 2 * z.clamp_min(0)
    if act == B.BL_ACT_SILU:
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if act == B.BL_ACT_GELU:
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


class Layer:
    def __init__(self, orc, N, K, fmt, seed):
        W = synth.normal_f32(seed, (N, K), 0.02)
        if fmt == B1:
            _, g, codes = orc.binarize_weights(W)
        else:
            g = orc.gamma(W)
            codes = orc.ternarize(W, g, 1e-5)
        self.N, self.K, self.fmt, self.orc = N, K, fmt, orc
        self.codes = torch.from_numpy(codes.astype(np.float64)).cuda()
        self.packed = dev(orc.pack(codes, fmt))
        self.gamma = torch.tensor([float(g)], device="cuda")

    def reference(self, x, bias, act, res):
        """acc c and z, y in fp64 from the oracle's codes and scales."""
        xq, s = self.orc.act_quant(host(x))
        acc = torch.from_numpy(xq.astype(np.float64)).cuda() @ self.codes.t()
        main = acc * (self.gamma.double() * torch.from_numpy(s).cuda().double() / 127)[:, None]
        z = main if bias is None else main + bias.double()
        y = act64(z, act)[0]
        return main, z, y if res is None else y + res.double(), xq, s

    def run(self, x, ydt, bias=None, act=0, res=None, pre=False, y=None, scale=None, ws=None, stream=None):
        M = x.shape[0]
        y = torch.full((M, self.N), float("nan"), dtype=ydt, device="cuda") if y is None else y
        z = torch.full((M, self.N), float("nan"), dtype=ydt, device="cuda") if pre else None
        scale = torch.empty(M, device="cuda") if scale is None else scale
        if ws is None:
            ws = torch.zeros(B.bitlinear_forward_epilogue_workspace_bytes(M, self.N, self.K, self.fmt, B.dtype_code(x)),
                             dtype=torch.uint8, device="cuda")
        B.bitlinear_forward_epilogue(self.packed, self.fmt, self.gamma, self.N, self.K, x, scale, y, ws, bias=bias,
                                     act=act, residual=res, preact=z, stream=stream)
        return y, z, scale


def bounds(main, z, y, act, ydt):
    a = act64(z, act)[0].abs()
    ez = 3 * U * main.abs() + U * z.abs()
    slope = 2 * z.abs() + ez if act == B.BL_ACT_RELU2 else 1.2
    own = 0 if act in (B.BL_ACT_NONE, B.BL_ACT_RELU) else 8 * U * a + (2 * U * z * z * a if act == B.BL_ACT_GELU else 0)
    ey = slope * ez + own + U * y.abs()
    h = half_step(ydt)
    return ez * (1 + h) + h * z.abs() + 1e-38, ey * (1 + h) + h * y.abs() + 1e-38


def check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {bad.nonzero()[:3].tolist()}, worst " \
                          f"{float(((got.double() - want).abs() / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


# every kernel that serves the forward: one token (each format, aligned and not), 2-4 tokens, the one-SM GEMM at
# each token tile with and without a split of K, the two-SM GEMM; N off every tile, rows of y not 16-byte multiples
SHAPES = [(1, 640, 512, I2), (1, 333, 320, T5), (1, 130, 256, B1), (1, 33, 77, I2), (1, 96, 28672, T5),
          (2, 200, 512, I2), (3, 131, 320, T5), (4, 65, 384, B1), (4, 8640, 256, I2), (7, 96, 130, T5), (9, 50, 77, B1),
          (5, 3200, 8640, I2), (16, 131, 384, B1), (17, 264, 2048, T5), (40, 130, 512, I2), (64, 129, 1024, I2),
          (100, 520, 256, I2), (128, 777, 640, T5), (129, 640, 512, I2), (300, 777, 336, B1), (515, 1032, 640, I2)]


@pytest.mark.parametrize("M,N,K,fmt", SHAPES)
@pytest.mark.parametrize("xdt,ydt", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_forward_epilogue(orc, M, N, K, fmt, xdt, ydt):
    L = Layer(orc, N, K, fmt, 900 + K)
    x = dev(synth.normal_f32(901 + M, (M, K))).to(xdt)
    bias, res = dev(synth.normal_f32(902, (N,), 0.3)), dev(synth.normal_f32(903 + M, (M, N))).to(ydt)
    act = ACTS[(M + N) % len(ACTS)]
    for b, a, r, pre in ((bias, act, res, True), (None, act, None, False), (bias, B.BL_ACT_NONE, None, True),
                         (None, B.BL_ACT_NONE, res, False)):
        y, z, s = L.run(x, ydt, b, a, r, pre)
        main, z64, y64, _, s_ref = L.reference(x, b, a, r)
        assert np.array_equal(host(s), s_ref)
        tz, ty = bounds(main, z64, y64, a, ydt)
        check(y, y64, ty, "y")
        if pre:
            check(z, z64, tz, "z")


# every form at its edges: the packed-weight product at one token and at 8, 16, 32 and 64, K over several parts of
# codes, one token group shared by several warps; the int8 product whole and with K in parts, rows of y and of x that
# are no multiple of 16 bytes, one tile and several; the decode kernels at two tokens
EDGES = [(1, 512, 512, T5), (1, 40, 1011, B1), (2, 8640, 3200, I2), (3, 1040, 77, B1), (8, 16, 16, I2), (16, 17, 9000, I2),
         (32, 50, 12000, T5), (33, 33, 20000, B1), (64, 40, 40, T5), (64, 3200, 3200, I2), (65, 777, 1011, B1),
         (65, 96, 4096, I2), (130, 3200, 640, T5), (257, 264, 130, I2), (600, 777, 1011, T5), (1030, 1000, 72, B1)]


@pytest.mark.parametrize("M,N,K,fmt", EDGES)
def test_forward_epilogue_at_the_edges_of_its_forms(orc, M, N, K, fmt):
    L = Layer(orc, N, K, fmt, 960 + K)
    bias = dev(synth.normal_f32(961, (N,), 0.3))
    x32 = dev(synth.normal_f32(962 + M, (M, K)))
    for act, xdt, ydt in ((B.BL_ACT_SILU, BF16, BF16), (B.BL_ACT_GELU, F32, F32), (B.BL_ACT_GELU, BF16, BF16)):
        x = x32.to(xdt)
        res = dev(synth.normal_f32(963 + M, (M, N))).to(ydt)
        y, z, s = L.run(x, ydt, bias, act, res, True)
        main, z64, y64, xq, s_ref = L.reference(x, bias, act, res)
        assert np.array_equal(host(s), s_ref)
        tz, ty = bounds(main, z64, y64, act, ydt)
        check(y, y64, ty, "y")
        check(z, z64, tz, "z")
        given, zg, _ = L.run(dev(xq), ydt, bias, act, res, True, scale=dev(s_ref))      # codes instead of x
        assert torch.equal(given, y) and torch.equal(zg, z)


def test_two_calls_at_once(orc):
    """Two streams, each with its own workspace and outputs."""
    for M, N, K, fmt in ((12, 1000, 2048, T5), (300, 777, 640, I2)):
        L = Layer(orc, N, K, fmt, 970)
        xs = [dev(synth.normal_f32(971 + i, (M, K))).to(BF16) for i in range(2)]
        want = [L.run(x, BF16, None, B.BL_ACT_SILU)[0] for x in xs]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream() for _ in range(2)], []
        for _ in range(4):
            got.append([L.run(x, BF16, None, B.BL_ACT_SILU, stream=st)[0] for x, st in zip(xs, streams)])
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 20, 140])
def test_every_activation(orc, M, act):
    L = Layer(orc, 264, 512, I2, 910)
    x = dev(synth.normal_f32(911 + M, (M, 512)))
    bias = dev(synth.normal_f32(912, (264,), 4.0))          # both tails of the activation
    y, z, _ = L.run(x, F32, bias, act, None, True)
    main, z64, y64, _, _ = L.reference(x, bias, act, None)
    tz, ty = bounds(main, z64, y64, act, F32)
    check(z, z64, tz, "z")
    check(y, y64, ty, "y")


def test_plain_epilogue_equals_forward(orc):
    """With nothing in the epilogue the outputs are bitlinear_forward's."""
    for M, N, K, fmt in SHAPES:
        L = Layer(orc, N, K, fmt, 920 + N)
        x = dev(synth.normal_f32(921 + M, (M, K))).to(BF16)
        y, _, s = L.run(x, BF16)
        y2, s2 = torch.empty_like(y), torch.empty_like(s)
        ws = torch.zeros(B.bitlinear_forward_workspace_bytes(M, N, K, fmt, B.BL_BF16), dtype=torch.uint8, device="cuda")
        B.bitlinear_forward(L.packed, fmt, L.gamma, N, K, x, s2, y2, ws)
        assert torch.equal(y, y2) and torch.equal(s, s2), (M, N, K, fmt)


@pytest.mark.parametrize("fmt", [I2, T5, B1])
def test_a_token_alone_and_in_a_batch(orc, fmt):
    """y of a token has the same bits whichever kernel serves the batch."""
    L = Layer(orc, 520, 640, fmt, 930)
    x = dev(synth.normal_f32(931, (300, 640))).to(BF16)
    bias, res = dev(synth.normal_f32(932, (520,), 0.3)), dev(synth.normal_f32(933, (300, 520)))
    whole, _, _ = L.run(x, F32, bias, B.BL_ACT_GELU, res)
    for m0, m1 in ((0, 1), (5, 8), (10, 22), (30, 130), (299, 300)):
        part, _, _ = L.run(x[m0:m1].contiguous(), F32, bias, B.BL_ACT_GELU, res[m0:m1].contiguous())
        assert torch.equal(part, whole[m0:m1]), (m0, m1)


@pytest.mark.parametrize("M", [1, 3, 16, 200])
def test_int8_input_and_in_place_residual(orc, M):
    L = Layer(orc, 192, 256, I2, 940)
    x = dev(synth.normal_f32(941 + M, (M, 256)))
    res = dev(synth.normal_f32(942, (M, 192))).to(BF16)
    want, _, s = L.run(x, BF16, None, B.BL_ACT_SILU, res)
    xq, s_ref = L.orc.act_quant(host(x))
    y = res.clone()
    L.run(dev(xq), BF16, None, B.BL_ACT_SILU, y, y=y, scale=dev(s_ref))
    assert torch.equal(y, want)


def test_guards_streams_and_graphs(orc):
    """No write outside y, z, scale and the queried workspace; another stream; two captured graphs on one workspace."""
    for M, N, K, fmt in ((1, 37, 77, I2), (3, 50, 128, I2), (17, 130, 256, T5), (200, 131, 336, I2)):
        L = Layer(orc, N, K, fmt, 950)
        x = dev(synth.normal_f32(951 + M, (M, K))).to(BF16)
        bias = dev(synth.normal_f32(952, (N,), 0.3))
        want, wz, _ = L.run(x, BF16, bias, B.BL_ACT_RELU2, None, True)
        need = B.bitlinear_forward_epilogue_workspace_bytes(M, N, K, fmt, B.BL_BF16)
        buf = torch.full((3, 8192 + -(-max(need, 2 * M * N) // 256) * 256), 0xA5, dtype=torch.uint8, device="cuda")
        ws, y, z = buf[0, 4096:4096 + need], buf[1, 4096:4096 + 2 * M * N], buf[2, 4096:4096 + 2 * M * N]
        ws.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        s = torch.empty(M, device="cuda")
        B.bitlinear_forward_epilogue(L.packed, fmt, L.gamma, N, K, x, s, y.view(BF16).view(M, N), ws, bias=bias,
                                     act=B.BL_ACT_RELU2, preact=z.view(BF16).view(M, N), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y.view(BF16).view(M, N), want) and torch.equal(z.view(BF16).view(M, N), wz)
        for i, n in ((0, need), (1, 2 * M * N), (2, 2 * M * N)):
            assert (buf[i, :4096] == 0xA5).all() and (buf[i, 4096 + n:] == 0xA5).all()
        graphs, outs = [], []
        for _ in range(2):
            g, yo = torch.cuda.CUDAGraph(), torch.empty_like(want)
            with torch.cuda.graph(g):
                L.run(x, BF16, bias, B.BL_ACT_RELU2, None, False, y=yo, scale=s, ws=ws)
            graphs.append(g)
            outs.append(yo)
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        assert B.bitlinear_device_status(ws) == B.BL_OK


# ---- gradients through the epilogue ------------------------------------------------

def slope_error(z, act, fast):
    """Bound of the error of act'(z) as computed.  The fast exponential is within (2 + 1.2 |t|) 2^-22 of exp(t), the
    other within 2^-22; products and the divide add a few roundings (16u of the terms' size, 1 + |z|)."""
    e = (2 + 1.2 * torch.maximum(z.abs(), z * z / 2) if fast else 1.0) * 2.0 ** -22
    if act in (B.BL_ACT_NONE, B.BL_ACT_RELU):
        return torch.zeros_like(z)
    if act == B.BL_ACT_RELU2:
        return U * 2 * z.abs()
    return (e + 16 * U + 2 * U * z * z * (act == B.BL_ACT_GELU)) * (1 + z.abs()) + 2.0 ** -100


@pytest.mark.parametrize("M,N", [(1, 64), (1, 33), (7, 8), (64, 264), (250, 321), (700, 1000), (513, 4096), (3, 1)])
@pytest.mark.parametrize("act", ACTS)
def test_epilogue_backward(M, N, act):
    gen = torch.Generator(device="cuda").manual_seed(M * 1000 + N)
    z32 = torch.randn(M, N, generator=gen, device="cuda") * 3
    z32[torch.rand(M, N, generator=gen, device="cuda") < 0.05] = 0.0
    dy32 = torch.randn(M, N, generator=gen, device="cuda") * 1e-3
    for dydt, zdt in ((BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)):
        z, dy = z32.to(zdt), dy32.to(dydt)
        need = B.bitlinear_epilogue_backward_workspace_bytes(M, N)
        buf = torch.full((4096 + need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[4096:4096 + need]
        ws[:256] = 0
        dz, db = torch.full_like(dy, float("nan")), torch.full((N,), float("nan"), device="cuda")
        B.bitlinear_epilogue_backward(dy, z, act, dz, db, ws)
        torch.cuda.synchronize()
        assert (buf[:4096] == 0xA5).all() and (buf[4096 + need:] == 0xA5).all()
        z64, dy64 = z.double(), dy.double()
        want = dy64 * act64(z64, act)[1]
        err = dy64.abs() * slope_error(z64, act, dydt == BF16) + U * want.abs()
        h = half_step(dydt)
        check(dz, want, err * (1 + h) + h * want.abs() + 1e-38, "dz")
        # sums of M terms in any order: at most M additions, each within u of the magnitudes added so far
        check(db, want.sum(0), err.sum(0) + (M + 8) * U * (want.abs() + err).sum(0) + 1e-38, "dbias")
        # the parts alone and in place give the same bits
        dz2, db2 = torch.empty_like(dz), torch.empty_like(db)
        B.bitlinear_epilogue_backward(dy, z, act, dz2, None, ws)
        B.bitlinear_epilogue_backward(dy, z, act, None, db2, ws)
        assert torch.equal(dz2, dz) and torch.equal(db2, db)
        g = dy.clone()
        B.bitlinear_epilogue_backward(g, z if act else None, act, g, db2, ws)
        assert torch.equal(g, dz) and torch.equal(db2, db)


def test_epilogue_backward_against_differences():
    """dz against central differences of the activation in fp64 (step 1e-5: truncation below 1e-9 away from the kinks)."""
    z = torch.linspace(-6, 6, 4001, device="cuda")
    z = z[z.abs() > 1e-3][None].contiguous()
    dy = torch.ones_like(z)
    ws = torch.zeros(B.bitlinear_epilogue_backward_workspace_bytes(*z.shape), dtype=torch.uint8, device="cuda")
    for act in ACTS:
        dz = torch.empty_like(dy)
        B.bitlinear_epilogue_backward(dy, z, act, dz, None, ws)
        z64 = z.double()
        diff = (act64(z64 + 1e-5, act)[0] - act64(z64 - 1e-5, act)[0]) / 2e-5
        check(dz, diff, slope_error(z64, act, False) + 2 * U * diff.abs() + 1e-9, f"act {act}")


def test_empty_batch_gives_zero_sums():
    ws = torch.zeros(B.bitlinear_epilogue_backward_workspace_bytes(0, 40), dtype=torch.uint8, device="cuda")
    db = torch.full((40,), 7.0, device="cuda")
    e = torch.empty(0, 40, device="cuda")
    B.bitlinear_epilogue_backward(e, e, B.BL_ACT_SILU, None, db, ws)
    assert (db == 0).all()
