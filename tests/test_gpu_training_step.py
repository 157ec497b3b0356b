"""A block's end and the feed-forward part behind it, forward and backward through
the calls as a training step makes them: norms with gate and residual scale ->
INT8 codes -> product with SiLU (pre-activation kept) -> product with bias and
residual; then the gradients back to the block's output.

The reference runs the same formulas in fp64 from the stored inputs, without
the roundings between the calls.  Tolerance: each bf16 value on the way is off by
at most h = 2^-8 of itself, and these errors go through the following formulas
like the gradients do (e below).  dy1 = dx of the second product: e1 = (h + a)
|dy1|-wise, a = 2^-16 of the magnitudes for the fp32 runs; dz1 = dy1 act'(z1) with
z1 stored in bf16: |act'| <= 1.1, |act''| <= 1/2, so e2 = 1.1 e1 + |dy1| h |z1| / 2 +
h |dz1|; the first product adds e2 over its rows; the norm's gradient passes e3
on as r2 (w2 e3 + |n2| mean(w2 e3 |n2|))."""
import numpy as np
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B
from bitlinear_b1_fwd_b200 import synth
from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu

H = 2.0 ** -8
A = 2.0 ** -15
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


class Linear:
    def __init__(self, orc, N, K, seed):
        W = synth.normal_f32(seed, (N, K), 0.02)
        g = orc.gamma(W)
        codes = orc.ternarize(W, g, 1e-5)
        self.codes = torch.from_numpy(codes.astype(np.float64)).cuda()
        self.packed, self.gamma = dev(orc.pack(codes, B.BL_PACK_I2)), torch.tensor([float(g)], device="cuda")
        self.N, self.K = N, K

    def forward(self, x, ws, scale, **kw):
        y = torch.empty(x.shape[0], self.N, dtype=BF16, device="cuda")
        B.bitlinear_forward_epilogue(self.packed, B.BL_PACK_I2, self.gamma, self.N, self.K, x, scale, y, ws, **kw)
        return y

    def backward(self, dz, xq, s, ws):
        dx = torch.empty(dz.shape[0], self.K, dtype=BF16, device="cuda")
        dw = torch.empty(self.N, self.K, device="cuda")
        B.bitlinear_backward_dx_bf16(self.packed, B.BL_PACK_I2, self.gamma, self.N, self.K, dz, dx, ws)
        B.bitlinear_backward_dw_bf16(dz, xq, s, self.gamma, dw, ws)
        return dx, dw


class Step:
    def __init__(self, orc, M, K, F):
        self.M, self.K, self.F = M, K, F
        gen = torch.Generator(device="cuda").manual_seed(7 + M)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.up, self.down = Linear(orc, F, K, 31), Linear(orc, K, F, 32)
        self.b, self.r = (rnd(M, K) * 2).to(BF16), (rnd(M, K) * 2).to(BF16)
        self.w1, self.w2, self.gate = 1 + 0.2 * rnd(K), 1 + 0.2 * rnd(K), 0.5 + 0.2 * rnd(1, K)
        self.bias = 0.2 * rnd(K)
        self.dout = (rnd(M, K) * 1e-2).to(BF16)
        i2 = B.BL_PACK_I2
        need = max(B.bitlinear_forward_epilogue_workspace_bytes(M, F, K, i2, B.BL_I8),
                   B.bitlinear_forward_epilogue_workspace_bytes(M, K, F, i2, B.BL_BF16),
                   B.bitlinear_epilogue_backward_workspace_bytes(M, F),
                   B.bitlinear_backward_dx_bf16_workspace_bytes(M, F, K, i2),
                   B.bitlinear_backward_dx_bf16_workspace_bytes(M, K, F, i2),
                   B.bitlinear_backward_dw_bf16_workspace_bytes(M, F, K),
                   B.bitlinear_backward_dw_bf16_workspace_bytes(M, K, F),
                   B.bitlinear_residual_norm_backward_workspace_bytes(M, K))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.norm = dict(post=B.BL_NORM_RMS, post_w=self.w1, gate=self.gate, res_scale=0.9, branch_scale=0.7,
                         pre=B.BL_NORM_RMS, pre_w=self.w2)

    def run(self):
        M, K, F, ws = self.M, self.K, self.F, self.ws
        new = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        f32 = torch.float32
        h, xq, s = new(M, K), new(M, K, dt=torch.int8), new(M, dt=f32)
        B.bitlinear_residual_norm(self.b, self.r, h, xq=xq, scale=s, **self.norm)
        z1 = new(M, F)
        y1 = self.up.forward(xq, ws, s, act=B.BL_ACT_SILU, preact=z1)
        s2 = new(M, dt=f32)
        out = self.down.forward(y1, ws, s2, bias=self.bias, residual=h)
        xq2 = new(M, F, dt=torch.int8)
        B.bitlinear_quantize_acts(y1, xq2, s2)
        dbias = new(K, dt=f32)
        B.bitlinear_epilogue_backward(self.dout, None, B.BL_ACT_NONE, None, dbias, ws)
        dy1, dw_down = self.down.backward(self.dout, xq2, s2, ws)
        dz1 = new(M, F)
        B.bitlinear_epilogue_backward(dy1, z1, B.BL_ACT_SILU, dz1, None, ws)
        dxn, dw_up = self.up.backward(dz1, xq, s, ws)
        dr, db = new(M, K), new(M, K)
        g = dict(dpost_w=new(K, dt=f32), dgate=new(1, K, dt=f32), dpre_w=new(K, dt=f32))
        B.bitlinear_residual_norm_backward(dxn, self.dout, self.b, h, dr, db, ws, **self.norm, **g)
        return dict(h=h, z1=z1, y1=y1, out=out, xq=xq, s=s, dbias=dbias, dw_down=dw_down, dw_up=dw_up, dr=dr, db=db, **g)


@pytest.mark.parametrize("M,K,F", [(3, 128, 320), (40, 256, 512), (200, 320, 136), (70, 200, 328)])
def test_step(orc, M, K, F):
    step = Step(orc, M, K, F)
    o = step.run()
    torch.cuda.synchronize()
    assert B.bitlinear_device_status(step.ws) == B.BL_OK
    d = lambda t: t.double()  # noqa: E731
    g1, g2 = d(step.up.gamma), d(step.down.gamma)
    # forward, from the codes that the norm wrote
    z64 = (d(o["xq"]) @ step.up.codes.t()) * (g1 * d(o["s"])[:, None] / 127)
    assert ((d(o["z1"]) - z64).abs() <= (H + A) * z64.abs() + 1e-30).all()
    xq2, s2 = (torch.from_numpy(v).cuda() for v in step_act_quant(orc, o["y1"]))
    out64 = (d(xq2) @ step.down.codes.t()) * (g2 * d(s2)[:, None] / 127) + d(step.bias) + d(o["h"])
    size = (d(xq2) @ step.down.codes.t()).abs() * (g2 * d(s2)[:, None] / 127) + d(step.bias).abs() + d(o["h"]).abs()
    assert ((d(o["out"]) - out64).abs() <= H * out64.abs() + A * size).all()
    # backward
    dout = d(step.dout)
    dy1 = g2 * (dout @ step.down.codes)
    e1 = H * dy1.abs() + A * g2 * (dout.abs() @ step.down.codes.abs())
    sg = torch.sigmoid(z64)
    dz1 = dy1 * (sg + z64 * sg * (1 - sg))
    e2 = 1.1 * e1 + dy1.abs() * H * z64.abs() / 2 + (H + A) * (dz1.abs() + e1)
    dxn = g1 * (dz1 @ step.up.codes)
    e3 = g1 * (e2 @ step.up.codes.abs()) + H * dxn.abs() + A * g1 * (dz1.abs() @ step.up.codes.abs())
    e3 = e3 * (1 + H)
    h, b, w1, w2, gate = d(o["h"]), d(step.b), d(step.w1), d(step.w2), d(step.gate)
    r2 = (h.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    n2 = h * r2
    dn = dxn * w2
    dh = dout + r2 * (dn - n2 * (dn * n2).mean(1, keepdim=True))
    eh = r2 * (w2.abs() * e3 + n2.abs() * (w2.abs() * e3 * n2.abs()).mean(1, keepdim=True)) + A * (
        dout.abs() + r2 * (dn.abs() + n2.abs() * (dn * n2).abs().mean(1, keepdim=True)))
    rs, bs = float(np.float32(0.9)), float(np.float32(0.7))
    assert ((d(o["dr"]) - rs * dh).abs() <= (rs * eh) * (1 + H) + H * (rs * dh).abs()).all()
    r1 = (b.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    n1 = b * r1
    # sums over the tokens: errors add up
    want, tol = (bs * dh * n1 * w1).sum(0), (bs * (eh + A * dh.abs()) * n1.abs() * w1.abs()).sum(0)
    assert ((d(o["dgate"])[0] - want).abs() <= tol).all()
    want, tol = (bs * gate * dh * n1).sum(0), (bs * gate.abs() * (eh + A * dh.abs()) * n1.abs()).sum(0)
    assert ((d(o["dpost_w"]) - want).abs() <= tol).all()
    want, tol = (dxn * n2).sum(0), ((e3 + A * dxn.abs()) * n2.abs()).sum(0)
    assert ((d(o["dpre_w"]) - want).abs() <= tol).all()
    assert ((d(o["dbias"]) - dout.sum(0)).abs() <= A * dout.abs().sum(0)).all()
    x = d(o["xq"]) * d(o["s"])[:, None] / 127
    tol = g1 * ((e2 * (1 + H) + A * dz1.abs()).t() @ x.abs())
    assert ((d(o["dw_up"]) - g1 * (dz1.t() @ x)).abs() <= tol + 1e-30).all()
    x = d(xq2) * d(s2)[:, None] / 127
    assert ((d(o["dw_down"]) - g2 * (dout.t() @ x)).abs() <= A * g2 * (dout.abs().t() @ x.abs()) + 1e-30).all()
    # the whole step captured, on the same workspace, gives the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = step.run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in o:
        assert torch.equal(c[k], o[k]), k


def step_act_quant(orc, y):
    return orc.act_quant(host(y))
