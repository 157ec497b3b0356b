"""The norms around a block's end with its gate and residual scale, forward and
backward, against the formulas in fp64 (the gradients differentiated by torch).

Tolerances (u = 2^-24).  A sum over a row adds up to 64 terms per thread and 10
levels of a tree, so it is within 80u of its terms' magnitudes (rows longer than
the registers hold: K / 512 more per thread); the statistics and every later
step carry that through the formulas: see row_errors.  Stored values add half a
step of their type (2^-8 for bf16)."""
import numpy as np
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B
from gpu_helpers import host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
NONE, RMS, LAYER = B.BL_NORM_NONE, B.BL_NORM_RMS, B.BL_NORM_LAYER


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()
    assert torch.cuda.is_available()


def half_step(t):
    return 0.0 if t == F32 else torch.finfo(t).eps / 2


def unit64(v, kind, eps):
    if kind == NONE:
        return v, torch.ones_like(v[:, :1])
    if kind == LAYER:
        v = v - v.mean(1, keepdim=True)
    r = (v.square().mean(1, keepdim=True) + eps).rsqrt()
    return v * r, r


def unit_error(v, ev, kind, eps):
    """Error of the normalised rows, from errors ev of v: the mean's, the deviation's (relative, halved by the root),
    and the sums'."""
    if kind == NONE:
        return ev
    c = (80 + v.shape[1] / 512) * U
    n, r = unit64(v, kind, eps)
    if kind == LAYER:
        ev = ev + ev.mean(1, keepdim=True) + c * v.abs().mean(1, keepdim=True) + U * v.abs()
    rel = (n.abs() * ev * r).mean(1, keepdim=True) + c + 8 * U
    return r * ev + n.abs() * rel


class Case:
    def __init__(self, M, K, bdt, rdt, post, pre, gate_rows=0, bias=True, affine=True, seed=0, eps=1e-5, offset=0.2):
        gen = torch.Generator(device="cuda").manual_seed(seed + 31 * M + K)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.M, self.K, self.post, self.pre = M, K, post, pre
        self.b, self.r = (rnd(M, K) * 2 + offset).to(bdt), (rnd(M, K) * 3 - offset).to(rdt)
        self.w1, self.w2 = ((1 + 0.3 * rnd(K), 1 + 0.3 * rnd(K)) if affine else (None, None))
        self.b1, self.b2 = ((0.2 * rnd(K), 0.2 * rnd(K)) if bias else (None, None))
        self.gate_rows = gate_rows
        self.gate = 0.5 + 0.5 * rnd(-(-M // gate_rows), K) if gate_rows else None
        self.rs, self.bs, self.eps = 0.9, -0.7, eps
        self.dy, self.dh = (rnd(M, K) * 1e-2).to(bdt), (rnd(M, K) * 1e-2).to(rdt)

    def params(self):
        return dict(post=self.post, post_w=self.w1, post_b=self.b1, post_eps=self.eps, gate=self.gate,
                    gate_rows=self.gate_rows, res_scale=self.rs, branch_scale=self.bs, pre=self.pre, pre_w=self.w2,
                    pre_eps=self.eps)

    def rows(self, g):
        return 1.0 if g is None else g.repeat_interleave(self.gate_rows, 0)[:self.M]

    def forward64(self):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        w1, w2 = (1.0 if w is None else w.double() for w in (self.w1, self.w2))
        b1, b2 = (0.0 if w is None else w.double() for w in (self.b1, self.b2))
        b, r, g = self.b.double(), self.r.double(), self.rows(d(self.gate))
        f32 = lambda v: float(np.float32(v))  # noqa: E731  (the scalars are fp32)
        rs, bs = f32(self.rs), f32(self.bs)
        n1 = unit64(b, self.post, self.eps)[0]
        e1 = unit_error(b, torch.zeros_like(b), self.post, self.eps)
        u = n1 * w1 + b1
        h = rs * r + bs * g * u
        eh = abs(bs) * (abs(g) * (e1 * abs(w1) + 3 * U * (n1.abs() * abs(w1) + abs(b1)))) + 3 * U * (
            abs(rs) * r.abs() + (bs * g * u).abs())
        n2 = unit64(h, self.pre, self.eps)[0]
        e2 = unit_error(h, eh, self.pre, self.eps)
        y = n2 * w2 + b2
        ey = e2 * abs(w2) + 3 * U * ((n2 * w2).abs() + abs(b2))
        return h, eh, y, ey

    def run(self, ydt=F32, codes=False, want_h=True, stream=None):
        M, K = self.M, self.K
        h = torch.full_like(self.r, float("nan")) if want_h else None
        y = torch.full((M, K), float("nan"), dtype=ydt, device="cuda") if ydt else None
        xq = torch.full((M, K), 77, dtype=torch.int8, device="cuda") if codes else None
        s = torch.full((M,), -1.0, device="cuda") if codes else None
        B.bitlinear_residual_norm(self.b, self.r, h, pre_b=self.b2, y=y, xq=xq, scale=s, stream=stream, **self.params())
        return h, y, xq, s


def check(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {bad.nonzero()[:3].tolist()}, worst " \
                          f"{float(((got.double() - want).abs() / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


# widths: one column, odd, the 8-wide form at 1, 2 and 4 chunks, the scalar form at 4 and 16, rows longer than the
# registers hold; tokens from one to more than a wave of blocks
SHAPES = [(1, 1), (3, 7), (1, 3200), (5, 64), (33, 333), (700, 256), (9, 1001), (4, 2055), (6, 4104), (3, 8640),
          (2, 16384), (2, 8195), (3, 20000), (2500, 40)]
KINDS = [(RMS, RMS), (LAYER, LAYER), (NONE, RMS), (RMS, LAYER), (NONE, NONE), (LAYER, NONE)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("post,pre", KINDS)
def test_forward(M, K, post, pre):
    for i, (bdt, rdt) in enumerate(((BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16))):
        c = Case(M, K, bdt, rdt, post, pre, gate_rows=(0, M, 1, 3)[i], bias=i % 2 == 0, affine=i != 3, seed=i)
        h64, eh, y64, ey = c.forward64()
        h, y, _, _ = c.run(F32)
        check(h, h64, eh + half_step(rdt) * (h64.abs() + eh) + 1e-38, "h")
        check(y, y64, ey + 1e-38, "y")
        _, yb, _, _ = c.run(BF16, want_h=False)
        assert torch.equal(yb, y.to(BF16))


@pytest.mark.parametrize("M,K", SHAPES)
def test_codes_are_those_of_y(orc, M, K):
    """xq and scale equal the oracle's quantization of the fp32 y, bit for bit, with y stored or not."""
    c = Case(M, K, BF16, BF16, RMS, LAYER, gate_rows=max(1, M // 2), seed=5)
    _, y, xq, s = c.run(F32, codes=True)
    xq_ref, s_ref = orc.act_quant(host(y))
    assert np.array_equal(host(s), s_ref) and np.array_equal(host(xq), xq_ref)
    h, _, xq2, s2 = c.run(None, codes=True)
    assert torch.equal(xq2, xq) and torch.equal(s2, s)


def test_special_rows():
    """Zero rows (eps keeps them finite and the codes 0), a large common offset, tiny and large values."""
    for K in (64, 333, 20000):
        c = Case(4, K, F32, F32, LAYER, LAYER, seed=7)
        c.b[0] = 0
        c.r[0] = 0
        c.b[1] = 1000 + torch.randn(K, device="cuda")
        c.b[2] *= 1e-12
        c.r[3] *= 1e6
        h64, eh, y64, ey = c.forward64()
        h, y, _, _ = c.run(F32)
        check(h, h64, eh + 1e-38, "h")
        check(y, y64, ey + 1e-38, "y")
    z = torch.zeros(2, 64, device="cuda")
    h, xq, s = torch.empty_like(z), torch.empty(2, 64, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    B.bitlinear_residual_norm(z, z, h, post=RMS, pre=RMS, xq=xq, scale=s)
    assert (h == 0).all() and (xq == 0).all() and (s == float(np.float32(1e-6))).all()


def test_a_token_alone_and_in_a_batch():
    c = Case(600, 320, BF16, F32, RMS, RMS, seed=9)
    h, y, _, _ = c.run(F32)
    for m in (0, 17, 599):
        one = Case(1, 320, BF16, F32, RMS, RMS, seed=9)
        for k in ("w1", "w2", "b1", "b2"):
            setattr(one, k, getattr(c, k))
        one.b, one.r = c.b[m:m + 1].contiguous(), c.r[m:m + 1].contiguous()
        h1, y1, _, _ = one.run(F32)
        assert torch.equal(h1[0], h[m]) and torch.equal(y1[0], y[m])


@pytest.mark.parametrize("K", [320, 333, 20000])
def test_in_place_and_layout(K):
    """h over r; a [K] gate; vectors at a 4-byte offset."""
    c = Case(5, K, BF16, BF16, RMS, RMS, gate_rows=5, seed=11)
    h, y, _, _ = c.run(F32)
    r, y2 = c.r.clone(), torch.empty_like(y)
    p = c.params()
    p["gate"], p["gate_rows"] = c.gate[0], 0
    for k in ("post_w", "pre_w", "post_b", "gate"):
        p[k] = torch.cat([p[k][:1], p[k]])[1:]
    b2 = torch.cat([c.b2[:1], c.b2])[1:]
    B.bitlinear_residual_norm(c.b, r, r, pre_b=b2, y=y2, **p)
    assert torch.equal(r, h) and torch.equal(y2, y)


# ---- backward ------------------------------------------------------------------------

class Grads:
    """Gradients in fp64: the pre norm sees h as stored."""

    def __init__(self, c, h):
        leaf = {k: getattr(c, k).double().requires_grad_(True) for k in ("b", "r", "w1", "b1", "w2", "b2", "gate")
                if getattr(c, k) is not None}
        self.b, self.h = leaf["b"], h.double().requires_grad_(True)
        f32 = lambda v: float(np.float32(v))  # noqa: E731
        n1, r1 = unit64(leaf["b"], c.post, c.eps)
        u = n1 * leaf.get("w1", 1.0) + leaf.get("b1", 0.0)
        g = c.rows(leaf.get("gate"))
        ht = f32(c.rs) * leaf["r"] + f32(c.bs) * g * u
        n2, r2 = unit64(self.h, c.pre, c.eps)
        y = n2 * leaf.get("w2", 1.0) + leaf.get("b2", 0.0)
        y.backward(c.dy.double())
        self.dh = self.h.grad + c.dh.double()
        ht.backward(self.dh)
        self.grad = {k: v.grad for k, v in leaf.items()}
        # error bounds
        K, cc = c.K, (80 + c.K / 512) * U
        with torch.no_grad():
            zero = torch.zeros_like(n1)
            e1 = unit_error(leaf["b"], zero, c.post, c.eps)
            e2 = unit_error(self.h, zero, c.pre, c.eps)
            w1, w2 = (leaf.get(k, torch.ones(K, device="cuda").double()).abs() for k in ("w1", "w2"))

            def through(dn, edn, n, en, r, kind):
                """r (dn - mean dn - n mean(dn n)): its error from dn's and n's."""
                if kind == NONE:
                    return edn
                m = lambda v: v.mean(1, keepdim=True)  # noqa: E731
                t = edn + m(edn) + cc * m(dn.abs())
                q = m(dn.abs() * n.abs())
                t = t + en * q + n.abs() * (m(edn * n.abs() + dn.abs() * en) + cc * q)
                size = dn.abs() + m(dn.abs()) + n.abs() * q
                rel = cc + 8 * U + m(n.abs() * en)
                return r * (t + (rel + 4 * U) * size)

            dy = c.dy.double().abs()
            edh = through(dy * w2, U * dy * w2, n2, e2, r2, c.pre) + 2 * U * self.dh.abs()
            gg = g.abs() if torch.is_tensor(g) else 1.0
            bs = abs(c.bs)
            ua = u.abs()
            eu = e1 * w1 + 3 * U * (n1.abs() * w1 + (leaf["b1"].abs() if "b1" in leaf else 0.0))
            du = bs * gg * self.dh.abs()
            edu = bs * gg * edh + 3 * U * du
            rows = (c.M + 16) * U
            self.tol = dict(
                r=abs(c.rs) * edh + 2 * U * self.grad["r"].abs(),
                b=through(du * w1, edu * w1 + U * du * w1, n1, e1, r1, c.post),
                w2=(dy * e2 + (rows + U) * dy * (n2.abs() + e2)).sum(0), b2=(rows * dy).sum(0),
                w1=(edu * n1.abs() + du * e1 + rows * (du + edu) * (n1.abs() + e1)).sum(0),
                b1=(edu + rows * (du + edu)).sum(0))
            eg = bs * (edh * ua + self.dh.abs() * eu + (rows + 3 * U) * (self.dh.abs() + edh) * (ua + eu))
            if c.gate is not None:
                n = c.gate.shape[0]
                pad = torch.zeros(n * c.gate_rows - c.M, K, device="cuda").double()
                self.tol["gate"] = torch.cat([eg, pad]).view(n, c.gate_rows, K).sum(1)


def backward(c, h, which=("b", "r", "w1", "b1", "w2", "b2", "gate"), dh=True, ws=None, stream=None, **over):
    M, K = c.M, c.K
    vec = lambda k: torch.full((K,), float("nan"), device="cuda") if k in which else None  # noqa: E731
    o = dict(b=torch.full_like(c.b, float("nan")) if "b" in which else None,
             r=torch.full_like(c.r, float("nan")) if "r" in which else None,
             w1=vec("w1"), b1=vec("b1"), w2=vec("w2"), b2=vec("b2"),
             gate=torch.full_like(c.gate, float("nan")) if c.gate is not None and "gate" in which else None)
    o.update(over)
    if ws is None:
        ws = torch.zeros(B.bitlinear_residual_norm_backward_workspace_bytes(M, K, c.gate_rows), dtype=torch.uint8,
                         device="cuda")
    B.bitlinear_residual_norm_backward(c.dy, c.dh if dh else None, c.b, h, o["r"], o["b"], ws, dpost_w=o["w1"],
                                       dpost_b=o["b1"], dgate=o["gate"], dpre_w=o["w2"], dpre_b=o["b2"], stream=stream,
                                       **c.params())
    return o


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("post,pre", KINDS)
def test_backward(M, K, post, pre):
    for i, (bdt, rdt) in enumerate(((BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16))):
        c = Case(M, K, bdt, rdt, post, pre, gate_rows=(M, 0, 1, 3)[i], bias=i % 2 == 0, affine=i != 3, seed=20 + i)
        h = c.run(None)[0]
        want = Grads(c, h)
        got = backward(c, h)
        for k, g in want.grad.items():
            t = want.tol[k] + 1e-38
            hs = half_step(got[k].dtype)
            check(got[k], g, t * (1 + hs) + hs * g.abs(), f"d{k} ({bdt}, {rdt})")
        # the same bits again, and from calls that want only some of them
        again = backward(c, h)
        some = backward(c, h, which=("b", "w2", "gate"))
        for k in want.grad:
            assert torch.equal(again[k], got[k]), k
            if some[k] is not None:
                assert torch.equal(some[k], got[k]), k


@pytest.mark.parametrize("K", [2944, 3001, 4000, 5000, 7000, 8704, 9208])
def test_widths_at_the_limits_of_shared_memory(K):
    """Rows whose column vectors take about 48 KB (with and without a bias), and the longest that stay in registers."""
    for bias in (True, False):
        c = Case(5, K, BF16, BF16, RMS, LAYER, gate_rows=2, bias=bias, seed=30)
        h64, eh, y64, ey = c.forward64()
        h, y, _, _ = c.run(F32)
        check(h, h64, eh + half_step(BF16) * (h64.abs() + eh) + 1e-38, "h")
        check(y, y64, ey + 1e-38, "y")
        want, got = Grads(c, h), backward(c, h)
        for k, g in want.grad.items():
            hs = half_step(got[k].dtype)
            check(got[k], g, (want.tol[k] + 1e-38) * (1 + hs) + hs * g.abs(), f"d{k}")


@pytest.mark.parametrize("M,K,gate_rows", [(1000, 64, 7), (301, 136, 301), (149, 48, 2), (148, 33, 148), (450, 20008, 100)])
def test_gate_rows_and_blocks_of_tokens(M, K, gate_rows):
    """Runs of tokens with one gate row that begin and end inside blocks of tokens."""
    c = Case(M, K, F32, F32, RMS, RMS, gate_rows=gate_rows, seed=40)
    h = c.run(None)[0]
    want, got = Grads(c, h), backward(c, h)
    check(got["gate"], want.grad["gate"], want.tol["gate"] + 1e-38, "dgate")


def test_backward_against_differences():
    """The inner product of the gradients with a direction against central differences of the fp64 formula (step 1e-5:
    truncation and cancellation below 1e-7 of sum |gradient direction|)."""
    c = Case(6, 96, F32, F32, LAYER, RMS, gate_rows=4, seed=50)
    h = c.run(None)[0]
    got = backward(c, h)
    want = Grads(c, h)
    gen = torch.Generator(device="cuda").manual_seed(51)
    cy, ch = c.dy.double(), c.dh.double()
    for k in ("b", "r", "w1", "b1", "w2", "b2", "gate"):
        base = getattr(c, k)
        v = torch.randn(base.shape, generator=gen, device="cuda")
        loss = []
        for sgn in (1, -1):
            setattr(c, k, base.double() + sgn * 1e-5 * v.double())
            h64, _, y64, _ = c.forward64()
            loss.append(float((y64 * cy).sum() + (h64 * ch).sum()))
        setattr(c, k, base)
        diff = (loss[0] - loss[1]) / 2e-5
        dot = float((got[k].double() * v.double()).sum())
        # h as stored (fp32) is within 2^-24 of the formula's: a relative change of the gradients of a few 2^-24
        tol = float((want.tol[k] * v.double().abs()).sum()) + (1e-7 + 64 * U) * float((got[k].double() * v.double()).abs().sum())
        assert abs(diff - dot) <= tol, (k, diff, dot, tol)


@pytest.mark.parametrize("K", [320, 333, 20000])
def test_backward_in_place_and_without_dh(K):
    c = Case(7, K, BF16, BF16, RMS, RMS, gate_rows=7, seed=60)
    h = c.run(None)[0]
    got = backward(c, h)
    dy, dh = c.dy.clone(), c.dh.clone()
    keep = (c.dy, c.dh)
    c.dy, c.dh = dy, dh
    backward(c, h, r=dh, b=dy)
    assert torch.equal(dh, got["r"]) and torch.equal(dy, got["b"])
    c.dy, c.dh = keep[0], torch.zeros_like(keep[1])
    a, b = backward(c, h), backward(c, h, dh=False)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_guards_streams_and_graphs():
    for M, K in ((3, 333), (20, 320), (2, 20008)):
        c = Case(M, K, BF16, BF16, RMS, LAYER, gate_rows=2, seed=70)
        h, y, xq, s = c.run(BF16, codes=True)
        want = backward(c, h)
        need = B.bitlinear_residual_norm_backward_workspace_bytes(M, K, 2)
        n = 2 * M * K
        buf = torch.full((4, 8192 + -(-max(need, n) // 256) * 256), 0xA5, dtype=torch.uint8, device="cuda")
        ws = buf[0, 4096:4096 + need]
        ws[:256] = 0
        out = [buf[i, 4096:4096 + n].view(BF16).view(M, K) for i in (1, 2)]
        q = buf[3, 4096:4096 + M * K].view(torch.int8).view(M, K)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = backward(c, h, ws=ws, stream=side, r=out[0], b=out[1])
        s2, h2 = torch.empty_like(s), torch.empty_like(h)
        B.bitlinear_residual_norm(c.b, c.r, h2, pre_b=c.b2, xq=q, scale=s2, stream=side, **c.params())
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert torch.equal(q, xq) and torch.equal(s2, s) and torch.equal(h2, h)
        for i, k in ((0, need), (1, n), (2, n), (3, M * K)):
            assert (buf[i, :4096] == 0xA5).all() and (buf[i, 4096 + k:] == 0xA5).all()
        graphs, outs = [], []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            o = {k: torch.empty_like(v) for k, v in want.items()}
            with torch.cuda.graph(g):
                backward(c, h, ws=ws, **o)
            graphs.append(g)
            outs.append(o)
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], want[k]) for o in outs for k in want)


def test_empty_batch():
    e = torch.empty(0, 48, device="cuda")
    ws = torch.zeros(B.bitlinear_residual_norm_backward_workspace_bytes(0, 48), dtype=torch.uint8, device="cuda")
    w = torch.full((48,), 3.0, device="cuda")
    B.bitlinear_residual_norm(e, e, e.clone())
    B.bitlinear_residual_norm_backward(e, None, e, e, e.clone(), e.clone(), ws, dpre_w=w)
    assert (w == 0).all()


def test_empty_batch_shared_gate():
    """No token: the gradient of a gate row shared by all tokens is zero, not what the buffer held."""
    e, gate = torch.empty(0, 48, device="cuda"), torch.ones(48, device="cuda")
    ws = torch.zeros(B.bitlinear_residual_norm_backward_workspace_bytes(0, 48), dtype=torch.uint8, device="cuda")
    dgate = torch.full((48,), 3.0, device="cuda")
    B.bitlinear_residual_norm_backward(e, None, e, e, e.clone(), e.clone(), ws, gate=gate, dgate=dgate)
    assert (dgate == 0).all()
