"""Cases of the operators around the BitLinear product, for measurement.

Four groups of calls, each with its plain form in elementary torch operations:

  forward        bitlinear_forward_epilogue: the ternary x INT8 product with
                 bias, activation and residual in its epilogue
  act_grad       bitlinear_epilogue_backward: the gradients through that
                 epilogue (of the pre-activation and of the bias)
  products       bitlinear_backward_dx_bf16 and bitlinear_backward_dw_bf16: the
                 two gradient products of a bf16 gradient
  norm, norm_grad  bitlinear_residual_norm and its backward: the norm after a
                 block, its gate and residual scale, and the norm before the
                 next block, with the INT8 codes for the next product

``own`` selects between the plain form and the library's calls.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PER = {"i2": 4, "t5": 5, "b1": 8}      # weights per packed byte


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token through a 3B up-projection: latency
        dict(name="forward_1x3200x8640", op="forward", M=1, K=3200, N=8640, fmt="i2", xdt="bf16", ydt="bf16",
             act="relu2", bias=True, res=False, pre=False),
        # a small decode batch through the down-projection, added to the residual stream
        dict(name="forward_16x8640x3200_res", op="forward", M=16, K=8640, N=3200, fmt="t5", xdt="bf16", ydt="bf16",
             act="none", bias=True, res=True, pre=False),
        # training forward: 4096 tokens, the pre-activation kept for the backward pass
        dict(name="forward_4096x3200x8640_pre", op="forward", M=4096, K=3200, N=8640, fmt="i2", xdt="bf16",
             ydt="bf16", act="silu", bias=True, res=False, pre=True),
        # ragged: 1-bit weights, an odd K, fp32 in and out
        dict(name="forward_37x1011x777_f32", op="forward", M=37, K=1011, N=777, fmt="b1", xdt="f32", ydt="f32",
             act="gelu", bias=True, res=True, pre=False),
        # the epilogue's gradient for that training step
        dict(name="act_grad_4096x8640", op="act_grad", M=4096, N=8640, dt="bf16", act="silu"),
        # a short fp32 batch with an odd width
        dict(name="act_grad_250x3201_f32", op="act_grad", M=250, N=3201, dt="f32", act="relu2"),
        # the two gradient products of that training step
        dict(name="products_4096x3200x8640", op="products", M=4096, K=3200, N=8640, fmt="i2", dxdt="bf16"),
        # a short sequence through a square projection
        dict(name="products_130x3200x3200", op="products", M=130, K=3200, N=3200, fmt="i2", dxdt="bf16"),
        # one decoded token between two blocks
        dict(name="norm_1x3200", op="norm", M=1, K=3200, dt="bf16", post="rms", pre="rms", gate_rows=0, bias=False,
             out="y"),
        # prefill or training: codes straight for the next product
        dict(name="norm_4096x3200_codes", op="norm", M=4096, K=3200, dt="bf16", post="rms", pre="rms", gate_rows=4096,
             bias=False, out="codes"),
        # its gradient, a learned gate shared by every token
        dict(name="norm_grad_4096x3200", op="norm_grad", M=4096, K=3200, dt="bf16", post="rms", pre="rms",
             gate_rows=4096, bias=False),
        # LayerNorms with bias, one gate row for every 100 tokens, an odd width, fp32
        dict(name="norm_grad_333x1001_f32", op="norm_grad", M=333, K=1001, dt="f32", post="layer", pre="layer",
             gate_rows=100, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "act_grad", "products", "norm", "norm_grad"])
    if op in ("forward", "products"):
        while True:
            M, K, N = _log(rng, 1, 4096), _log(rng, 48, 8640), _log(rng, 48, 8640)
            if rng.random() < 0.6:      # hidden sizes are mostly multiples of 64
                K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
            if M * K * N <= 4096 * 3200 * 8640:
                break
        fmt = rng.choice(["i2", "i2", "t5", "b1"])
        if op == "products":
            return dict(op=op, M=M, K=K, N=N, fmt=fmt, dxdt=rng.choice(["bf16", "f32"]))
        return dict(op=op, M=M, K=K, N=N, fmt=fmt, xdt=rng.choice(["bf16", "f32"]), ydt=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["none", "relu", "relu2", "silu", "gelu"]), bias=rng.random() < 0.7,
                    res=rng.random() < 0.5, pre=rng.random() < 0.4)
    if op == "act_grad":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 48, 8640), dt=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["relu", "relu2", "silu", "gelu"]))
    M, K = _log(rng, 1, 4096), _log(rng, 48, 8640)
    while M * K > 4096 * 3200:
        M //= 2
    post = rng.choice(["none", "rms", "layer"])
    case = dict(op=op, M=M, K=K, dt=rng.choice(["bf16", "f32"]), post=post, pre=rng.choice(["rms", "layer"]),
                gate_rows=rng.choice([0, M, max(1, M // 3)]), bias=rng.random() < 0.5)
    if op == "norm":
        case["out"] = rng.choice(["y", "codes"])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pack(codes, fmt):
    """Packed rows (16-byte multiples) of int codes [N, K]."""
    N, K = codes.shape
    per = PER[fmt]
    rb = (-(-K // per) + 15) // 16 * 16
    pad, base, shift = (0, 2, 0) if fmt == "b1" else (1, 4 if fmt == "i2" else 3, 1)
    d = torch.full((N, rb * per), pad, dtype=torch.int32, device=codes.device)
    d[:, :K] = (codes > 0).int() if fmt == "b1" else codes.int() + shift
    w = torch.tensor([base ** i for i in range(per)], dtype=torch.int32, device=codes.device)
    return (d.view(N, rb, per) * w).sum(-1).to(torch.uint8)


def _weights(N, K, fmt, gen):
    """gamma (or beta) and the packed codes of a latent N(0, 0.02) matrix."""
    W = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    gamma = W.abs().mean(dtype=torch.float64).to(torch.float32).reshape(1)
    if fmt == "b1":
        codes = torch.where(W > W.mean(dtype=torch.float64).to(torch.float32), 1, -1)
    else:
        codes = (W / (gamma + 1e-5)).round().clamp(-1, 1)
    return gamma, _pack(codes.to(torch.int8), fmt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st, M = dict(case=dict(case)), case["M"]
    if case["op"] == "forward":
        N, K = case["N"], case["K"]
        st["gamma"], st["packed"] = _weights(N, K, case["fmt"], gen)
        x = rnd(M, K)
        x[:, torch.rand(K, generator=gen, device="cuda") < 0.005] *= 30.0   # outlier channels
        st["x"] = x.to(DT[case["xdt"]])
        st["bias"] = rnd(N) * 0.2 if case["bias"] else None
        st["res"] = rnd(M, N).to(DT[case["ydt"]]) if case["res"] else None
    elif case["op"] == "act_grad":
        N, dt = case["N"], DT[case["dt"]]
        st["z"], st["dy"] = (rnd(M, N) * 1.5).to(dt), (rnd(M, N) * 1e-3).to(dt)
    elif case["op"] == "products":
        N, K = case["N"], case["K"]
        st["gamma"], st["packed"] = _weights(N, K, case["fmt"], gen)
        st["dz"] = (rnd(M, N) * 1e-3 * (0.25 + 2 * torch.rand(M, 1, generator=gen, device="cuda"))).to(torch.bfloat16)
        x = rnd(M, K) * (0.5 + torch.rand(M, 1, generator=gen, device="cuda"))
        st["scale"] = x.abs().amax(1).clamp_min(1e-6)
        st["xq"] = (x / st["scale"][:, None] * 127).round().clamp(-127, 127).to(torch.int8)
    else:
        K, dt, g = case["K"], DT[case["dt"]], case["gate_rows"]
        st["b"], st["r"] = (rnd(M, K) * 3 + 0.1).to(dt), (rnd(M, K) * 2).to(dt)
        vec = lambda mean, dev: mean + dev * rnd(K)  # noqa: E731
        affine1, affine2 = (vec(1, 0.2), vec(0, 0.1)), (vec(1, 0.2), vec(0, 0.1))
        st["w1"] = affine1[0] if case["post"] != "none" else None
        st["b1"] = affine1[1] if case["post"] != "none" and case["bias"] else None
        st["w2"], st["b2"] = affine2[0], affine2[1] if case["bias"] else None
        st["gate"] = 0.5 + 0.3 * rnd(-(-M // g), K) if g else None
        st["rs"], st["bs"], st["eps1"], st["eps2"] = 0.9, 0.6, 1e-5, 1e-6
        if case["op"] == "norm_grad":
            u = _unit(st["b"].double(), case["post"], st["eps1"])[0]
            h = _affine(u, st["w1"], st["b1"]) * st["bs"] * _rows(st["gate"], g, M) + st["rs"] * st["r"].double()
            st["h"] = h.to(dt)              # as the forward stored it
            st["dy"], st["dh"] = (rnd(M, K) * 1e-3).to(dt), (rnd(M, K) * 1e-3).to(dt)
    return st


# ---------------------------------------------------------------------------
# the plain form: elementary operations in 32 bits, rounded once at the end
# ---------------------------------------------------------------------------

def _codes(packed, K, fmt):
    """Codes [N, K] of packed rows, as fp32."""
    p = packed.int()[:, :, None]
    i = torch.arange(PER[fmt], device=p.device, dtype=torch.int32)
    if fmt == "i2":
        c = ((p >> (2 * i)) & 3) - 1
    elif fmt == "t5":
        c = (p // 3 ** i) % 3 - 1
    else:
        c = ((p >> i) & 1) * 2 - 1
    return c.view(packed.shape[0], -1)[:, :K].float()


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "relu2":
        return z.clamp_min(0) ** 2
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * z.clamp_min(0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _unit(v, kind, eps):
    """The normalised rows of v and 1 / their deviation."""
    if kind == "none":
        return v, None
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return v * r, r


def _affine(v, w, b):
    v = v if w is None else v * w
    return v if b is None else v + b


def _rows(gate, g, M):
    """The gate's row of each of M tokens."""
    return 1.0 if gate is None else gate[torch.arange(M, device=gate.device) // g]


def _quantized(v):
    """Per-token absmax INT8 of v as the values the codes stand for."""
    s = v.abs().amax(-1, keepdim=True).clamp_min(1e-6)
    return (v / s * 127).round().clamp(-127, 127) * s / 127


def _plain_forward(st, c):
    x = st["x"].float()
    s = x.abs().amax(-1, keepdim=True).clamp_min(1e-6)
    q = (x / s * 127).round().clamp(-127, 127)
    z = (q @ _codes(st["packed"], c["K"], c["fmt"]).t()) * (st["gamma"] * s / 127)
    z = z if st["bias"] is None else z + st["bias"]
    y = _act(z, c["act"])
    y = y if st["res"] is None else y + st["res"].float()
    out = dict(y=y.to(DT[c["ydt"]]))
    if c["pre"]:
        out["z"] = z.to(DT[c["ydt"]])
    return out


def _plain_act_grad(st, c):
    dz = st["dy"].float() * _act_slope(st["z"].float(), c["act"])
    return dict(dz=dz.to(DT[c["dt"]]), dbias=dz.sum(0))


def _plain_products(st, c):
    dz, gamma = st["dz"].float(), st["gamma"]
    dx = gamma * (dz @ _codes(st["packed"], c["K"], c["fmt"]))
    dw = gamma * (dz.t() @ (st["xq"].float() * (st["scale"][:, None] / 127)))
    return dict(dx=dx.to(DT[c["dxdt"]]), dw=dw)


def _plain_norm(st, c):
    dt = DT[c["dt"]]
    u = _affine(_unit(st["b"].float(), c["post"], st["eps1"])[0], st["w1"], st["b1"])
    h = st["rs"] * st["r"].float() + st["bs"] * _rows(st["gate"], c["gate_rows"], c["M"]) * u
    y = _affine(_unit(h, c["pre"], st["eps2"])[0], st["w2"], st["b2"])
    if c["out"] == "codes":
        return dict(h=h.to(dt), codes=_quantized(y).to(torch.bfloat16))
    return dict(h=h.to(dt), y=y.to(dt))


def _unit_grad(dn, n, r, kind):
    if kind == "none":
        return dn
    mean = dn.mean(-1, keepdim=True) if kind == "layer" else 0
    return r * (dn - mean - n * (dn * n).mean(-1, keepdim=True))


def _gate_sum(v, g, M):
    """Sums of v's rows over the tokens of each gate row."""
    n = -(-M // g)
    pad = torch.zeros(n * g - M, v.shape[1], dtype=v.dtype, device=v.device)
    return torch.cat([v, pad]).view(n, g, -1).sum(1)


def _plain_norm_grad(st, c):
    dt, M, g = DT[c["dt"]], c["M"], c["gate_rows"]
    dy = st["dy"].float()
    n2, r2 = _unit(st["h"].float(), c["pre"], st["eps2"])
    dh = st["dh"].float() + _unit_grad(dy * st["w2"], n2, r2, c["pre"])
    n1, r1 = _unit(st["b"].float(), c["post"], st["eps1"])
    du = st["bs"] * _rows(st["gate"], g, M) * dh
    dn1 = du if st["w1"] is None else du * st["w1"]
    out = dict(dr=(st["rs"] * dh).to(dt), db=_unit_grad(dn1, n1, r1, c["post"]).to(dt), dw2=(dy * n2).sum(0))
    if c["bias"]:
        out["db2"] = dy.sum(0)
    if st["gate"] is not None:
        out["dgate"] = _gate_sum(st["bs"] * dh * _affine(n1, st["w1"], st["b1"]), g, M)
    if st["w1"] is not None:
        out["dw1"] = (du * n1).sum(0)
    if st["b1"] is not None:
        out["db1"] = du.sum(0)
    return out


# ---------------------------------------------------------------------------
# the library's calls (outputs and workspaces are the caller's, kept in the state)
# ---------------------------------------------------------------------------

def _own_forward(st, c):
    from bitlinear_b1_fwd_b200 import binding as bl
    M, N, K = c["M"], c["N"], c["K"]
    if "ws" not in st:
        fmt = dict(i2=bl.BL_PACK_I2, t5=bl.BL_PACK_T5, b1=bl.BL_PACK_B1)[c["fmt"]]
        act = dict(none=bl.BL_ACT_NONE, relu=bl.BL_ACT_RELU, relu2=bl.BL_ACT_RELU2, silu=bl.BL_ACT_SILU,
                   gelu=bl.BL_ACT_GELU)[c["act"]]
        need = bl.bitlinear_forward_epilogue_workspace_bytes(M, N, K, fmt, bl.dtype_code(st["x"]))
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        st["scale"] = torch.empty(M, device="cuda")
        st["y"] = torch.empty(M, N, dtype=DT[c["ydt"]], device="cuda")
        st["z"] = torch.empty_like(st["y"]) if c["pre"] else None
        st["fmt"], st["act"] = fmt, act
    bl.bitlinear_forward_epilogue(st["packed"], st["fmt"], st["gamma"], N, K, st["x"], st["scale"], st["y"], st["ws"],
                                  bias=st["bias"], act=st["act"], residual=st["res"], preact=st["z"])
    return dict(y=st["y"], z=st["z"]) if c["pre"] else dict(y=st["y"])


def _own_act_grad(st, c):
    from bitlinear_b1_fwd_b200 import binding as bl
    if "ws" not in st:
        st["act"] = dict(relu=bl.BL_ACT_RELU, relu2=bl.BL_ACT_RELU2, silu=bl.BL_ACT_SILU, gelu=bl.BL_ACT_GELU)[c["act"]]
        st["ws"] = torch.zeros(bl.bitlinear_epilogue_backward_workspace_bytes(c["M"], c["N"]), dtype=torch.uint8,
                               device="cuda")
        st["dz"], st["dbias"] = torch.empty_like(st["dy"]), torch.empty(c["N"], device="cuda")
    bl.bitlinear_epilogue_backward(st["dy"], st["z"], st["act"], st["dz"], st["dbias"], st["ws"])
    return dict(dz=st["dz"], dbias=st["dbias"])


def _own_products(st, c):
    from bitlinear_b1_fwd_b200 import binding as bl
    M, N, K = c["M"], c["N"], c["K"]
    if "ws" not in st:
        st["fmt"] = dict(i2=bl.BL_PACK_I2, t5=bl.BL_PACK_T5, b1=bl.BL_PACK_B1)[c["fmt"]]
        need = max(bl.bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, st["fmt"]),
                   bl.bitlinear_backward_dw_bf16_workspace_bytes(M, N, K))
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        st["dx"] = torch.empty(M, K, dtype=DT[c["dxdt"]], device="cuda")
        st["dw"] = torch.empty(N, K, device="cuda")
    bl.bitlinear_backward_dx_bf16(st["packed"], st["fmt"], st["gamma"], N, K, st["dz"], st["dx"], st["ws"])
    bl.bitlinear_backward_dw_bf16(st["dz"], st["xq"], st["scale"], st["gamma"], st["dw"], st["ws"])
    return dict(dx=st["dx"], dw=st["dw"])


def _own_norm(st, c):
    from bitlinear_b1_fwd_b200 import binding as bl
    kind = dict(none=bl.BL_NORM_NONE, rms=bl.BL_NORM_RMS, layer=bl.BL_NORM_LAYER)
    codes = c["out"] == "codes"
    if "ho" not in st:
        st["ho"] = torch.empty_like(st["r"])
        st["y"] = None if codes else torch.empty_like(st["r"])
        st["xq"] = torch.empty(st["r"].shape, dtype=torch.int8, device="cuda") if codes else None
        st["scale"] = torch.empty(c["M"], device="cuda") if codes else None
        st["values"] = torch.empty(st["r"].shape, dtype=torch.bfloat16, device="cuda") if codes else None
    bl.bitlinear_residual_norm(st["b"], st["r"], st["ho"], post=kind[c["post"]], post_w=st["w1"], post_b=st["b1"],
                               post_eps=st["eps1"], gate=st["gate"], gate_rows=c["gate_rows"], res_scale=st["rs"],
                               branch_scale=st["bs"], pre=kind[c["pre"]], pre_w=st["w2"], pre_b=st["b2"],
                               pre_eps=st["eps2"], y=st["y"], xq=st["xq"], scale=st["scale"])
    if codes:
        return dict(h=st["ho"], codes=torch.mul(st["xq"], (st["scale"] / 127)[:, None], out=st["values"]))
    return dict(h=st["ho"], y=st["y"])


def _own_norm_grad(st, c):
    from bitlinear_b1_fwd_b200 import binding as bl
    kind = dict(none=bl.BL_NORM_NONE, rms=bl.BL_NORM_RMS, layer=bl.BL_NORM_LAYER)
    M, K, g = c["M"], c["K"], c["gate_rows"]
    if "ws" not in st:
        st["ws"] = torch.zeros(bl.bitlinear_residual_norm_backward_workspace_bytes(M, K, g), dtype=torch.uint8,
                               device="cuda")
        vec = lambda on: torch.empty(K, device="cuda") if on else None  # noqa: E731
        st["out"] = dict(dr=torch.empty_like(st["r"]), db=torch.empty_like(st["b"]), dw2=vec(True), db2=vec(c["bias"]),
                         dgate=None if st["gate"] is None else torch.empty_like(st["gate"]),
                         dw1=vec(st["w1"] is not None), db1=vec(st["b1"] is not None))
    o = st["out"]
    bl.bitlinear_residual_norm_backward(st["dy"], st["dh"], st["b"], st["h"], o["dr"], o["db"], st["ws"],
                                        post=kind[c["post"]], post_w=st["w1"], post_b=st["b1"], post_eps=st["eps1"],
                                        gate=st["gate"], gate_rows=g, res_scale=st["rs"], branch_scale=st["bs"],
                                        pre=kind[c["pre"]], pre_w=st["w2"], pre_eps=st["eps2"], dpost_w=o["dw1"],
                                        dpost_b=o["db1"], dgate=o["dgate"], dpre_w=o["dw2"], dpre_b=o["db2"])
    return {k: v for k, v in o.items() if v is not None}


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state, state["case"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    f64 = lambda k: None if st.get(k) is None else st[k].double()  # noqa: E731
    M = case["M"]
    if op == "forward":
        x = st["x"].float()
        s = torch.clamp(x.abs().max(dim=1).values, min=1e-6)
        q = torch.clamp(torch.round(torch.div(x, s.unsqueeze(1)) * 127.0), -127, 127).double()   # fp32 by definition
        w = _digits64(st["packed"], case["K"], case["fmt"])
        z = torch.mm(q, w.T) * (st["gamma"].double() * s.double() / 127.0).unsqueeze(1)
        if st["bias"] is not None:
            z = z + f64("bias")
        y = _act64(z, case["act"])[0]
        if st["res"] is not None:
            y = y + f64("res")
        return dict(y=y, z=z) if case["pre"] else dict(y=y)
    if op == "act_grad":
        dz = f64("dy") * _act64(f64("z"), case["act"])[1]
        return dict(dz=dz, dbias=dz.sum(0))
    if op == "products":
        g, dz = st["gamma"].double(), f64("dz")
        xd = f64("xq") * f64("scale").unsqueeze(1) / 127.0
        return dict(dx=torch.mm(dz, _digits64(st["packed"], case["K"], case["fmt"])) * g, dw=torch.mm(dz.T, xd) * g)
    # the norms: differentiated by torch in 64 bits
    g, leaf = case["gate_rows"], {}
    for k in ("b", "r", "w1", "b1", "w2", "b2", "gate"):
        if st.get(k) is not None:
            leaf[k] = f64(k).requires_grad_(op == "norm_grad")

    def norm(v, kind, eps, w, b):
        if kind == "layer":
            v = v - torch.mean(v, dim=1, keepdim=True)
        if kind != "none":
            v = v * torch.rsqrt(torch.mean(torch.square(v), dim=1, keepdim=True) + eps)
        v = v * leaf[w] if w in leaf else v
        return v + leaf[b] if b in leaf else v

    u = norm(leaf["b"], case["post"], st["eps1"], "w1", "b1")
    if "gate" in leaf:
        u = u * torch.repeat_interleave(leaf["gate"], g, dim=0)[:M]
    h = st["rs"] * leaf["r"] + st["bs"] * u
    if op == "norm":
        y = norm(h, case["pre"], st["eps2"], "w2", "b2")
        return dict(h=h, codes=None) if case["out"] == "codes" else dict(h=h, y=y)
    # the second norm sees h as stored: its gradient arrives there
    hs = f64("h").requires_grad_(True)
    y = norm(hs, case["pre"], st["eps2"], "w2", "b2")
    y.backward(f64("dy"))
    h.backward(hs.grad + f64("dh"))
    names = dict(r="dr", b="db", w1="dw1", b1="db1", w2="dw2", b2="db2", gate="dgate")
    return {names[k]: v.grad for k, v in leaf.items()}


def _digits64(packed, K, fmt):
    cols, p = [], packed.to(torch.int64)
    for _ in range(PER[fmt]):
        base = dict(i2=4, t5=3, b1=2)[fmt]
        d = torch.remainder(p, base)
        cols.append(2 * d - 1 if fmt == "b1" else d - 1)
        p = torch.div(p, base, rounding_mode="floor")
    return torch.stack(cols, dim=2).reshape(packed.shape[0], -1)[:, :K].double()


def _act64(z, act):
    """The activation and its slope."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if act == "relu2":
        return torch.relu(z) * z, 2 * torch.relu(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z * cdf, cdf + z * torch.exp(-z * z / 2) * (1 / math.sqrt(2 * math.pi))


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    M, e = case["M"], {"f32": 4, "bf16": 2}
    if case["op"] in ("forward", "products"):
        N, K = case["N"], case["K"]
        packed = N * ((-(-K // PER[case["fmt"]]) + 15) // 16 * 16)
        if case["op"] == "forward":
            ys = e[case["ydt"]] * M * N
            return dict(bytes=packed + e[case["xdt"]] * M * K + ys * (1 + case["res"] + case["pre"]) + 4 * M +
                        4 * N * case["bias"], flops=2 * M * N * K)
        return dict(bytes=packed + 2 * M * N + M * K + 4 * M + e[case["dxdt"]] * M * K + 4 * N * K, flops=4 * M * N * K)
    if case["op"] == "act_grad":
        return dict(bytes=3 * e[case["dt"]] * M * case["N"] + 4 * case["N"], flops=10 * M * case["N"])
    K, s = case["K"], e[case["dt"]]
    vectors = 4 * K * (1 + (case["post"] != "none")) * (1 + case["bias"])
    gate = 4 * K * (-(-M // case["gate_rows"]) if case["gate_rows"] else 0)
    if case["op"] == "norm":
        out = 1 if case["out"] == "codes" else s
        return dict(bytes=M * K * (3 * s + out) + vectors + gate, flops=16 * M * K)
    return dict(bytes=M * K * 6 * s + 2 * (vectors + gate), flops=30 * M * K)
