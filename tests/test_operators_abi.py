"""The epilogue product, its gradients and the norms around a block on the CPU:
every call rejects bad arguments on the host before any CUDA call, empty
batches are no-ops, the workspace queries hold their formulas, and the binding
refuses tensors of the wrong shape, type, layout or device."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def bl():
    from bitlinear_b1_fwd_b200 import build, binding
    build.build()
    return binding


P = C.c_void_p(1 << 20)            # aligned, never dereferenced
Q = C.c_void_p(1 << 21)
R = C.c_void_p(1 << 22)
ODD = C.c_void_p((1 << 20) + 4)
OVER = 1 << 31
BIG = 1 << 62


def _with(defaults, **kw):
    return [kw.get(k, v) for k, v in defaults.items()]


def test_forward_epilogue_refusals(bl):
    base = dict(packed=P, fmt=0, gamma=P, N=4, K=16, x=P, xdt=1, scale=P, M=1, bias=P, act=1, res=P, pre=Q, y=R, ydt=1,
                ws=P, ws_bytes=4096, stream=None)
    call = lambda **kw: bl.lib().bitlinear_forward_epilogue(*_with(base, **kw))  # noqa: E731
    for bad in (dict(act=-1), dict(act=5), dict(ydt=3), dict(ydt=2), dict(fmt=3), dict(xdt=3), dict(packed=None),
                dict(gamma=None), dict(x=None), dict(scale=None), dict(y=None), dict(ws=None), dict(K=0), dict(M=-1),
                dict(M=OVER, ws_bytes=BIG), dict(N=OVER, K=1, ws_bytes=BIG), dict(pre=R), dict(pre=P)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(res=ODD), dict(pre=ODD), dict(y=ODD), dict(x=ODD), dict(bias=C.c_void_p((1 << 20) + 2))):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(ws_bytes=8) == bl.BL_ERR_WORKSPACE_TOO_SMALL
    assert call(M=0, x=None, y=None, pre=None, res=None) == bl.BL_OK
    assert call(N=0) == bl.BL_OK
    assert call() == bl.BL_ERR_CUDA                   # passes every check: no device here
    assert call(bias=None, res=None, pre=None) == bl.BL_ERR_CUDA
    assert call(res=R) == bl.BL_ERR_CUDA              # in place
    q = bl.bitlinear_forward_epilogue_workspace_bytes
    assert q(1, 8640, 3200, 0, 1) == 256              # the decode kernel
    # 16 tokens in 16-byte pieces: 27 chunks of four 80-weight segments, and a sum each
    assert q(16, 3200, 8640, 1, 1) == 256 + 27 * 4 * 80 * 16 + 16 * 4
    # codes and int8 weights
    assert q(4096, 8640, 3200, 2, 0) == 256 + 4096 * 3200 + 8640 * 3200
    assert q(4096, 8640, 3200, 0, 2) == 256 + 8640 * 3200
    assert q(0, 8640, 3200, 0, 1) == 256 and q(-1, 8, 8, 0, 1) == 0 and q(4, 8, 8, 3, 1) == 0


def test_epilogue_backward_refusals(bl):
    base = dict(dy=P, dydt=1, z=Q, zdt=1, act=3, M=4, N=8, dz=R, dbias=P, ws=P, ws_bytes=4096, stream=None)
    call = lambda **kw: bl.lib().bitlinear_epilogue_backward(*_with(base, **kw))  # noqa: E731
    for bad in (dict(dydt=2), dict(zdt=3), dict(act=7), dict(act=-1), dict(M=-1), dict(M=OVER), dict(N=0),
                dict(N=OVER), dict(dy=None), dict(z=None), dict(dz=None, dbias=None), dict(ws=None), dict(dz=Q)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(dy=ODD), dict(z=ODD), dict(dz=ODD), dict(ws=ODD)):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(ws_bytes=8) == bl.BL_ERR_WORKSPACE_TOO_SMALL
    assert call(M=0, dbias=None) == bl.BL_OK
    assert call() == bl.BL_ERR_CUDA
    assert call(z=None, act=0) == bl.BL_ERR_CUDA
    assert call(dz=P) == bl.BL_ERR_CUDA               # over dy
    q = bl.bitlinear_epilogue_backward_workspace_bytes
    assert q(8, 256) == 256 + 1024                    # one block of rows
    assert q(1, 0) == 0 and q(OVER, 8) == 0 and q(-1, 8) == 0


def test_gradient_product_refusals(bl):
    base = dict(packed=P, fmt=0, gamma=P, N=4, K=16, dz=P, M=2, dx=P, dxdt=1, ws=P, ws_bytes=1 << 20, stream=None)
    call = lambda **kw: bl.lib().bitlinear_backward_dx_bf16(*_with(base, **kw))  # noqa: E731
    for bad in (dict(fmt=3), dict(dxdt=2), dict(M=-1), dict(M=OVER), dict(N=0), dict(K=0), dict(packed=None),
                dict(gamma=None), dict(dz=None), dict(dx=None), dict(ws=None)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(packed=ODD), dict(dz=ODD), dict(dx=ODD), dict(ws=ODD)):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(ws_bytes=8) == bl.BL_ERR_WORKSPACE_TOO_SMALL
    assert call(M=0, dz=None, dx=None) == bl.BL_OK
    assert call() == bl.BL_ERR_CUDA
    base = dict(dz=P, xq=P, scale=P, gamma=P, M=2, N=4, K=16, dw=P, ws=P, ws_bytes=1 << 20, stream=None)
    call = lambda **kw: bl.lib().bitlinear_backward_dw_bf16(*_with(base, **kw))  # noqa: E731
    for bad in (dict(M=-1), dict(M=OVER), dict(N=0), dict(K=0), dict(N=OVER, K=1), dict(dz=None), dict(xq=None),
                dict(scale=None), dict(gamma=None), dict(dw=None), dict(ws=None)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(dz=ODD), dict(xq=ODD), dict(dw=ODD), dict(ws=ODD)):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(ws_bytes=8) == bl.BL_ERR_WORKSPACE_TOO_SMALL
    assert call() == bl.BL_ERR_CUDA
    assert bl.bitlinear_backward_dx_bf16_workspace_bytes(1, 0, 16, 0) == 0
    assert bl.bitlinear_backward_dw_bf16_workspace_bytes(OVER, 4, 16) == 0


def _params(bl, **kw):
    d = dict(post=1, post_eps=1e-5, post_w=None, post_b=None, gate=None, gate_rows=0, res_scale=1.0, branch_scale=1.0,
             pre=2, pre_eps=1e-5, pre_w=None, pre_b=None)
    d.update(kw)
    return bl.ResidualNormParams(*d.values())


BAD_PARAMS = (dict(post=3), dict(pre=-1), dict(post_eps=0.0), dict(pre_eps=float("nan")), dict(pre_eps=float("inf")),
              dict(res_scale=float("nan")), dict(branch_scale=float("inf")), dict(gate=1 << 20, gate_rows=0),
              dict(gate=1 << 20, gate_rows=-1))


def test_residual_norm_refusals(bl):
    base = dict(b=P, bdt=1, r=Q, rdt=1, M=2, K=16, h=R, y=None, ydt=1, xq=P, scale=P, stream=None)

    def call(params=None, null=False, **kw):
        p = _params(bl, **(params or {}))
        return bl.lib().bitlinear_residual_norm(None if null else C.addressof(p), *_with(base, **kw))

    assert call(null=True) == bl.BL_ERR_INVALID_VALUE
    for bad in BAD_PARAMS:
        assert call(params=bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(bdt=2), dict(rdt=3), dict(y=C.c_void_p(1 << 23), ydt=2), dict(M=-1), dict(M=OVER), dict(K=0),
                dict(K=(1 << 20) + 1), dict(xq=None), dict(scale=None), dict(h=None, xq=None, scale=None),
                dict(b=None), dict(r=None), dict(y=P), dict(y=Q), dict(y=R), dict(h=P)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(b=ODD), dict(r=ODD), dict(h=ODD), dict(y=ODD), dict(xq=ODD)):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(params=dict(pre_w=(1 << 20) + 2)) == bl.BL_ERR_MISALIGNED
    assert call(M=0, b=None, r=None) == bl.BL_OK
    assert call() == bl.BL_ERR_CUDA
    assert call(h=Q) == bl.BL_ERR_CUDA                # over r
    assert call(params=dict(post=0, post_eps=0.0)) == bl.BL_ERR_CUDA


def test_residual_norm_backward_refusals(bl):
    S, T = C.c_void_p(1 << 24), C.c_void_p(1 << 25)
    base = dict(dy=P, dydt=1, dh=Q, b=R, bdt=1, h=S, rdt=1, M=2, K=16, dr=T, db=C.c_void_p(1 << 26))
    tail = dict(ws=P, ws_bytes=1 << 20, stream=None)

    def call(params=None, grads=(None,) * 5, null=False, **kw):
        p = _params(bl, **(params or {}))
        g = bl.ResidualNormGrads(*grads)
        return bl.lib().bitlinear_residual_norm_backward(C.addressof(p), *_with(base, **kw),
                                                         None if null else C.addressof(g), *_with(tail, **kw))

    assert call(null=True) == bl.BL_ERR_INVALID_VALUE
    for bad in BAD_PARAMS:
        assert call(params=bad) == bl.BL_ERR_INVALID_VALUE, bad
    for bad in (dict(dydt=2), dict(bdt=2), dict(rdt=3), dict(M=-1), dict(M=OVER), dict(K=0), dict(dy=None),
                dict(b=None), dict(h=None), dict(ws=None), dict(dr=None, db=None), dict(dr=P), dict(dr=R), dict(dr=S),
                dict(db=T), dict(db=Q), dict(db=R), dict(db=S), dict(db=P, dydt=0)):
        assert call(**bad) == bl.BL_ERR_INVALID_VALUE, bad
    assert call(grads=(None, None, 1 << 20, None, None)) == bl.BL_ERR_INVALID_VALUE      # dgate without a gate
    for bad in (dict(dy=ODD), dict(dh=ODD), dict(b=ODD), dict(h=ODD), dict(dr=ODD), dict(db=ODD), dict(ws=ODD)):
        assert call(**bad) == bl.BL_ERR_MISALIGNED, bad
    assert call(grads=((1 << 20) + 2, None, None, None, None)) == bl.BL_ERR_MISALIGNED
    assert call(ws_bytes=8) == bl.BL_ERR_WORKSPACE_TOO_SMALL
    assert call(M=0, dy=None) == bl.BL_OK
    assert call() == bl.BL_ERR_CUDA
    assert call(dr=Q, db=P) == bl.BL_ERR_CUDA         # over dh and dy
    q = bl.lib().bitlinear_residual_norm_backward_workspace_bytes
    assert q(1, 64, 0) == 256 + 4 * 64 * 4 + 256      # one block, one row's statistics
    assert q(1, 64, 1) == q(1, 64, BIG) == 256 + 4 * 64 * 4 + 2 * 64 * 4 + 256
    assert q(-1, 64, 0) == 0 and q(1, 0, 0) == 0 and q(1, 64, -1) == 0


def test_binding_refuses_tensors(bl):
    """Shapes, types and devices are checked before the library is called (CPU tensors are refused)."""
    ws = torch.zeros(4096, dtype=torch.uint8)
    f = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        bl.bitlinear_residual_norm(f, f, f)
    with pytest.raises(ValueError, match="dimensions"):
        bl.bitlinear_epilogue_backward(torch.zeros(4), None, 0, None, f, ws)
    y = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="h: unsupported dtype"):
        bl.bitlinear_residual_norm(f, f, f.half())
    with pytest.raises(ValueError, match="r: shape"):
        bl.bitlinear_residual_norm(f, torch.zeros(8, 4), f)
    with pytest.raises(ValueError, match="y must be contiguous"):
        bl.bitlinear_residual_norm(f, f, f, y=torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="one row, expected 2"):
        bl.bitlinear_residual_norm(f, f, f, gate=torch.zeros(8), gate_rows=2)
    with pytest.raises(ValueError, match="gate: shape"):
        bl.bitlinear_residual_norm(f, f, f, gate=torch.zeros(3, 8), gate_rows=2)
    with pytest.raises(ValueError, match="dgate without"):
        bl.bitlinear_residual_norm_backward(f, None, f, f, f, f, ws, dgate=y)
    with pytest.raises(ValueError, match="dh: shape"):
        bl.bitlinear_residual_norm_backward(f, torch.zeros(4, 9), f, f, f, f, ws)
    with pytest.raises(TypeError, match="must be a tensor"):
        bl.bitlinear_residual_norm(f, None, f)
    codes, s = torch.zeros(16, 16, dtype=torch.uint8), torch.zeros(4)
    with pytest.raises(ValueError, match="packed: shape"):
        bl.bitlinear_forward_epilogue(codes, 0, torch.zeros(1), 16, 128, torch.zeros(4, 128), s, torch.zeros(4, 16), ws)
    with pytest.raises(TypeError, match="residual: unsupported dtype"):
        bl.bitlinear_forward_epilogue(codes, 0, torch.zeros(1), 16, 8, f, s, torch.zeros(4, 16), ws,
                                      residual=torch.zeros(4, 16).bfloat16())
    with pytest.raises(TypeError, match="dz: unsupported dtype"):
        bl.bitlinear_backward_dw_bf16(f, torch.zeros(4, 8, dtype=torch.int8), s, torch.zeros(1), torch.zeros(8, 8), ws)
    with pytest.raises(ValueError, match="dw: shape"):
        bl.bitlinear_backward_dw_bf16(f.bfloat16(), torch.zeros(4, 8, dtype=torch.int8), s, torch.zeros(1),
                                      torch.zeros(8, 9), ws)
    with pytest.raises(ValueError, match="dx: shape"):
        bl.bitlinear_backward_dx_bf16(codes[:8], 0, torch.zeros(1), 8, 8, f.bfloat16(), torch.zeros(4, 9), ws)
