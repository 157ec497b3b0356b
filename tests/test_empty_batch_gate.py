"""Gates of a batch without tokens: a gate shared by every token has its one row
all the same ([K] or [1, K]), and its gradient is zeros; a gate with rows of its
own has none, or one."""
import pytest
import torch

from bitlinear_b1_fwd_b200 import binding as B

K = 48


def gates(device):
    """(gate, gate_rows) of every accepted form."""
    one, none = torch.ones(1, K, device=device), torch.ones(0, K, device=device)
    return [(one, 0), (one[0], 0), (one, 7), (one[0], 7), (none, 7)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from bitlinear_b1_fwd_b200 import build
    build.build()


@pytest.mark.parametrize("i", range(5))
def test_shapes_are_accepted(i):
    """CPU tensors get as far as the complaint about their device, the last of the checks."""
    gate, rows = gates("cpu")[i]
    e, ws = torch.empty(0, K), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitlinear_residual_norm(e, e, e, gate=gate, gate_rows=rows)
    with pytest.raises(ValueError, match="CUDA"):
        B.bitlinear_residual_norm_backward(e, None, e, e, e, e, ws, gate=gate, gate_rows=rows,
                                           dgate=torch.empty_like(gate))


@pytest.mark.parametrize("rows", [0, 7])
def test_shapes_are_refused(rows):
    e, ws = torch.empty(0, K), torch.zeros(256, dtype=torch.uint8)
    for bad in (torch.ones(2, K), torch.ones(1, K + 1), torch.ones(K + 1), torch.ones(1, 1, K)) + \
            (() if rows else (torch.ones(0, K),)):
        with pytest.raises(ValueError, match="gate: shape"):
            B.bitlinear_residual_norm(e, e, e, gate=bad, gate_rows=rows)
        with pytest.raises(ValueError, match="gate: shape"):
            B.bitlinear_residual_norm_backward(e, None, e, e, e, e, ws, gate=bad, gate_rows=rows)
    with pytest.raises(ValueError, match="dgate: shape"):
        B.bitlinear_residual_norm_backward(e, None, e, e, e, e, ws, gate=torch.ones(1, K), gate_rows=rows,
                                           dgate=torch.ones(0, K))


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(5))
def test_forward_and_gradient(i):
    gate, rows = gates("cuda")[i]
    e = torch.empty(0, K, device="cuda")
    ws = torch.zeros(B.bitlinear_residual_norm_backward_workspace_bytes(0, K, rows), dtype=torch.uint8, device="cuda")
    B.bitlinear_residual_norm(e, e, torch.empty_like(e), gate=gate, gate_rows=rows)
    guard = torch.full((3, K), 5.0, device="cuda")
    dgate = guard[1:2].view(gate.shape) if gate.numel() else guard[1:1]
    dw = torch.full((K,), 5.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.bitlinear_residual_norm_backward(e, None, e, e, torch.empty_like(e), torch.empty_like(e), ws, gate=gate,
                                       gate_rows=rows, dgate=dgate, dpre_w=dw, stream=side)
    side.synchronize()
    assert not dw.any() and not dgate.any()
    guard[1:1 + gate.numel() // K] = 5.0
    assert (guard == 5.0).all()


@pytest.mark.gpu
def test_c_entry_clears_the_shared_row():
    import ctypes as C
    buf = torch.full((2, K), 5.0, device="cuda")
    gate = torch.ones(K, device="cuda")
    p = B.ResidualNormParams(post=B.BL_NORM_NONE, post_eps=1e-5, gate=gate.data_ptr(), gate_rows=1, res_scale=1.0,
                             branch_scale=1.0, pre=B.BL_NORM_RMS, pre_eps=1e-5)
    g = B.ResidualNormGrads(dgate=buf.data_ptr())
    null = C.c_void_p(None)
    status = B.lib().bitlinear_residual_norm_backward(
        C.addressof(p), null, B.BL_F32, null, null, B.BL_F32, null, B.BL_F32, 0, K, null, null, C.addressof(g), null, 0,
        C.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == B.BL_OK
    assert not buf[0].any() and (buf[1] == 5.0).all()
