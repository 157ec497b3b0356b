"""ctypes binding of ``libbitlinear.so`` (the C ABI in ``include/bitlinear.h``).

Argument marshalling only: every function here turns torch tensors into
pointers, sizes and a stream handle and calls the library entry point of the
same name.  All computation runs in the library's CUDA kernels; there is no
CPU path.  If the library has not been built the first call raises.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libbitlinear.so")
CALLS_PATH = os.path.join(HERE, "_calls.so")

BL_OK, BL_ERR_INVALID_VALUE, BL_ERR_UNSUPPORTED, BL_ERR_MISALIGNED = 0, 1, 2, 3
BL_ERR_WORKSPACE_TOO_SMALL, BL_ERR_CUDA, BL_ERR_DEVICE_TIMEOUT, BL_ERR_BAD_CODE = 4, 5, 6, 7
BL_ERR_SCRATCH_LIMIT = 8
BL_F32, BL_BF16, BL_I8, BL_I32 = 0, 1, 2, 3
BL_PACK_I2, BL_PACK_T5, BL_PACK_B1 = 0, 1, 2
BL_ACT_NONE, BL_ACT_RELU, BL_ACT_RELU2, BL_ACT_SILU, BL_ACT_GELU = 0, 1, 2, 3, 4
BL_NORM_NONE, BL_NORM_RMS, BL_NORM_LAYER = 0, 1, 2
BL_WS_HEADER_BYTES = 256

# (name, restype, argtypes) of every exported entry point
_P, _I64, _I, _F, _SZ = C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_size_t
SIGNATURES = {
    "bitlinear_packed_row_bytes": (_I64, [_I64, _I]),
    "bitlinear_quantize_weights_workspace_bytes": (_SZ, [_I64, _I64]),
    "bitlinear_forward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "bitlinear_workspace_init": (_I, [_P, _SZ, _P]),
    "bitlinear_quantize_weights": (_I, [_P, _I, _I64, _I64, _F, _I, _P, _P, _P, _P, _SZ, _P]),
    "bitlinear_absmean": (_I, [_P, _I, _I64, _I64, _P, _P, _SZ, _P]),
    "bitlinear_absmean_noalloc": (_I, [_P, _I, _I64, _I64, _P, _P]),
    "bitlinear_ternarize_pack": (_I, [_P, _I, _I64, _I64, _P, _F, _I, _P, _P, _P]),
    "bitlinear_pack": (_I, [_P, _I64, _I64, _I, _P, _P, _SZ, _P]),
    "bitlinear_binarize_weights_workspace_bytes": (_SZ, [_I64, _I64]),
    "bitlinear_binarize_weights": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "bitlinear_quantize_acts": (_I, [_P, _I, _I64, _I64, _P, _P, _P]),
    "bitlinear_layernorm_quantize_acts": (_I, [_P, _I, _P, _P, _F, _I64, _I64, _P, _P, _P, _P]),
    "bitlinear_forward": (_I, [_P, _I, _P, _I64, _I64, _P, _I, _P, _I64, _P, _I, _P, _SZ, _P]),
    "bitlinear_forward_grouped_workspace_bytes": (_SZ, [_I64, _I64, _P, _I64, _I, _I]),
    "bitlinear_forward_grouped": (_I, [_P, _I, _P, _I64, _P, _I64, _P, _I, _P, _I64, _P, _I, _P, _SZ, _P]),
    "bitlinear_backward_dx_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "bitlinear_backward_dx": (_I, [_P, _I, _P, _I64, _I64, _P, _I, _I64, _P, _P, _SZ, _P]),
    "bitlinear_backward_dw": (_I, [_P, _I, _P, _P, _P, _I64, _I64, _I64, _P, _P]),
    "bitlinear_forward_epilogue_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "bitlinear_forward_epilogue": (_I, [_P, _I, _P, _I64, _I64, _P, _I, _P, _I64, _P, _I, _P, _P, _P, _I, _P, _SZ, _P]),
    "bitlinear_epilogue_backward_workspace_bytes": (_SZ, [_I64, _I64]),
    "bitlinear_epilogue_backward": (_I, [_P, _I, _P, _I, _I, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitlinear_backward_dx_bf16_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "bitlinear_backward_dx_bf16": (_I, [_P, _I, _P, _I64, _I64, _P, _I64, _P, _I, _P, _SZ, _P]),
    "bitlinear_backward_dw_bf16_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "bitlinear_backward_dw_bf16": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "bitlinear_residual_norm": (_I, [_P, _P, _I, _P, _I, _I64, _I64, _P, _P, _I, _P, _P, _P]),
    "bitlinear_residual_norm_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "bitlinear_residual_norm_backward": (_I, [_P, _P, _I, _P, _P, _I, _P, _I, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
    "bitlinear_selftest_wait_timeout": (_I, [_P, _SZ, _P]),
    "bitlinear_device_status": (_I, [_P, _P]),
    "bitlinear_status_string": (C.c_char_p, [_I]),
    "bitlinear_version": (_I, []),
}


class ResidualNormParams(C.Structure):
    """bl_residual_norm_params"""
    _fields_ = [("post", _I), ("post_eps", _F), ("post_w", _P), ("post_b", _P), ("gate", _P), ("gate_rows", _I64),
                ("res_scale", _F), ("branch_scale", _F), ("pre", _I), ("pre_eps", _F), ("pre_w", _P), ("pre_b", _P)]


class ResidualNormGrads(C.Structure):
    """bl_residual_norm_grads"""
    _fields_ = [("dpost_w", _P), ("dpost_b", _P), ("dgate", _P), ("dpre_w", _P), ("dpre_b", _P)]


_lib = None
_lock = threading.Lock()


class BitLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib() -> C.CDLL:
    """Load the CUDA library (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                                   "(python -m bitlinear_b1_fwd_b200.build)")
            L = C.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().bitlinear_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != BL_OK:
        raise BitLinearError(status, where)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


_DT = {torch.float32: BL_F32, torch.bfloat16: BL_BF16, torch.int8: BL_I8, torch.int32: BL_I32}


def dtype_code(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


# --- size queries -----------------------------------------------------------

def bitlinear_packed_row_bytes(K: int, fmt: int) -> int:
    return int(lib().bitlinear_packed_row_bytes(K, fmt))


def bitlinear_quantize_weights_workspace_bytes(N: int, K: int) -> int:
    return int(lib().bitlinear_quantize_weights_workspace_bytes(N, K))


def bitlinear_binarize_weights_workspace_bytes(N: int, K: int) -> int:
    return int(lib().bitlinear_binarize_weights_workspace_bytes(N, K))


def bitlinear_forward_workspace_bytes(M: int, N: int, K: int, fmt: int, xdt: int) -> int:
    return int(lib().bitlinear_forward_workspace_bytes(M, N, K, fmt, xdt))


def _rows_array(group_rows):
    rows = [int(r) for r in group_rows]
    return (C.c_int64 * len(rows))(*rows), len(rows)


def bitlinear_forward_grouped_workspace_bytes(M: int, group_rows, K: int, fmt: int, xdt: int) -> int:
    arr, n = _rows_array(group_rows)
    return int(lib().bitlinear_forward_grouped_workspace_bytes(M, n, arr, K, fmt, xdt))


# --- entry points -------------------------------------------------------------

def bitlinear_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check(lib().bitlinear_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_workspace_init")


def bitlinear_quantize_weights(W, eps, fmt, packed, codes, gamma, ws, stream=None) -> None:
    _contig(W, packed, codes, gamma, ws)
    N, K = W.shape
    _check(lib().bitlinear_quantize_weights(_ptr(W), dtype_code(W), N, K, float(eps), fmt, _ptr(packed),
                                            _ptr(codes), _ptr(gamma), _ptr(ws),
                                            ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_quantize_weights")


def bitlinear_absmean(W, gamma, ws, stream=None) -> None:
    _contig(W, gamma, ws)
    N, K = W.shape
    _check(lib().bitlinear_absmean(_ptr(W), dtype_code(W), N, K, _ptr(gamma), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "bitlinear_absmean")


def bitlinear_absmean_noalloc(W, gamma, stream=None) -> None:
    """gamma of W without a workspace (the library's fixed device scratch)."""
    _contig(W, gamma)
    N, K = W.shape
    _check(lib().bitlinear_absmean_noalloc(_ptr(W), dtype_code(W), N, K, _ptr(gamma), _stream(stream)),
           "bitlinear_absmean_noalloc")


def bitlinear_ternarize_pack(W, gamma, eps, fmt, packed, codes, stream=None) -> None:
    _contig(W, packed, codes, gamma)
    N, K = W.shape
    _check(lib().bitlinear_ternarize_pack(_ptr(W), dtype_code(W), N, K, _ptr(gamma), float(eps), fmt,
                                          _ptr(packed), _ptr(codes), _stream(stream)),
           "bitlinear_ternarize_pack")


def bitlinear_pack(codes, fmt, packed, ws, stream=None) -> None:
    _contig(codes, packed, ws)
    N, K = codes.shape
    _check(lib().bitlinear_pack(_ptr(codes), N, K, fmt, _ptr(packed), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "bitlinear_pack")


def bitlinear_quantize_acts(x, xq, scale, stream=None) -> None:
    _contig(x, xq, scale)
    M, K = x.shape
    _check(lib().bitlinear_quantize_acts(_ptr(x), dtype_code(x), M, K, _ptr(xq), _ptr(scale),
                                         _stream(stream)), "bitlinear_quantize_acts")


def bitlinear_layernorm_quantize_acts(x, ln_w, ln_b, eps, xq, scale, y=None, stream=None) -> None:
    """LayerNorm of each token (y: optional bf16 output), then per-token INT8."""
    _contig(x, ln_w, ln_b, xq, scale, y)
    M, K = x.shape
    _check(lib().bitlinear_layernorm_quantize_acts(_ptr(x), dtype_code(x), _ptr(ln_w), _ptr(ln_b), float(eps), M, K,
                                                   _ptr(y), _ptr(xq), _ptr(scale), _stream(stream)),
           "bitlinear_layernorm_quantize_acts")


def bitlinear_binarize_weights(W, packed, codes, beta, alpha, ws, stream=None) -> None:
    _contig(W, packed, codes, beta, alpha, ws)
    N, K = W.shape
    _check(lib().bitlinear_binarize_weights(_ptr(W), dtype_code(W), N, K, _ptr(packed), _ptr(codes), _ptr(beta),
                                            _ptr(alpha), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_binarize_weights")


def bitlinear_forward(packed, fmt, gamma, N, K, x, scale, y, ws, stream=None) -> None:
    _contig(packed, gamma, x, scale, y, ws)
    M = x.shape[0]
    _check(lib().bitlinear_forward(_ptr(packed), fmt, _ptr(gamma), N, K, _ptr(x), dtype_code(x),
                                   _ptr(scale), M, _ptr(y), dtype_code(y), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_forward")


def bitlinear_forward_grouped(packed, fmt, gammas, group_rows, K, x, scale, y, ws, stream=None) -> None:
    _contig(packed, gammas, x, scale, y, ws)
    M = x.shape[0]
    arr, n = _rows_array(group_rows)
    _check(lib().bitlinear_forward_grouped(_ptr(packed), fmt, _ptr(gammas), n, arr, K, _ptr(x), dtype_code(x),
                                           _ptr(scale), M, _ptr(y), dtype_code(y), _ptr(ws),
                                           ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_forward_grouped")


def bitlinear_backward_dx_workspace_bytes(M: int, N: int, K: int, fmt: int) -> int:
    return int(lib().bitlinear_backward_dx_workspace_bytes(M, N, K, fmt))


def bitlinear_backward_dx(packed, fmt, gamma, N, K, dy, dx, ws, stream=None) -> None:
    _contig(packed, gamma, dy, dx, ws)
    M = dy.shape[0]
    _check(lib().bitlinear_backward_dx(_ptr(packed), fmt, _ptr(gamma), N, K, _ptr(dy), dtype_code(dy), M, _ptr(dx),
                                       _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_backward_dx")


def bitlinear_backward_dw(dy, xq, scale, gamma, dw, stream=None) -> None:
    _contig(dy, xq, scale, gamma, dw)
    M, N = dy.shape
    K = xq.shape[1]
    _check(lib().bitlinear_backward_dw(_ptr(dy), dtype_code(dy), _ptr(xq), _ptr(scale), _ptr(gamma), M, N, K,
                                       _ptr(dw), _stream(stream)),
           "bitlinear_backward_dw")


# --- the product with its epilogue, its gradients, the norms around a block -------
#
# These calls check shapes, dtypes, contiguity and that every tensor is on one
# CUDA device, and run on that device (the current stream there unless one is
# given); the current device of the caller does not change.  The checks and the
# marshalling are compiled (csrc/bl_calls.cpp): in Python they took longer than a
# launch.

_native = None


def _calls():
    """The compiled marshalling (raises if it, or the library, has not been built)."""
    global _native
    if _native is None:
        lib()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} is missing: build it first (python -m bitlinear_b1_fwd_b200.build)")
        try:
            from . import _calls as native
        except ImportError as e:  # compiled for another Python or torch
            raise RuntimeError(f"{CALLS_PATH} does not load here: build it again "
                               f"(python -m bitlinear_b1_fwd_b200.build)") from e
        _native = native
    return _native


def bitlinear_forward_epilogue_workspace_bytes(M: int, N: int, K: int, fmt: int, xdt: int) -> int:
    return int(lib().bitlinear_forward_epilogue_workspace_bytes(M, N, K, fmt, xdt))


def bitlinear_forward_epilogue(packed, fmt, gamma, N, K, x, scale, y, ws, bias=None, act=BL_ACT_NONE, residual=None,
                               preact=None, stream=None) -> None:
    """y = act(x W_q^T dequantized + bias) + residual; preact receives the argument of act."""
    status = (_native or _calls()).forward_epilogue(packed, fmt, gamma, N, K, x, scale, y, ws, bias, act, residual,
                                                    preact, stream)
    if status:
        raise BitLinearError(status, "bitlinear_forward_epilogue")


def bitlinear_epilogue_backward_workspace_bytes(M: int, N: int) -> int:
    return int(lib().bitlinear_epilogue_backward_workspace_bytes(M, N))


def bitlinear_epilogue_backward(dy, z, act, dz, dbias, ws, stream=None) -> None:
    """dz = dy act'(z) and dbias = its column sums (either may be None)."""
    status = (_native or _calls()).epilogue_backward(dy, z, act, dz, dbias, ws, stream)
    if status:
        raise BitLinearError(status, "bitlinear_epilogue_backward")


def bitlinear_backward_dx_bf16_workspace_bytes(M: int, N: int, K: int, fmt: int) -> int:
    return int(lib().bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, fmt))


def bitlinear_backward_dx_bf16(packed, fmt, gamma, N, K, dz, dx, ws, stream=None) -> None:
    """dx = gamma dz W_q on the tensor cores (bf16 dz, dx bf16 or fp32)."""
    status = (_native or _calls()).backward_dx_bf16(packed, fmt, gamma, N, K, dz, dx, ws, stream)
    if status:
        raise BitLinearError(status, "bitlinear_backward_dx_bf16")


def bitlinear_backward_dw_bf16_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().bitlinear_backward_dw_bf16_workspace_bytes(M, N, K))


def bitlinear_backward_dw_bf16(dz, xq, scale, gamma, dw, ws, stream=None) -> None:
    """dW = gamma dz^T x_deq on the tensor cores (bf16 dz, fp32 dW)."""
    status = (_native or _calls()).backward_dw_bf16(dz, xq, scale, gamma, dw, ws, stream)
    if status:
        raise BitLinearError(status, "bitlinear_backward_dw_bf16")


def bitlinear_residual_norm(b, r, h, post=BL_NORM_NONE, post_w=None, post_b=None, post_eps=1e-5, gate=None,
                            gate_rows=0, res_scale=1.0, branch_scale=1.0, pre=BL_NORM_RMS, pre_w=None, pre_b=None,
                            pre_eps=1e-5, y=None, xq=None, scale=None, stream=None) -> None:
    """h = res_scale r + branch_scale gate norm_post(b); y = norm_pre(h); xq, scale its INT8 codes.

    gate: [rows, K] with one row for every gate_rows tokens (0: one row for all, also as [K]).  Without tokens a shared
    gate keeps its row, one with rows of its own has one or none."""
    status = (_native or _calls()).residual_norm(b, r, h, post, post_w, post_b, post_eps, gate, gate_rows, res_scale,
                                                 branch_scale, pre, pre_w, pre_b, pre_eps, y, xq, scale, stream)
    if status:
        raise BitLinearError(status, "bitlinear_residual_norm")


def bitlinear_residual_norm_backward_workspace_bytes(M: int, K: int, gate_rows: int = 0) -> int:
    """gate_rows as for the call; 0 without a gate or with one row for every token."""
    return int(lib().bitlinear_residual_norm_backward_workspace_bytes(M, K, gate_rows if gate_rows > 0 else max(M, 1)))


def bitlinear_residual_norm_backward(dy, dh, b, h, dr, db, ws, post=BL_NORM_NONE, post_w=None, post_b=None,
                                     post_eps=1e-5, gate=None, gate_rows=0, res_scale=1.0, branch_scale=1.0,
                                     pre=BL_NORM_RMS, pre_w=None, pre_eps=1e-5, dpost_w=None, dpost_b=None, dgate=None,
                                     dpre_w=None, dpre_b=None, stream=None) -> None:
    """Gradients of bitlinear_residual_norm from dy (of y) and dh (of h, or None)."""
    status = (_native or _calls()).residual_norm_backward(dy, dh, b, h, dr, db, ws, post, post_w, post_b, post_eps,
                                                          gate, gate_rows, res_scale, branch_scale, pre, pre_w, pre_eps,
                                                          dpost_w, dpost_b, dgate, dpre_w, dpre_b, stream)
    if status:
        raise BitLinearError(status, "bitlinear_residual_norm_backward")


def bitlinear_device_status(ws, stream=None) -> int:
    """Synchronize and return (and clear) the workspace's device status."""
    return int(lib().bitlinear_device_status(_ptr(ws), _stream(stream)))


def bitlinear_selftest_wait_timeout(ws, stream=None) -> None:
    _check(lib().bitlinear_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "bitlinear_selftest_wait_timeout")


def bitlinear_version() -> int:
    return int(lib().bitlinear_version())


# --- convenience layer (allocation through torch, then the calls above) ----------

class BitLinear:
    """A BitLinear layer holding packed ternary weights and gamma on the GPU.

    ``BitLinear.from_weight(W)`` runs steps 1-3 once; calling the layer on
    activations x [M, K] (fp32 / bf16) runs steps 4-6 and returns y [M, N].
    """

    def __init__(self, packed, gamma, N, K, fmt=BL_PACK_I2):
        self.packed, self.gamma, self.N, self.K, self.fmt = packed, gamma, N, K, fmt
        self._ws = None

    @classmethod
    def from_weight(cls, W: torch.Tensor, fmt: int = BL_PACK_I2, eps: float = 1e-5, stream=None):
        N, K = W.shape
        dev = W.device
        packed = torch.empty((N, bitlinear_packed_row_bytes(K, fmt)), dtype=torch.uint8, device=dev)
        gamma = torch.empty(1, dtype=torch.float32, device=dev)
        ws = torch.zeros(bitlinear_quantize_weights_workspace_bytes(N, K), dtype=torch.uint8, device=dev)
        bitlinear_quantize_weights(W, eps, fmt, packed, None, gamma, ws, stream)
        return cls(packed, gamma, N, K, fmt)

    def workspace(self, M: int, xdt: int) -> torch.Tensor:
        need = bitlinear_forward_workspace_bytes(M, self.N, self.K, self.fmt, xdt)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.zeros(need, dtype=torch.uint8, device=self.packed.device)
        return self._ws

    def __call__(self, x: torch.Tensor, out_dtype=torch.bfloat16, stream=None):
        M = x.shape[0]
        y = torch.empty((M, self.N), dtype=out_dtype, device=x.device)
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
        ws = self.workspace(M, dtype_code(x))
        bitlinear_forward(self.packed, self.fmt, self.gamma, self.N, self.K, x, scale, y, ws, stream)
        return y
