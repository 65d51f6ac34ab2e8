"""ctypes binding of ``libw4b200.so`` (C ABI in ``include/w4.h``).

Argument marshalling only: every computation runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (torch provides device memory and the
current stream); there is no CPU path, and importing this module fails loudly
when the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libw4b200.so")
LIB_CHECKED_PATH = os.path.join(_PKG, "libw4b200_checked.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "w4.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m weight_only_bit_gemm_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t

_SIGS = {
    "w4_status_string": (ctypes.c_char_p, [_i]),
    "w4_version": (_i, []),
    "w4_checked_build": (_i, []),
    "w4_device_status": (_i, [_p]),
    "w4_selftest_wait_timeout": (_i, [_p]),
    "w4_weight_bytes": (ctypes.c_double, [_i, _i, _i]),
    "w4_quantize_rtn": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p]),
    "w4_quantize_sym": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p]),
    "w4_awq_scale_weights": (_i, [_p, _p, _i, _i, _p, _p]),
    "w4_awq_scale_activations": (_i, [_p, _p, _i, _i, _p, _p]),
    "w4_gptq_workspace_bytes": (_sz, [_i, _i, _i]),
    "w4_gptq_quantize": (_i, [_p, _p, _i, _i, _i, _i, ctypes.c_float, _p, _p, _p, _p, _p, _sz,
                              _p]),
    "w4_gptq_hessian": (_i, [_p, _i, _i, _p, _p]),
    "llm_int8_quantize_weights": (_i, [_p, _i, _i, _p, _p, _p]),
    "llm_int8_workspace_bytes": (_sz, [_i, _i, _i]),
    "llm_int8_gemm": (_i, [_p, _p, _p, _i, _i, _i, ctypes.c_float, _p, _p, _sz, _p]),
    "w4_dequant": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p]),
    "w4_prepacked_bytes": (_sz, [_i, _i, _i, _i]),
    "w4_prepack": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p]),
    "w4_unprepack": (_i, [_p, _i, _i, _i, _i, _p, _p, _p, _p, _p]),
    "w4_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "w4a16_gemm": (_i, [_p, _p, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "w4a16_gemm_static_scratch": (_i, [_p, _p, _i, _i, _i, _i, _i, _p, _p]),
    "w4_awq_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "w4a16_awq_gemm": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "nf4_quantize": (_i, [_p, _i, _i, _i, _i, _p, _p, _p, _p]),
    "nf4_dequant": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "nf4_levels": (None, [_p]),
    "nf4_prepacked_bytes": (_sz, [_i, _i]),
    "nf4_prepack": (_i, [_p, _p, _i, _i, _p, _p]),
    "nf4_workspace_bytes": (_sz, [_i, _i, _i]),
    "nf4_gemm": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "nf4_quantize_meandq": (_i, [_p, _i, _i, _i, _i, _p, _p, _p, _p, _p]),
    "nf4_dequant_meandq": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "nf4_gemm_meandq": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "fp4_quantize": (_i, [_p, _i, _i, _i, _i, _p, _p, _p, _p]),
    "fp4_dequant": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p]),
    "fp4_levels": (None, [_p]),
    "fp4_gemm": (_i, [_p, _p, _p, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "fp8_quantize_weights": (_i, [_p, _i, _i, _i, _p, _p, _p]),
    "fp8_quantize_activations": (_i, [_p, _i, _i, _p, _p, _p]),
    "fp8_add_rmsnorm": (_i, [_p, _p, _p, ctypes.c_float, _i, _i, _p, _p, _p, _p, _p]),
    "fp8_gemm_workspace_bytes": (_sz, [_i, _i, _i]),
    "fp8_gemm": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "fp8_selftest_wait_timeout": (_i, [_p]),
    "fp8_moe_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fp8_moe": (_i, [_p, _p, _p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p, _p, _sz, _p]),
}
def _bind(handle):
    for name, (res, args) in _SIGS.items():
        f = getattr(handle, name)
        f.restype = res
        f.argtypes = args
    return handle


_bind(lib)
_checked = None


def checked_library():
    """The bounds-checked build (libw4b200_checked.so), loaded on first use;
    ImportError if it has not been built."""
    global _checked
    if _checked is None:
        if not os.path.exists(LIB_CHECKED_PATH):
            raise ImportError(f"{LIB_CHECKED_PATH} is missing: build it with "
                              "`python -m weight_only_bit_gemm_b200.build --checked`")
        _checked = _bind(ctypes.CDLL(LIB_CHECKED_PATH))
    return _checked


@contextlib.contextmanager
def using(handle):
    """Route every wrapper of this module through another build of the
    library (e.g. checked_library()) inside the block."""
    global lib
    saved = lib
    lib = handle
    try:
        yield handle
    finally:
        lib = saved


W4_OK, W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED, W4_ERR_CUDA, W4_ERR_TIMEOUT, \
    W4_ERR_DEVICE_INPUT = range(6)
W4_ERR_SCRATCH_LIMIT = 6
W4_ERR_BOUNDS = 7
W4_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024


class W4Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.w4_status_string(status).decode()} ({status})")


def header_functions() -> list:
    """Names of the functions declared in include/w4.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(\w+)\s*\(", text)) - {"defined", "if"})


def _check(status: int, what: str) -> None:
    if status != W4_OK:
        raise W4Error(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _raw_stream(dev):
    """The current stream of device index dev, as an integer."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _cuda(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")
    return t


def device_status() -> int:
    """Synchronise the current stream and return/clear the device error word.
    After a call that did not run through (W4_ERR_TIMEOUT, W4_ERR_BOUNDS) the
    fp8 calls' default workspaces on this device, whose counters it may have
    left nonzero, are given up: the next calls make new ones."""
    status = lib.w4_device_status(_stream())
    if status in (W4_ERR_TIMEOUT, W4_ERR_BOUNDS):
        dev = torch.cuda.current_device()
        for key in list(_FP8_WS):
            if key[0] == dev:
                _FP8_WS.pop(key, None)
    return status


def selftest_wait_timeout() -> None:
    """Run the bounded-wait failure path once (see w4.h); device_status() then
    reports W4_ERR_TIMEOUT."""
    _check(lib.w4_selftest_wait_timeout(_stream()), "w4_selftest_wait_timeout")


def fp8_selftest_wait_timeout() -> None:
    """The same for the expert layer's wait on a counter in global memory."""
    _check(lib.fp8_selftest_wait_timeout(_stream()), "fp8_selftest_wait_timeout")


# ----------------------------------------------------------------- INT4 RTN

def _quantize_int4(fn, name, W, G, g_idx):
    _cuda(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    sc = torch.empty((N, K // G), dtype=torch.float16, device=dev)
    zr = torch.empty((N, K // G), dtype=torch.uint8, device=dev)
    if g_idx is not None:
        _cuda(g_idx, torch.int32, "g_idx")
    _check(fn(_ptr(W), N, K, G, _ptr(g_idx), _ptr(Wq), _ptr(sc), _ptr(zr), _stream()), name)
    return Wq, sc, zr


def quantize_rtn(W, G, g_idx=None):
    """fp32 W [N, K] -> (Wq uint8 [N, K/2], scales fp16 [N, K/G], zeros uint8 [N, K/G])."""
    return _quantize_int4(lib.w4_quantize_rtn, "w4_quantize_rtn", W, G, g_idx)


def quantize_sym(W, G, g_idx=None):
    """Symmetric INT4 (scale max|w|/7, zero point 8), same outputs as quantize_rtn."""
    return _quantize_int4(lib.w4_quantize_sym, "w4_quantize_sym", W, G, g_idx)


def awq_scale_weights(W, s, out=None):
    """fp32 W [N, K] * s [K] (per input channel) in fp32."""
    _cuda(W, torch.float32, "W")
    _cuda(s, torch.float32, "s")
    N, K = W.shape
    if out is None:
        out = torch.empty_like(W)
    _check(lib.w4_awq_scale_weights(_ptr(W), _ptr(s), N, K, _ptr(out), _stream()),
           "w4_awq_scale_weights")
    return out


def awq_scale_activations(X, s, out=None):
    """bf16 X [M, K] / s [K] per input channel, rounded to bf16."""
    _cuda(X, torch.bfloat16, "X")
    _cuda(s, torch.float32, "s")
    M, K = X.shape
    if out is None:
        out = torch.empty_like(X)
    _check(lib.w4_awq_scale_activations(_ptr(X), _ptr(s), M, K, _ptr(out), _stream()),
           "w4_awq_scale_activations")
    return out


def gptq_hessian(X):
    """H = 2 X^T X (fp32 [K, K]) for bf16 calibration activations X [n, K]."""
    _cuda(X, torch.bfloat16, "X")
    n, K = X.shape
    H = torch.empty((K, K), dtype=torch.float32, device=X.device)
    _check(lib.w4_gptq_hessian(_ptr(X), n, K, _ptr(H), _stream()), "w4_gptq_hessian")
    return H


def gptq_quantize(W, H, G, act_order=False, damp=0.01):
    """INT4 codes with GPTQ error compensation: (Wq, scales, zeros, g_idx)
    in the format of quantize_rtn (g_idx None without act-order)."""
    _cuda(W, torch.float32, "W")
    _cuda(H, torch.float32, "H")
    N, K = W.shape
    dev = W.device
    need = lib.w4_gptq_workspace_bytes(N, K, G)
    if need == 0:
        raise W4Error(W4_ERR_INVALID_ARG, "w4_gptq_workspace_bytes")
    ws = _ws_view(torch.empty(need + 256, dtype=torch.uint8, device=dev))
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    sc = torch.empty((N, K // G), dtype=torch.float16, device=dev)
    zr = torch.empty((N, K // G), dtype=torch.uint8, device=dev)
    gi = torch.empty(K, dtype=torch.int32, device=dev) if act_order else None
    _check(lib.w4_gptq_quantize(_ptr(W), _ptr(H), N, K, G, int(bool(act_order)), float(damp),
                                _ptr(Wq), _ptr(sc), _ptr(zr), _ptr(gi), _ptr(ws), ws.numel(),
                                _stream()), "w4_gptq_quantize")
    return Wq, sc, zr, gi


def llm_int8_quantize_weights(W):
    """fp32 W [N, K] -> (q_w int8 [N, K], s_w fp32 [N]), one scale per output row."""
    _cuda(W, torch.float32, "W")
    N, K = W.shape
    qw = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sw = torch.empty(N, dtype=torch.float32, device=W.device)
    _check(lib.llm_int8_quantize_weights(_ptr(W), N, K, _ptr(qw), _ptr(sw), _stream()),
           "llm_int8_quantize_weights")
    return qw, sw


def llm_int8_gemm(X, qw, sw, threshold=6.0, out=None, workspace=None):
    """Y = X . W^T by the LLM.int8 mixed decomposition (outliers |x| > threshold)."""
    _cuda(X, torch.bfloat16, "X")
    M, K = X.shape
    N = qw.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    need = lib.llm_int8_workspace_bytes(M, N, K)
    if need == 0:
        raise W4Error(W4_ERR_INVALID_ARG, "llm_int8_workspace_bytes")
    ws = _ws_view(workspace if workspace is not None else _WS_SCRATCH.get(need, X.device))
    _check(lib.llm_int8_gemm(_ptr(X), _ptr(qw), _ptr(sw), M, N, K, float(threshold), _ptr(out),
                             _ptr(ws), ws.numel(), _stream()), "llm_int8_gemm")
    return out


def dequant(Wq, scales, zeros, G, g_idx=None):
    N, K = Wq.shape[0], Wq.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.bfloat16, device=Wq.device)
    _check(lib.w4_dequant(_ptr(Wq), _ptr(scales), _ptr(zeros), _ptr(g_idx), N, K, G, _ptr(out),
                          _stream()), "w4_dequant")
    return out


def prepacked_bytes(N, K, G, act_order=False) -> int:
    return lib.w4_prepacked_bytes(N, K, G, int(bool(act_order)))


def prepack(Wq, scales, zeros, G, g_idx=None):
    N, K = Wq.shape[0], Wq.shape[1] * 2
    nbytes = prepacked_bytes(N, K, G, g_idx is not None)
    if nbytes == 0:
        raise W4Error(W4_ERR_INVALID_ARG, "w4_prepacked_bytes")
    Wp = torch.empty(nbytes, dtype=torch.uint8, device=Wq.device)
    _check(lib.w4_prepack(_ptr(Wq), _ptr(scales), _ptr(zeros), _ptr(g_idx), N, K, G, _ptr(Wp),
                          _stream()), "w4_prepack")
    return Wp


def unprepack(Wp, N, K, G, act_order=False):
    dev = Wp.device
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    sc = torch.empty((N, K // G), dtype=torch.float16, device=dev)
    zr = torch.empty((N, K // G), dtype=torch.uint8, device=dev)
    perm = torch.empty(K, dtype=torch.int32, device=dev) if act_order else None
    _check(lib.w4_unprepack(_ptr(Wp), N, K, G, int(bool(act_order)), _ptr(Wq), _ptr(sc),
                            _ptr(zr), _ptr(perm), _stream()), "w4_unprepack")
    return Wq, sc, zr, perm


class Workspace:
    """Per-device scratch buffer, zero-filled once when (re)allocated; the
    library leaves it zeroed after each call."""

    def __init__(self):
        self._buf = {}

    def get(self, nbytes: int, device) -> torch.Tensor:
        dev = torch.device(device)
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        buf = self._buf.get(key)
        if buf is None or buf.numel() < nbytes:
            size = max(nbytes, 1 << 20)
            buf = torch.zeros(size + 256, dtype=torch.uint8, device=dev)
            self._buf[key] = buf
        return buf


_WS = Workspace()
# scratch whose contents the library does not keep zeroed (LLM.int8): never
# the zero-kept workspace of the W4A16 / NF4 GEMMs
_WS_SCRATCH = Workspace()


def _ws_view(buf):
    off = (-buf.data_ptr()) % 256
    return buf[off:]


def workspace_bytes(M, N, K, G, act_order=False) -> int:
    return lib.w4_workspace_bytes(M, N, K, G, int(bool(act_order)))


def w4a16_gemm(X, Wp, N, K, G, act_order=False, out=None, workspace=None):
    """Y[M, N] = X . dequant(W)^T for bf16 X [M, K] and prepacked Wp."""
    _cuda(X, torch.bfloat16, "X")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    need = workspace_bytes(M, N, K, G, act_order)
    ws = _ws_view(workspace if workspace is not None else _WS.get(need, X.device))
    _check(lib.w4a16_gemm(_ptr(X), _ptr(Wp), M, N, K, G, int(bool(act_order)), _ptr(out),
                          _ptr(ws), ws.numel(), _stream()), "w4a16_gemm")
    return out


def w4a16_gemm_static_scratch(X, Wp, N, K, G, act_order=False, out=None):
    """w4a16_gemm with the library's static device scratch as workspace (the
    call allocates nothing); shapes needing more than W4_STATIC_SCRATCH_BYTES
    raise W4Error with status W4_ERR_SCRATCH_LIMIT."""
    _cuda(X, torch.bfloat16, "X")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _check(lib.w4a16_gemm_static_scratch(_ptr(X), _ptr(Wp), M, N, K, G, int(bool(act_order)),
                                         _ptr(out), _stream()), "w4a16_gemm_static_scratch")
    return out


def awq_workspace_bytes(M, N, K, G, act_order=False) -> int:
    return lib.w4_awq_workspace_bytes(M, N, K, G, int(bool(act_order)))


def w4a16_awq_gemm(X, s, Wp, N, K, G, act_order=False, out=None, workspace=None):
    """Y[M, N] = (X / s) . dequant(W s)^T for bf16 X [M, K], the AWQ factor
    s [K] and prepacked Wp of weights quantized after awq_scale_weights."""
    _cuda(X, torch.bfloat16, "X")
    _cuda(s, torch.float32, "s")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    need = awq_workspace_bytes(M, N, K, G, act_order)
    ws = _ws_view(workspace if workspace is not None else _WS.get(need, X.device))
    _check(lib.w4a16_awq_gemm(_ptr(X), _ptr(s), _ptr(Wp), M, N, K, G, int(bool(act_order)),
                              _ptr(out), _ptr(ws), ws.numel(), _stream()), "w4a16_awq_gemm")
    return out


# ----------------------------------------------------------------- NF4

def _levels(fn):
    buf = (ctypes.c_float * 16)()
    fn(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


def nf4_levels():
    return _levels(lib.nf4_levels)


def fp4_levels():
    return _levels(lib.fp4_levels)


def _blockwise_quantize(fn, name, W, blocksize, dq_group):
    _cuda(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    nb = N * K // blocksize
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    aq = torch.empty(nb, dtype=torch.uint8, device=dev)
    s2 = torch.empty((nb + dq_group - 1) // dq_group, dtype=torch.float32, device=dev)
    _check(fn(_ptr(W), N, K, blocksize, dq_group, _ptr(Wq), _ptr(aq), _ptr(s2), _stream()), name)
    return Wq, aq, s2


def _blockwise_dequant(fn, name, Wq, absmax_q, s2, dq_group, blocksize):
    N, K = Wq.shape[0], Wq.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.bfloat16, device=Wq.device)
    _check(fn(_ptr(Wq), _ptr(absmax_q), _ptr(s2), N, K, blocksize, dq_group, _ptr(out),
              _stream()), name)
    return out


def nf4_quantize(W, blocksize=64, dq_group=256):
    return _blockwise_quantize(lib.nf4_quantize, "nf4_quantize", W, blocksize, dq_group)


def nf4_dequant(Wq, absmax_q, s2, dq_group=256, blocksize=64):
    return _blockwise_dequant(lib.nf4_dequant, "nf4_dequant", Wq, absmax_q, s2, dq_group,
                              blocksize)


def nf4_quantize_meandq(W, blocksize=64, dq_group=256):
    """NF4 with mean-offset double quantization of the block constants:
    (Wq, absmax codes int8, run means fp32, s2 fp32)."""
    _cuda(W, torch.float32, "W")
    N, K = W.shape
    dev = W.device
    nb = N * K // blocksize
    runs = (nb + dq_group - 1) // dq_group
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    aq = torch.empty(nb, dtype=torch.int8, device=dev)
    mean = torch.empty(runs, dtype=torch.float32, device=dev)
    s2 = torch.empty(runs, dtype=torch.float32, device=dev)
    _check(lib.nf4_quantize_meandq(_ptr(W), N, K, blocksize, dq_group, _ptr(Wq), _ptr(aq),
                                   _ptr(mean), _ptr(s2), _stream()), "nf4_quantize_meandq")
    return Wq, aq, mean, s2


def nf4_dequant_meandq(Wq, absmax_q, mean, s2, dq_group=256, blocksize=64):
    N, K = Wq.shape[0], Wq.shape[1] * 2
    out = torch.empty((N, K), dtype=torch.bfloat16, device=Wq.device)
    _check(lib.nf4_dequant_meandq(_ptr(Wq), _ptr(absmax_q), _ptr(mean), _ptr(s2), N, K,
                                  blocksize, dq_group, _ptr(out), _stream()),
           "nf4_dequant_meandq")
    return out


def nf4_gemm_meandq(X, Wp, mean, s2, N, K, dq_group=256, out=None, workspace=None):
    """Y = X . w_hat^T for NF4 weights with mean-offset constants (Wp from
    nf4_prepack of the codes and the int8 constants)."""
    _cuda(X, torch.bfloat16, "X")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    need = nf4_workspace_bytes(M, N, K)
    ws = _ws_view(workspace if workspace is not None else _WS.get(need, X.device))
    _check(lib.nf4_gemm_meandq(_ptr(X), _ptr(Wp), _ptr(mean), _ptr(s2), M, N, K, dq_group,
                               _ptr(out), _ptr(ws), ws.numel(), _stream()), "nf4_gemm_meandq")
    return out


def fp4_quantize(W, blocksize=64, dq_group=256):
    """FP4 (E2M1 / 6) codes in the NF4 block-wise layout: (Wq, absmax codes, s2)."""
    return _blockwise_quantize(lib.fp4_quantize, "fp4_quantize", W, blocksize, dq_group)


def fp4_dequant(Wq, absmax_q, s2, dq_group=256, blocksize=64):
    return _blockwise_dequant(lib.fp4_dequant, "fp4_dequant", Wq, absmax_q, s2, dq_group,
                              blocksize)


def nf4_prepack(Wq, absmax_q):
    """Prepack NF4 or FP4 codes (the layout is shared)."""
    N, K = Wq.shape[0], Wq.shape[1] * 2
    nbytes = lib.nf4_prepacked_bytes(N, K)
    if nbytes == 0:
        raise W4Error(W4_ERR_INVALID_ARG, "nf4_prepacked_bytes")
    Wp = torch.empty(nbytes, dtype=torch.uint8, device=Wq.device)
    _check(lib.nf4_prepack(_ptr(Wq), _ptr(absmax_q), N, K, _ptr(Wp), _stream()), "nf4_prepack")
    return Wp


def nf4_workspace_bytes(M, N, K) -> int:
    return lib.nf4_workspace_bytes(M, N, K)


def _blockwise_gemm(fn, name, X, Wp, s2, N, K, dq_group, out, workspace):
    _cuda(X, torch.bfloat16, "X")
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    need = nf4_workspace_bytes(M, N, K)
    ws = _ws_view(workspace if workspace is not None else _WS.get(need, X.device))
    _check(fn(_ptr(X), _ptr(Wp), _ptr(s2), M, N, K, dq_group, _ptr(out), _ptr(ws), ws.numel(),
              _stream()), name)
    return out


def nf4_gemm(X, Wp, s2, N, K, dq_group=256, out=None, workspace=None):
    return _blockwise_gemm(lib.nf4_gemm, "nf4_gemm", X, Wp, s2, N, K, dq_group, out, workspace)


def fp4_gemm(X, Wp, s2, N, K, dq_group=256, out=None, workspace=None):
    """Y = X . w_hat^T for FP4 weights prepacked with nf4_prepack."""
    return _blockwise_gemm(lib.fp4_gemm, "fp4_gemm", X, Wp, s2, N, K, dq_group, out, workspace)


# ----------------------------------------------------------------- FP8 (e4m3)

FP8_BLOCK = 128
_E4M3 = torch.float8_e4m3fn
_BF16 = torch.bfloat16
_F32 = torch.float32
# The decode calls below take a few microseconds on the GPU, so their checks
# are kept cheap: pointers as plain integers, the stream without a Stream
# object, one comparison per property.


def _blocks(n):
    return (n + 127) >> 7


def _fp8_arg(t, dtype, shape, dev, name):
    """The address of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr()


def _fp8_first(t, dtype, dim, name):
    """Device index of a call's first tensor, which has to be the current
    device (the stream is that device's)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    if t.dtype is not dtype or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dim}-dimensional {dtype} tensor")
    return dev


def _fp8_out(out, shape, like, dev):
    if out is None:
        return torch.empty(*shape, dtype=_BF16, device=like.device)
    _fp8_arg(out, _BF16, shape, dev, "out")
    return out


_FP8_WS = {}
_FP8_COUNTER_BYTES = 65536 * 4


def _fp8_workspace(need, workspace, like, dev, stream):
    """(address, bytes, tensor) of the caller's workspace, or of one of this
    (device, stream), zeroed when it is made.  A call that is being captured
    into a graph gets its own, zeroed by the graph at each replay: graphs then
    share none.  The caller keeps the tensor until its kernels are launched:
    another thread may put a larger one in its place meanwhile, and memory given
    back before the launch could be handed to someone else ahead of it."""
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or workspace.get_device() != dev or \
                not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous torch.uint8 tensor on cuda:{dev}")
        buf = workspace
    elif torch.cuda.is_current_stream_capturing():
        buf = torch.empty(need + 256, dtype=torch.uint8, device=like.device)
        if need > _FP8_COUNTER_BYTES:  # (a call without partial sums counts nothing)
            buf[:_FP8_COUNTER_BYTES + 256].zero_()
    else:
        buf = _FP8_WS.get((dev, stream))
        if buf is None or buf.numel() < need + 256:
            buf = torch.zeros(max(need, 1 << 20) + 256, dtype=torch.uint8, device=like.device)
            _FP8_WS[dev, stream] = buf
    at = buf.data_ptr()
    skip = -at & 255
    return at + skip, max(0, buf.numel() - skip), buf


def fp8_quantize_weights(W):
    """fp32 W [N, K] or [..., N, K] -> (e4m3 codes of W's shape, fp32 scales
    [..., ceil(N/128), ceil(K/128)]), one scale per 128 x 128 block; K % 16 == 0."""
    if W.dim() < 2:
        raise ValueError("W must have at least two dimensions")
    dev = _fp8_first(W, _F32, W.dim(), "W")
    N, K = W.shape[-2:]
    B = W.numel() // (N * K) if N * K > 0 else 0
    qw = torch.empty_like(W, dtype=_E4M3)
    sw = torch.empty(W.shape[:-2] + (_blocks(N), _blocks(K)), dtype=_F32, device=W.device)
    _check(lib.fp8_quantize_weights(W.data_ptr(), B, N, K, qw.data_ptr(), sw.data_ptr(),
                                    _raw_stream(dev)), "fp8_quantize_weights")
    return qw, sw


def fp8_quantize_activations(X):
    """bf16 X [M, K] -> (e4m3 codes [M, K], fp32 scales [M, ceil(K/128)]), one
    scale per token and 128 channels; K % 16 == 0."""
    dev = _fp8_first(X, _BF16, 2, "X")
    M, K = X.shape
    qx = torch.empty_like(X, dtype=_E4M3)
    sx = torch.empty(M, _blocks(K), dtype=_F32, device=X.device)
    _check(lib.fp8_quantize_activations(X.data_ptr(), M, K, qx.data_ptr(), sx.data_ptr(),
                                        _raw_stream(dev)), "fp8_quantize_activations")
    return qx, sx


def fp8_add_rmsnorm(X, weight, residual=None, eps=1e-6, want_y=False, residual_out=None):
    """r = X + residual, y = r * rsqrt(mean(r^2) + eps) * weight for bf16 X
    [M, K] and weight [K]: (codes and scales of y as fp8_quantize_activations
    gives them, bf16 r or None without a residual, bf16 y or None unless
    want_y).  residual_out may be residual (in place)."""
    dev = _fp8_first(X, _BF16, 2, "X")
    M, K = X.shape
    w = _fp8_arg(weight, _BF16, (K,), dev, "weight")
    device = X.device
    res = res_out = None
    if residual is not None:
        res = _fp8_arg(residual, _BF16, X.shape, dev, "residual")
        if residual_out is None:
            residual_out = torch.empty_like(X)
            res_out = residual_out.data_ptr()
        else:
            res_out = _fp8_arg(residual_out, _BF16, X.shape, dev, "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    y = torch.empty_like(X) if want_y else None
    qy = torch.empty_like(X, dtype=_E4M3)
    sy = torch.empty(M, _blocks(K), dtype=_F32, device=device)
    _check(lib.fp8_add_rmsnorm(X.data_ptr(), res, w, eps, M, K, res_out,
                               None if y is None else y.data_ptr(), qy.data_ptr(), sy.data_ptr(),
                               _raw_stream(dev)), "fp8_add_rmsnorm")
    return qy, sy, residual_out, y


def fp8_gemm(qx, sx, qw, sw, out=None, workspace=None):
    """bf16 Y[M, N] = (qx sx) . (qw sw)^T for codes and scales as
    fp8_quantize_activations / fp8_add_rmsnorm and fp8_quantize_weights give them."""
    dev = _fp8_first(qx, _E4M3, 2, "qx")
    M, K = qx.shape
    N = qw.shape[0]
    w = _fp8_arg(qw, _E4M3, (N, K), dev, "qw")
    kb = _blocks(K)
    s1 = _fp8_arg(sx, _F32, (M, kb), dev, "sx")
    s2 = _fp8_arg(sw, _F32, (_blocks(N), kb), dev, "sw")
    out = _fp8_out(out, (M, N), qx, dev)
    need = lib.fp8_gemm_workspace_bytes(M, N, K)
    if need == 0:
        valid = M >= 1 and N >= 1 and K >= 16 and K % 16 == 0
        raise W4Error(W4_ERR_UNSUPPORTED if valid else W4_ERR_INVALID_ARG,
                      "fp8_gemm_workspace_bytes")
    stream = _raw_stream(dev)
    ws, ws_bytes, _held = _fp8_workspace(need, workspace, qx, dev, stream)
    _check(lib.fp8_gemm(qx.data_ptr(), s1, w, s2, M, N, K, out.data_ptr(), ws, ws_bytes, stream),
           "fp8_gemm")
    return out


def fp8_moe(X, router, w13, s13, w2, s2, top_k, renormalize=True, out=None, workspace=None):
    """A mixture-of-experts layer for up to 128 tokens: bf16 X [T, H], bf16
    router [E, H], gate and up weights w13 [E, 2, I, H] and down weights w2
    [E, H, I] with their scales as fp8_quantize_weights gives them ->
    (bf16 Y [T, H], int32 expert ids [T, top_k], their fp32 weights [T, top_k])."""
    dev = _fp8_first(X, _BF16, 2, "X")
    T, H = X.shape
    if w13.dim() != 4:
        raise ValueError("w13 must have shape (E, 2, I, H)")
    E, _, I, _ = w13.shape
    hb, ib = _blocks(H), _blocks(I)
    r = _fp8_arg(router, _BF16, (E, H), dev, "router")
    p13 = _fp8_arg(w13, _E4M3, (E, 2, I, H), dev, "w13")
    q13 = _fp8_arg(s13, _F32, (E, 2, ib, hb), dev, "s13")
    p2 = _fp8_arg(w2, _E4M3, (E, H, I), dev, "w2")
    q2 = _fp8_arg(s2, _F32, (E, hb, ib), dev, "s2")
    need = lib.fp8_moe_workspace_bytes(T, E, top_k, H, I)
    if need == 0:
        supported = T <= 128 and E <= 512 and top_k <= 16 and H <= 1 << 19 and I <= 1 << 19
        raise W4Error(W4_ERR_INVALID_ARG if supported else W4_ERR_UNSUPPORTED,
                      "fp8_moe_workspace_bytes")
    out = _fp8_out(out, (T, H), X, dev)
    ids = torch.empty(T, top_k, dtype=torch.int32, device=X.device)
    weights = torch.empty(T, top_k, dtype=_F32, device=X.device)
    stream = _raw_stream(dev)
    ws, ws_bytes, _held = _fp8_workspace(need, workspace, X, dev, stream)
    _check(lib.fp8_moe(X.data_ptr(), r, p13, q13, p2, q2, T, E, top_k, H, I,
                       1 if renormalize else 0, out.data_ptr(), ids.data_ptr(),
                       weights.data_ptr(), ws, ws_bytes, stream), "fp8_moe")
    return out, ids, weights
