"""Binding of the 8-bit floating-point entry points of include/w8a8.h: rows to e4m3
with scales (plain, of a SwiGLU, or behind an RMS norm), and the products on them,
dense and by expert.  Argument marshalling only, as in binding.py and moe.py: every
function keeps the name of the C entry point it calls, device buffers are PyTorch
tensors, and there is no fallback.

    n = w8a8_rms_norm(X, weight, residual=residual)
    G = w8a8_gemm(n.codes, n.scales, gate_up, gate_up_scales)
    h = w8a8_quantize(G, swiglu=True)
    Y = w8a8_gemm(h.codes, h.scales, down, down_scales)

Codes are torch.float8_e4m3fn (uint8 is taken as well), scales fp32, one for 128
neighbouring features of a row or 128 x 128 weights.  Outputs that are not passed are
allocated on the stream the call runs on.  Every call runs on its tensors' device,
whichever is current.
"""

from __future__ import annotations

from collections import namedtuple

import numpy as np

from .binding import W4A16_OK, W4A16Error, load
from .moe import _code

BLOCK = 128
W8A8_KERNEL_SKINNY = 1
W8A8_KERNEL_TILE = 2

# codes [M][K], scales fp32 [M][ceil(K / 128)]
W8A8Rows = namedtuple("W8A8Rows", "codes scales")
# codes and scales as W8A8Rows, Y (the normed rows) and H (X + residual) [M][K]; None: not made
W8A8Norm = namedtuple("W8A8Norm", "codes scales Y H", defaults=(None, None))

_torch = None  # imported by the first call


def _types():
    """torch, and the dtypes of codes, once it is imported."""
    global _torch, _E4M3, _I32, _F32
    if _torch is None:
        import torch
        _E4M3 = (torch.float8_e4m3fn, torch.uint8)
        _I32, _F32 = (torch.int32,), (torch.float32,)
        _torch = torch
    return _torch


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _check(t, dtypes, shape, name, index):
    """The address of t: a contiguous tensor of one of `dtypes` and of `shape` (any if
    None) on ROCm device `index`.  One condition for the tensors that are in order: a call
    takes up to seven, and a small kernel no longer than its arguments' checks."""
    try:
        if (t.get_device() == index and t.dtype in dtypes and
                (shape is None or t.shape == shape) and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a tensor on a ROCm device")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, not on device {index}")


def _elsewhere(device, index, stream):
    """None where the call's stream is the current one of the current device; else a context
    in which it is."""
    if stream is None:
        return None if _torch._C._cuda_getDevice() == index else _torch.cuda.device(index)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return _torch.cuda.stream(stream)


def _rows_2d(X, dtypes=None):
    """(address, rows, features, device index) of a 2-D X of one of `dtypes`, or of any that
    activations have."""
    if not getattr(X, "is_cuda", False):
        raise TypeError("X must be a tensor on a ROCm device")
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    index = X.get_device()
    return (_check(X, dtypes or (X.dtype,), None, "X", index), *X.shape, index)


def w8a8_quantize_weights(W: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """Host quantizer: W fp32 [N][K] -> (codes uint8 [N][K] (e4m3), scales fp32
    [ceil(N/128)][ceil(K/128)])."""
    W = np.ascontiguousarray(W)
    if W.dtype != np.float32 or W.ndim != 2:
        raise TypeError("W must be a 2-D float32 array")
    N, K = W.shape
    codes = np.empty((N, K), dtype=np.uint8)
    scales = np.empty((_blocks(N), _blocks(K)), dtype=np.float32)
    st = load().w8a8_quantize_weights(W.ctypes.data, codes.ctypes.data, scales.ctypes.data, N, K,
                                      BLOCK)
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_quantize_weights")
    return codes, scales


def _new_rows(M, K, device):
    return (_torch.empty((M, K), dtype=_E4M3[0], device=device),
            _torch.empty((M, _blocks(K)), dtype=_F32[0], device=device))


def w8a8_quantize(X, swiglu: bool = False, num_rows=None, out=None, stream=None) -> W8A8Rows:
    """Rows X [M][K] (fp32, fp16 or bf16) to e4m3 with a scale per 128 features;
    with `swiglu` silu(gate) * up of rows X [M][2K] = [gate | up].  num_rows (int32
    device tensor of one element): rows behind it are left as they were."""
    _types()
    x, M, K, index = _rows_2d(X)
    context = _elsewhere(X.device, index, stream)
    if context is not None:
        with context:
            return w8a8_quantize(X, swiglu, num_rows, out)
    code = _code(X.dtype)
    if swiglu:
        if K % 2:
            raise ValueError("rows of gate and up need an even number of features")
        K //= 2
    num = None
    if num_rows is not None:
        num = _check(num_rows, _I32, None, "num_rows", index)
        if num_rows.numel() != 1:
            raise ValueError("num_rows must have one element")
    if out is None:
        out = W8A8Rows(*_new_rows(M, K, X.device))
    st = load().w8a8_quantize(
        x, num, _check(out[0], _E4M3, (M, K), "codes", index),
        _check(out[1], _F32, (M, _blocks(K)), "scales", index), M, K, bool(swiglu), code,
        _torch._C._cuda_getCurrentRawStream(index))
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_quantize")
    return out


def w8a8_rms_norm(X, weight, residual=None, eps: float = 1e-6, normed: bool = False,
                  quantized: bool = True, out=None, stream=None) -> W8A8Norm:
    """h = X + residual, y = h * weight / sqrt(mean(h^2) + eps); returns y in e4m3
    (codes and scales), y itself where `normed` (Y), and h where there is a residual (H).
    X, residual [M][K] fp32, fp16 or bf16; weight [K] of the same type or fp32.  `out`, a
    W8A8Norm, gives the buffers; what is None in it is not made.  out.H may be `residual`
    or X, which are then updated in place."""
    torch = _types()
    x, M, K, index = _rows_2d(X)
    context = _elsewhere(X.device, index, stream)
    if context is not None:
        with context:
            return w8a8_rms_norm(X, weight, residual, eps, normed, quantized, out)
    code, own = _code(X.dtype), (X.dtype,)
    w = _check(weight, (X.dtype, torch.float32), (K,), "weight", index)
    r = None if residual is None else _check(residual, own, (M, K), "residual", index)
    if out is None:
        codes, scales = _new_rows(M, K, X.device) if quantized else (None, None)
        out = W8A8Norm(codes, scales, torch.empty_like(X) if normed else None,
                       torch.empty_like(X) if residual is not None else None)
    codes, scales, Y, H = out
    st = load().w8a8_rms_norm(
        x, r, w, None if H is None else _check(H, own, (M, K), "H", index),
        None if Y is None else _check(Y, own, (M, K), "Y", index),
        None if codes is None else _check(codes, _E4M3, (M, K), "codes", index),
        None if scales is None else _check(scales, _F32, (M, _blocks(K)), "scales", index),
        M, K, eps, code, _code(weight.dtype), _torch._C._cuda_getCurrentRawStream(index))
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_rms_norm")
    return out


def w8a8_kernel(R: int, E: int = 0) -> int:
    """Kernel of w8a8_gemm for R rows, or of w8a8_gemm_grouped for R slots over E experts
    (W8A8_KERNEL_*), 0 for extents they refuse."""
    return load().w8a8_kernel(R, E)


def _out(Y, shape, dtype, device, index):
    """(Y, its address), allocated if None"""
    if Y is None:
        Y = _torch.empty(shape, dtype=dtype or _torch.bfloat16, device=device)
        return Y, Y.data_ptr()
    return Y, _check(Y, (Y.dtype if dtype is None else dtype,), shape, "Y", index)


def w8a8_gemm(X, scales, weight, weight_scales, Y=None, dtype=None, stream=None):
    """Y [M][N] = X . W^T on e4m3 codes X [M][K] and weight [N][K] with scales
    [M][ceil(K/128)] and weight_scales [ceil(N/128)][ceil(K/128)], summed in fp32.  Y is
    fp32, fp16 or bf16: that of `Y`, or `dtype` (bf16 if neither is given)."""
    _types()
    x, M, K, index = _rows_2d(X, _E4M3)
    context = _elsewhere(X.device, index, stream)
    if context is not None:
        with context:
            return w8a8_gemm(X, scales, weight, weight_scales, Y, dtype)
    KB = _blocks(K)
    xs = _check(scales, _F32, (M, KB), "scales", index)
    w = _check(weight, _E4M3, None, "weight", index)
    if weight.dim() != 2 or weight.shape[1] != K:
        raise ValueError(f"weight shape {tuple(weight.shape)} does not take {K} features")
    N = weight.shape[0]
    ws = _check(weight_scales, _F32, (_blocks(N), KB), "weight_scales", index)
    Y, y = _out(Y, (M, N), dtype, X.device, index)
    st = load().w8a8_gemm(x, xs, w, ws, y, M, N, K, BLOCK, _code(Y.dtype),
                          _torch._C._cuda_getCurrentRawStream(index))
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_gemm")
    return Y


def w8a8_gemm_grouped(X, scales, token_index, expert_offsets, weight, weight_scales, Y=None,
                      dtype=None, stream=None):
    """Y[r] = X[token_index[r]] . W_e^T for every slot r of every expert e (the lists of
    w4a16_moe_route); token_index None: slot r reads row r.  weight [E][N][K] e4m3,
    weight_scales [E][ceil(N/128)][ceil(K/128)]; Y [R][N] as in w8a8_gemm.  Rows of Y
    behind expert_offsets[E] are left as they were."""
    _types()
    x, T, K, index = _rows_2d(X, _E4M3)
    context = _elsewhere(X.device, index, stream)
    if context is not None:
        with context:
            return w8a8_gemm_grouped(X, scales, token_index, expert_offsets, weight,
                                     weight_scales, Y, dtype)
    KB = _blocks(K)
    xs = _check(scales, _F32, (T, KB), "scales", index)
    if token_index is None:
        R, tokens = T, None
    else:
        tokens = _check(token_index, _I32, None, "token_index", index)
        R = token_index.numel()
    w = _check(weight, _E4M3, None, "weight", index)
    if weight.dim() != 3 or weight.shape[2] != K:
        raise ValueError(f"weight shape {tuple(weight.shape)} does not take {K} features")
    E, N = weight.shape[:2]
    ws = _check(weight_scales, _F32, (E, _blocks(N), KB), "weight_scales", index)
    offsets = _check(expert_offsets, _I32, None, "expert_offsets", index)
    if expert_offsets.numel() != E + 1:
        raise ValueError("expert_offsets must have E + 1 entries")
    Y, y = _out(Y, (R, N), dtype, X.device, index)
    st = load().w8a8_gemm_grouped(x, xs, tokens, offsets, w, ws, y, T, R, E, N, K, BLOCK,
                                  _code(Y.dtype), _torch._C._cuda_getCurrentRawStream(index))
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_gemm_grouped")
    return Y
