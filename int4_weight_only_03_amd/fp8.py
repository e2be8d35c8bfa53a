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
from .moe import _code, _launch, _pointer, _tensor

BLOCK = 128
W8A8_KERNEL_SKINNY = 1
W8A8_KERNEL_TILE = 2

# codes [M][K], scales fp32 [M][ceil(K / 128)]
W8A8Rows = namedtuple("W8A8Rows", "codes scales")
# codes and scales as W8A8Rows, Y (the normed rows) and H (X + residual) [M][K]; None: not made
W8A8Norm = namedtuple("W8A8Norm", "codes scales Y H", defaults=(None, None))

_E4M3 = None


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _e4m3(t, name, device=None):
    """t, checked: contiguous codes on `device` (any ROCm device if None)."""
    global _E4M3
    if _E4M3 is None:
        import torch
        _E4M3 = (torch.float8_e4m3fn, torch.uint8)
    _tensor(t, None, name, device)
    if t.dtype not in _E4M3:
        raise TypeError(f"{name} must be torch.float8_e4m3fn")
    return t


def _shaped(t, shape, name):
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
    return t


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
    import torch
    return (torch.empty((M, K), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((M, _blocks(K)), dtype=torch.float32, device=device))


def _check_rows(codes, scales, M, K, device):
    import torch
    _shaped(_e4m3(codes, "codes", device), (M, K), "codes")
    _shaped(_tensor(scales, torch.float32, "scales", device), (M, _blocks(K)), "scales")


def w8a8_quantize(X, swiglu: bool = False, num_rows=None, out=None, stream=None) -> W8A8Rows:
    """Rows X [M][K] (fp32, fp16 or bf16) to e4m3 with a scale per 128 features;
    with `swiglu` silu(gate) * up of rows X [M][2K] = [gate | up].  num_rows (int32
    device tensor of one element): rows behind it are left as they were."""
    import torch
    _tensor(X, None, "X")
    code, device = _code(X.dtype), X.device
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    if swiglu:
        if K % 2:
            raise ValueError("rows of gate and up need an even number of features")
        K //= 2
    if num_rows is not None and _tensor(num_rows, torch.int32, "num_rows", device).numel() != 1:
        raise ValueError("num_rows must have one element")
    at, context = _launch(device, stream)
    with context:
        if out is None:
            codes, scales = _new_rows(M, K, device)
            out = W8A8Rows(codes, scales)
        else:
            codes, scales = out
            _check_rows(codes, scales, M, K, device)
        st = load().w8a8_quantize(X.data_ptr(), _pointer(num_rows), codes.data_ptr(),
                                  scales.data_ptr(), M, K, int(bool(swiglu)), code, at)
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
    import torch
    _tensor(X, None, "X")
    code, device = _code(X.dtype), X.device
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    _shaped(_tensor(weight, None, "weight", device), (K,), "weight")
    if weight.dtype is not X.dtype and weight.dtype is not torch.float32:
        raise TypeError(f"weight must be {X.dtype} or torch.float32")
    if residual is not None:
        _shaped(_tensor(residual, X.dtype, "residual", device), (M, K), "residual")
    at, context = _launch(device, stream)
    with context:
        if out is None:
            codes, scales = _new_rows(M, K, device) if quantized else (None, None)
            out = W8A8Norm(codes, scales, torch.empty_like(X) if normed else None,
                           torch.empty_like(X) if residual is not None else None)
        else:
            codes, scales = out.codes, out.scales
            if codes is not None and scales is not None:
                _check_rows(codes, scales, M, K, device)
            for name, t in (("Y", out.Y), ("H", out.H)):
                if t is not None:
                    _shaped(_tensor(t, X.dtype, name, device), (M, K), name)
        st = load().w8a8_rms_norm(
            X.data_ptr(), _pointer(residual), weight.data_ptr(), _pointer(out.H), _pointer(out.Y),
            _pointer(codes), _pointer(scales), M, K, eps, code, _code(weight.dtype), at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_rms_norm")
    return out


def w8a8_kernel(R: int, E: int = 0) -> int:
    """Kernel of w8a8_gemm for R rows, or of w8a8_gemm_grouped for R slots over E experts
    (W8A8_KERNEL_*), 0 for extents they refuse."""
    return load().w8a8_kernel(R, E)


def _rows_in(X, scales):
    """(rows, features, device) of quantized rows."""
    import torch
    _e4m3(X, "X")
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, K = X.shape
    _shaped(_tensor(scales, torch.float32, "scales", X.device), (M, _blocks(K)), "scales")
    return M, K, X.device


def _out(Y, shape, dtype, device):
    import torch
    if Y is None:
        return torch.empty(shape, dtype=dtype or torch.bfloat16, device=device)
    _shaped(_tensor(Y, None, "Y", device), shape, "Y")
    if dtype is not None and Y.dtype is not dtype:
        raise TypeError(f"Y must be {dtype}")
    return Y


def w8a8_gemm(X, scales, weight, weight_scales, Y=None, dtype=None, stream=None):
    """Y [M][N] = X . W^T on e4m3 codes X [M][K] and weight [N][K] with scales
    [M][ceil(K/128)] and weight_scales [ceil(N/128)][ceil(K/128)], summed in fp32.  Y is
    fp32, fp16 or bf16: that of `Y`, or `dtype` (bf16 if neither is given)."""
    import torch
    M, K, device = _rows_in(X, scales)
    _e4m3(weight, "weight", device)
    if weight.dim() != 2 or weight.shape[1] != K:
        raise ValueError(f"weight shape {tuple(weight.shape)} does not take {K} features")
    N = weight.shape[0]
    _shaped(_tensor(weight_scales, torch.float32, "weight_scales", device),
            (_blocks(N), _blocks(K)), "weight_scales")
    at, context = _launch(device, stream)
    with context:
        Y = _out(Y, (M, N), dtype, device)
        st = load().w8a8_gemm(X.data_ptr(), scales.data_ptr(), weight.data_ptr(),
                              weight_scales.data_ptr(), Y.data_ptr(), M, N, K, BLOCK,
                              _code(Y.dtype), at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_gemm")
    return Y


def w8a8_gemm_grouped(X, scales, token_index, expert_offsets, weight, weight_scales, Y=None,
                      dtype=None, stream=None):
    """Y[r] = X[token_index[r]] . W_e^T for every slot r of every expert e (the lists of
    w4a16_moe_route); token_index None: slot r reads row r.  weight [E][N][K] e4m3,
    weight_scales [E][ceil(N/128)][ceil(K/128)]; Y [R][N] as in w8a8_gemm.  Rows of Y
    behind expert_offsets[E] are left as they were."""
    import torch
    T, K, device = _rows_in(X, scales)
    R = T if token_index is None else \
        _tensor(token_index, torch.int32, "token_index", device).numel()
    _e4m3(weight, "weight", device)
    if weight.dim() != 3 or weight.shape[2] != K:
        raise ValueError(f"weight shape {tuple(weight.shape)} does not take {K} features")
    E, N = weight.shape[:2]
    _shaped(_tensor(weight_scales, torch.float32, "weight_scales", device),
            (E, _blocks(N), _blocks(K)), "weight_scales")
    if _tensor(expert_offsets, torch.int32, "expert_offsets", device).numel() != E + 1:
        raise ValueError("expert_offsets must have E + 1 entries")
    at, context = _launch(device, stream)
    with context:
        Y = _out(Y, (R, N), dtype, device)
        st = load().w8a8_gemm_grouped(
            X.data_ptr(), scales.data_ptr(), _pointer(token_index), expert_offsets.data_ptr(),
            weight.data_ptr(), weight_scales.data_ptr(), Y.data_ptr(), T, R, E, N, K, BLOCK,
            _code(Y.dtype), at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w8a8_gemm_grouped")
    return Y
