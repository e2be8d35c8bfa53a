"""Binding of the mixture-of-experts entry points: routing of tokens to
experts, the experts' fused gate/up projection, and their down projections
combined back into the tokens.  Argument marshalling only, as in binding.py:
every function keeps the name of the C entry point it calls, device buffers are
PyTorch tensors, and there is no fallback.

    r = w4a16_moe_route(logits, topk)
    H = w4a16_gemm_grouped_swiglu(X, r.token_index, r.expert_offsets, gate_up, gate_up_scales)
    Y = w4a16_gemm_grouped_combine(H, r.expert_offsets, down, down_scales, r.slots, r.weights)

Outputs and workspaces that are not passed are allocated on the stream the call
runs on.  Every call runs on its tensors' device, whichever is current.
"""

from __future__ import annotations

import contextlib
from collections import namedtuple

from .binding import GROUP, W4A16_OK, W4A16Error, load

W4A16_DTYPE_F32 = 0
W4A16_DTYPE_F16 = 1
W4A16_DTYPE_BF16 = 2
W4A16_SCORE_SOFTMAX = 0
W4A16_SCORE_SIGMOID = 1
W4A16_EXPERTS_SKINNY = 1
W4A16_EXPERTS_TILE = 2

_SCORES = {"softmax": W4A16_SCORE_SOFTMAX, "sigmoid": W4A16_SCORE_SIGMOID,
           W4A16_SCORE_SOFTMAX: W4A16_SCORE_SOFTMAX, W4A16_SCORE_SIGMOID: W4A16_SCORE_SIGMOID}
_CODES = None

# ids, weights, slots: [T][topk]; token_index: [T * topk]; expert_offsets: [E + 1]
W4A16Routing = namedtuple("W4A16Routing", "ids weights slots token_index expert_offsets")


def _code(dtype):
    """W4A16_DTYPE_* of a torch dtype."""
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.float32: W4A16_DTYPE_F32, torch.float16: W4A16_DTYPE_F16,
                  torch.bfloat16: W4A16_DTYPE_BF16}
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"activations must be float32, float16 or bfloat16, not {dtype}")
    return code


def _tensor(t, dtype, name, device=None):
    """t, checked: a contiguous tensor of `dtype` on `device` (any ROCm device if None)."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a tensor on a ROCm device")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t


_HERE = contextlib.nullcontext()


def _launch(device, stream):
    """(stream handle, context) of one call: in the context the device is current and
    new tensors belong to the stream."""
    import torch
    if stream is None:
        # the current stream's handle alone: a torch.cuda.Stream object of it takes
        # 1.7 us more, as long as a small kernel
        here = torch.cuda.current_device() == device.index
        return (torch._C._cuda_getCurrentRawStream(device.index),
                _HERE if here else torch.cuda.device(device))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def _workspace(workspace, device, need, *extents):
    """(tensor, address, bytes): the caller's, whose size the entry point checks, or a
    new one of need(*extents) bytes"""
    import torch
    if workspace is None:
        size = need(*extents)
        if not size:
            return None, None, 0
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        _tensor(workspace, torch.uint8, "workspace", device)
    return workspace, workspace.data_ptr(), workspace.numel()


def _pointer(t):
    return None if t is None else t.data_ptr()


def w4a16_moe_route_workspace_bytes(T: int, E: int, topk: int) -> int:
    return int(load().w4a16_moe_route_workspace_bytes(T, E, topk))


def w4a16_moe_routing(T: int, E: int, topk: int, device="cuda") -> W4A16Routing:
    """Uninitialised buffers for w4a16_moe_route(..., out=...)."""
    import torch
    i32 = dict(dtype=torch.int32, device=device)
    return W4A16Routing(torch.empty(T, topk, **i32),
                        torch.empty(T, topk, dtype=torch.float32, device=device),
                        torch.empty(T, topk, **i32), torch.empty(T * topk, **i32),
                        torch.empty(E + 1, **i32))


def w4a16_moe_route(logits, topk: int, bias=None, score="softmax", groups: int = 1,
                    group_limit: int = 1, group_top: int = 1, renormalize: bool = True,
                    scale: float = 1.0, num_tokens=None, out=None, workspace=None, stream=None):
    """Route tokens to their `topk` experts (logits [T][E], fp32, fp16 or bf16) and
    build the slot lists; returns a W4A16Routing (`out` if given).

    score "softmax" or "sigmoid"; bias fp32 [E] is added to the scores for the
    choice only; experts come from `group_limit` of `groups` groups valued by
    their `group_top` largest keys; weights are the scores of the chosen,
    divided by their sum if `renormalize`, times `scale`.  num_tokens (int32
    device tensor of one element) marks the tokens behind it as padding."""
    import torch
    logits = _tensor(logits, None, "logits")
    code, device = _code(logits.dtype), logits.device
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    T, E = logits.shape
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r}")
    if not 1 <= topk <= E:  # W4A16_ERR_ARG, before buffers are made for it
        raise W4A16Error(1, "w4a16_moe_route")
    if bias is not None and tuple(_tensor(bias, torch.float32, "bias", device).shape) != (E,):
        raise ValueError(f"bias shape {tuple(bias.shape)} != {(E,)}")
    if num_tokens is not None and \
            _tensor(num_tokens, torch.int32, "num_tokens", device).numel() != 1:
        raise ValueError("num_tokens must have one element")
    at, context = _launch(device, stream)
    with context:
        lib = load()
        ws, ws_at, ws_bytes = _workspace(workspace, device, lib.w4a16_moe_route_workspace_bytes,
                                         T, E, topk)
        if out is None:
            out = w4a16_moe_routing(T, E, topk, device)
        else:
            each = (T, topk)
            for name, t, dtype, shape in zip(
                    W4A16Routing._fields, out,
                    (torch.int32, torch.float32, torch.int32, torch.int32, torch.int32),
                    (each, each, each, (T * topk,), (E + 1,))):
                if _tensor(t, dtype, name, device).shape != shape:
                    raise ValueError(f"{name} shape {tuple(t.shape)} != {shape}")
        st = lib.w4a16_moe_route(
            logits.data_ptr(), _pointer(bias), _pointer(num_tokens), out[0].data_ptr(),
            out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), T, E,
            topk, _SCORES[score], groups, group_limit, group_top, int(bool(renormalize)), scale,
            code, ws_at, ws_bytes, at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w4a16_moe_route")
    return out


def w4a16_experts_kernel(R: int, E: int, dtype) -> int:
    """Kernel of the two products below for R slots over E experts (W4A16_EXPERTS_*)."""
    return load().w4a16_experts_kernel(R, E, _code(dtype))


def w4a16_grouped_swiglu_workspace_bytes(T: int, R: int, E: int, F: int, K: int, dtype) -> int:
    return int(load().w4a16_grouped_swiglu_workspace_bytes(T, R, E, F, K, _code(dtype)))


def _experts(qweight, scales, expert_offsets, K, device):
    """(E, rows) of the experts' weights, shapes checked against K features."""
    import torch
    qweight = _tensor(qweight, torch.int32, "qweight", device)
    scales = _tensor(scales, torch.float32, "scales", device)
    if qweight.dim() != 3 or scales.dim() != 3:
        raise ValueError("qweight and scales must be 3-D [E][N][...]")
    E, N, words = qweight.shape
    if 8 * words != K or K % GROUP or tuple(scales.shape) != (E, N, K // GROUP):
        raise ValueError(f"shapes disagree: {K} features, qweight {tuple(qweight.shape)}, "
                         f"scales {tuple(scales.shape)}")
    if _tensor(expert_offsets, torch.int32, "expert_offsets", device).numel() != E + 1:
        raise ValueError("expert_offsets must have E + 1 entries")
    return E, N


def w4a16_gemm_grouped_swiglu(X, token_index, expert_offsets, qweight, scales, H=None,
                              workspace=None, stream=None):
    """H[r] = silu(x . gate^T) * (x . up^T), x = X[token_index[r]], for every slot r of
    every expert; qweight [E][2F][K/8] and scales [E][2F][K/32] hold each expert's
    gate rows, then its up rows.  X [T][K] and H [R][F] are fp32, fp16 or bf16.
    Rows of H behind expert_offsets[E] are left as they were."""
    import torch
    X = _tensor(X, None, "X")
    code, device = _code(X.dtype), X.device
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    T, K = X.shape
    E, rows = _experts(qweight, scales, expert_offsets, K, device)
    if rows % 2:
        raise ValueError("the gate/up weights need an even number of rows")
    F = rows // 2
    R = _tensor(token_index, torch.int32, "token_index", device).numel()
    at, context = _launch(device, stream)
    with context:
        if H is None:
            H = torch.empty((R, F), dtype=X.dtype, device=device)
        elif tuple(_tensor(H, X.dtype, "H", device).shape) != (R, F):
            raise ValueError(f"H shape {tuple(H.shape)} != {(R, F)}")
        lib = load()
        ws, ws_at, ws_bytes = _workspace(
            workspace, device, lib.w4a16_grouped_swiglu_workspace_bytes, T, R, E, F, K, code)
        st = lib.w4a16_gemm_grouped_swiglu(
            X.data_ptr(), token_index.data_ptr(), expert_offsets.data_ptr(), qweight.data_ptr(),
            scales.data_ptr(), H.data_ptr(), T, R, E, F, K, GROUP, code, ws_at, ws_bytes, at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w4a16_gemm_grouped_swiglu")
    return H


def w4a16_grouped_combine_workspace_bytes(T: int, topk: int, E: int, N: int, K: int,
                                          dtype) -> int:
    return int(load().w4a16_grouped_combine_workspace_bytes(T, topk, E, N, K, _code(dtype)))


def w4a16_gemm_grouped_combine(H, expert_offsets, qweight, scales, slots, weights, Y=None,
                               workspace=None, stream=None):
    """Y[t] = sum_j weights[t][j] * (H[slots[t][j]] . W_e^T), e the expert that owns the
    slot; qweight [E][N][K/8], scales [E][N][K/32], H [T*topk][K] and Y [T][N] fp32,
    fp16 or bf16.  Slots below 0 add nothing."""
    import torch
    H = _tensor(H, None, "H")
    code, device = _code(H.dtype), H.device
    slots = _tensor(slots, torch.int32, "slots", device)
    weights = _tensor(weights, torch.float32, "weights", device)
    if H.dim() != 2 or slots.dim() != 2 or weights.shape != slots.shape:
        raise ValueError("H, slots and weights must be 2-D, slots and weights alike")
    T, topk = slots.shape
    R, K = H.shape
    if R != T * topk:
        raise ValueError(f"H has {R} rows, the slots take {T * topk}")
    E, N = _experts(qweight, scales, expert_offsets, K, device)
    at, context = _launch(device, stream)
    with context:
        if Y is None:
            Y = torch.empty((T, N), dtype=H.dtype, device=device)
        elif tuple(_tensor(Y, H.dtype, "Y", device).shape) != (T, N):
            raise ValueError(f"Y shape {tuple(Y.shape)} != {(T, N)}")
        lib = load()
        ws, ws_at, ws_bytes = _workspace(
            workspace, device, lib.w4a16_grouped_combine_workspace_bytes, T, topk, E, N, K, code)
        st = lib.w4a16_gemm_grouped_combine(
            H.data_ptr(), expert_offsets.data_ptr(), qweight.data_ptr(), scales.data_ptr(),
            slots.data_ptr(), weights.data_ptr(), Y.data_ptr(), T, topk, E, N, K, GROUP, code,
            ws_at, ws_bytes, at)
    if st != W4A16_OK:
        raise W4A16Error(st, "w4a16_gemm_grouped_combine")
    return Y
