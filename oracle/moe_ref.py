"""Plain NumPy definition of the mixture-of-experts layer around the grouped
GEMM: routing of tokens to experts, the slot lists, the experts' SwiGLU and the
combination of their down projections.  fp64 throughout, one token or one
expert at a time; imports nothing from the product."""

from __future__ import annotations

import numpy as np

from .w4a16_ref import (ABS_TOL, EPILOGUE_ULPS, GROUP, REL_TOL, SILU_LIPSCHITZ, abs_gemm, gemm,
                        silu, unpack)

# unit roundoff of the output types and the spacing of their smallest numbers
HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -24, "bf16": 2.0 ** -133}


def route(logits, topk, bias=None, score="softmax", groups=1, group_limit=1, group_top=1,
          renormalize=True, scale=1.0, num_tokens=None):
    """(ids int32 [T][topk], weights fp64 [T][topk]); -1 and 0 where no expert is left."""
    L = np.asarray(logits, dtype=np.float64)
    T, E = L.shape
    ids = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    live = T if num_tokens is None else min(max(int(num_tokens), 0), T)
    for t in range(live):
        x = np.where(np.isnan(L[t]), -np.inf, L[t])
        open_ = x > -np.inf
        if not open_.any():
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = 1.0 / (1.0 + np.exp(-x))
            else:
                p = np.where(x == x.max(), 1.0, np.exp(x - x.max()))
                s = np.where(open_, p, 0.0) / p[open_].sum()
            key = x.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
            # what groups are valued by
            worth = s if bias is None and group_top == 2 else key
        masked = ~open_ | np.isnan(key) | (key == -np.inf)
        if group_limit < groups:
            size = E // groups
            value = np.full(groups, -np.inf)
            for g in range(groups):
                part = [worth[e] for e in range(g * size, (g + 1) * size) if not masked[e]]
                if part:
                    value[g] = sum(sorted(part, reverse=True)[:group_top])
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:group_limit]
            for g in range(groups):
                if g not in best or value[g] == -np.inf:
                    masked[g * size:(g + 1) * size] = True
        order = sorted((e for e in range(E) if not masked[e]), key=lambda e: (-key[e], e))[:topk]
        total = s[order].sum()
        for j, e in enumerate(order):
            ids[t, j] = e
            share = (s[e] / total if total > 0 else 0.0) if renormalize else s[e]
            weights[t, j] = share * scale
    return ids, weights


def slot_lists(ids, E):
    """(slots [T][topk], token_index [T*topk], expert_offsets [E+1]) of the choices:
    slots sorted by expert, then token; -1 where there is none."""
    ids = np.asarray(ids)
    T, topk = ids.shape
    slots = np.full((T, topk), -1, np.int32)
    token_index = np.full(T * topk, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    r = 0
    for e in range(E):
        for t, j in np.argwhere(ids == e):
            slots[t, j], token_index[r] = r, t
            r += 1
        offsets[e + 1] = r
    return slots, token_index, offsets


def terms_bound(X, qweight, scales, dtype, tile=False):
    """Allowed error of the sums X . W^T, element by element: the GEMM's relative
    tolerance of the terms a kernel adds up, plus its absolute tolerance.  For
    bf16 the terms are x * scale * (q + 16) and x * scale * 24, q the nibble, or
    in the tile kernel x * w with the scale and w rounded to fp16."""
    if dtype != "bf16" or tile:
        rel = REL_TOL + (2.01 * HALF_STEP["fp16"] if dtype == "bf16" else 0.0)
        return rel * abs_gemm(X, qweight, scales) + ABS_TOL
    q = unpack(qweight).astype(np.float64)
    W = (q + 40.0) * np.repeat(np.abs(np.asarray(scales, np.float64)), GROUP, axis=1)
    return REL_TOL * (np.abs(np.asarray(X, np.float64)) @ W.T) + ABS_TOL


def rounded(Y, dtype):
    """Error of storing values of magnitude Y in the output type."""
    return HALF_STEP[dtype] * np.abs(Y) + SMALLEST[dtype]


def expert_rows(offsets, E):
    for e in range(E):
        if offsets[e + 1] > offsets[e]:
            yield e, slice(int(offsets[e]), int(offsets[e + 1]))


def experts_swiglu(X, token_index, offsets, qweight, scales, dtype, tile=False):
    """(H fp64 [R][F], allowed error): silu(x . gate^T) * (x . up^T) per slot."""
    X = np.asarray(X, np.float32)  # 16-bit activations are fp32 numbers too
    E, F = qweight.shape[0], qweight.shape[1] // 2
    H = np.zeros((len(token_index), F))
    tol = np.zeros_like(H)
    for e, r in expert_rows(offsets, E):
        x = X[np.asarray(token_index)[r]]
        y = gemm(x, qweight[e], scales[e])
        b = terms_bound(x, qweight[e], scales[e], dtype, tile)
        g, u, eg, eu = y[:, :F], y[:, F:], b[:, :F], b[:, F:]
        sg = np.abs(silu(g))
        H[r] = silu(g) * u
        tol[r] = (SILU_LIPSCHITZ * eg * (np.abs(u) + eu) + sg * eu +
                  EPILOGUE_ULPS * 2.0 ** -24 * (sg + SILU_LIPSCHITZ * eg) * (np.abs(u) + eu))
    return H, tol + rounded(np.abs(H) + tol, dtype)


def experts_combine(H, offsets, qweight, scales, slots, weights, dtype, tile=False):
    """(Y fp64 [T][N], allowed error): sum_j weights[t][j] * (H[slots[t][j]] . W_e^T)."""
    H = np.asarray(H, np.float32)
    weights = np.asarray(weights, np.float64)
    E, N = qweight.shape[0], qweight.shape[1]
    D = np.zeros((H.shape[0], N))
    tol = np.zeros_like(D)
    for e, r in expert_rows(offsets, E):
        D[r] = gemm(H[r], qweight[e], scales[e])
        tol[r] = terms_bound(H[r], qweight[e], scales[e], dtype, tile)
    T, topk = np.asarray(slots).shape
    Y, err, size = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        for j in range(topk):
            s = int(slots[t, j])
            if s >= 0:
                Y[t] += weights[t, j] * D[s]
                err[t] += abs(weights[t, j]) * tol[s]
                size[t] += np.abs(weights[t, j]) * (np.abs(D[s]) + tol[s])
    err += topk * 2.0 ** -24 * size  # topk fp32 FMAs, each rounded once
    return Y, err + rounded(np.abs(Y) + err, dtype)
