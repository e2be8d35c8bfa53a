"""Plain NumPy definition of the 8-bit floating-point operators: e4m3, rows and
weights with scales, the RMS norm, the products.  fp64 throughout (the weights'
quantizer in its stated fp32 steps); imports nothing from the product."""

from __future__ import annotations

import numpy as np

from .moe_ref import HALF_STEP, SMALLEST

BLOCK = 128
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -126
U = 2.0 ** -24  # fp32's unit roundoff


def _table():
    """Value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -mag if c >> 7 else mag
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = _table()


def blocks(n):
    return -(-n // BLOCK)


def e4m3_step(q):
    """Spacing of the e4m3 values in the binade of |q|."""
    q = np.clip(np.abs(q), 2.0 ** -6, E4M3_MAX)
    return 2.0 ** (np.floor(np.log2(q)) - 3)


def e4m3_codes(q):
    """Codes (uint8) of the nearest e4m3 values, ties to even, magnitudes past 448 to 448."""
    q = np.asarray(q, dtype=np.float64)
    mags = E4M3[:127]
    a = np.minimum(np.abs(q), E4M3_MAX)
    hi = np.clip(np.searchsorted(mags, a, side="left"), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    # neighbouring codes: the even one has an even mantissa
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | (np.signbit(q).astype(np.uint8) << 7)


def wide(scales, K):
    """One scale a feature from one a block."""
    return np.repeat(np.asarray(scales, np.float64), BLOCK, axis=-1)[..., :K]


def row_values(codes, scales):
    codes = np.asarray(codes)
    return E4M3[codes] * wide(scales, codes.shape[-1])


def weight_values(codes, scales):
    codes = np.asarray(codes)
    w = wide(scales, codes.shape[-1])
    return E4M3[codes] * np.repeat(w, BLOCK, axis=-2)[..., :codes.shape[-2], :]


def row_scales(v):
    """Scale of every 128 features of rows v, NaN where one is not finite."""
    v = np.asarray(v, np.float64)
    M, K = v.shape
    s = np.empty((M, blocks(K)))
    for b in range(blocks(K)):
        part = np.abs(v[:, b * BLOCK:(b + 1) * BLOCK])
        a = part.max(1)
        s[:, b] = np.where(a == 0, 0.0, np.maximum(a / E4M3_MAX, LEAST_SCALE))
        s[~np.all(np.isfinite(part), axis=1), b] = np.nan
    return s


def quantize_weights(W):
    """(codes uint8 [N][K], scales fp32 [NB][KB]) in the library's fp32 steps."""
    W = np.asarray(W, np.float32)
    N, K = W.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            a = np.abs(W[at]).max()
            if a == 0:
                continue
            s = np.maximum(np.float32(a) / np.float32(448), np.float32(LEAST_SCALE))
            scales[i, j] = s
            codes[at] = e4m3_codes((W[at] / s).astype(np.float32))
    return codes, scales


def swiglu_rows(x):
    x = np.asarray(x, np.float64)
    K = x.shape[1] // 2
    with np.errstate(over="ignore", invalid="ignore"):
        return x[:, :K] / (1.0 + np.exp(-x[:, :K])) * x[:, K:]


def rms_norm(x, weight, residual=None, eps=1e-6):
    """(y, h) in fp64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return y, h


def check_rows(codes, scales, v, dv):
    """Asserts that (codes, scales) are rows v (fp64, known to dv, elementwise) in e4m3:
    a scale is a fp32 quotient of a largest magnitude known to dv; a code is the
    nearest one to v / scale but for three roundings of 2^-24 and dv / scale."""
    v, scales = np.asarray(v, np.float64), np.asarray(scales, np.float64)
    K = v.shape[1]
    want = row_scales(v)
    most = np.stack([np.max(dv[:, b * BLOCK:(b + 1) * BLOCK], 1) for b in range(blocks(K))], 1)
    bad = np.isnan(want)
    assert np.array_equal(bad, np.isnan(scales)), "scales that are NaN"
    # the scale jumps from 0 to its least as the largest magnitude leaves 0: a run whose
    # every |v| is at most its dv may hold nothing but zeros
    none = np.stack([np.all(np.abs(v[:, b * BLOCK:(b + 1) * BLOCK]) <=
                            dv[:, b * BLOCK:(b + 1) * BLOCK], 1) for b in range(blocks(K))], 1)
    want = np.where(none & (scales == 0), 0.0, want)
    err = np.abs(np.where(bad, 0.0, scales - want))
    assert np.all(err <= np.where(bad, 0.0, U * want + most / E4M3_MAX * (1 + U))), \
        f"scales: worst {np.max(err / np.maximum(want, LEAST_SCALE)):.3e}"
    got, s = E4M3[np.asarray(codes)], wide(scales, K)
    assert np.array_equal(np.isnan(got), np.isnan(s)), "codes that are NaN"
    live = ~np.isnan(s) & (s > 0)
    assert np.all(got[s == 0] == 0)
    q = np.where(live, v / np.where(live, s, 1.0), 0.0)
    tol = e4m3_step(np.maximum(np.abs(q), np.abs(np.where(live, got, 0.0)))) / 2 \
        + 3 * U * np.abs(q) + dv / np.where(live, s, 1.0)
    off = np.abs(np.where(live, got - q, 0.0))
    assert np.all(off <= np.where(live, tol, 0.0)), f"codes: worst {np.max(off / tol):.6f} of bound"


# The products.  Every product of two e4m3 values is exact in fp32.
#   fp32 sums: a chain of at most 128 additions a block, each off by at most one
#   unit 2^-23 of the sum of magnitudes (whichever way the matrix units round), one
#   rounding each for the scales' product, its FMA and the addition of the waves' sums:
#   (2 * 128 + KB + 4) 2^-24 sum |x w|.
#   Window: the fp8 instructions add 8 products cut off at 2^-13 of the largest's power
#   of two, so that 7 of them lose at most 7 * 2^-13 sum |x w|.
WINDOW = 7 * 2.0 ** -13


def bound(abs_sum, want, K, dtype, window):
    tol = ((2 * BLOCK + blocks(K) + 4) * U + (WINDOW if window else 0.0)) * abs_sum
    return tol + HALF_STEP[dtype] * (np.abs(want) + tol) + SMALLEST[dtype]


def gemm(codes, scales, W, ws):
    """(Y, sum |x w|) in fp64."""
    x, w = row_values(codes, scales), weight_values(W, ws)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def grouped(codes, scales, token_index, offsets, W, ws, R):
    """(Y, sum |x w|) [R][N] in fp64, zeros behind the last slot."""
    N = W.shape[1]
    y, mag = np.zeros((R, N)), np.zeros((R, N))
    for e in range(W.shape[0]):
        r = np.arange(offsets[e], offsets[e + 1])
        if len(r):
            at = r if token_index is None else np.asarray(token_index)[r]
            y[r], mag[r] = gemm(codes[at], scales[at], W[e], ws[e])
    return y, mag
