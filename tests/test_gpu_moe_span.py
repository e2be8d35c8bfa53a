"""fp32 and bf16 rows whose magnitudes lie far apart in the experts' products."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from moe_cases import PER, big_kernel, close, codes_of, device, on  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    return device()


@pytest.mark.parametrize("per", PER)
@pytest.mark.parametrize("span", [20, 24, 26, 30])
def test_fp32_rows_of_wide_span(dev, span, per):
    """Rows whose largest entry lies 2^span above the others and meets zero weights:
    the sums' terms are the small ones alone."""
    E, N, K = 2, 40, 160
    rng = np.random.default_rng(span)
    T = 2 * per
    off = np.array([0, per, T], np.int32)
    qw = codes_of(rng, E, 2 * N, K)
    qw[..., 0] = (qw[..., 0] & ~15) | 8  # nibble 8 of k = 0: weight 0
    sc = (2.0 ** 14 * (0.5 + rng.random((E, 2 * N, K // 32)))).astype(np.float32)
    x = (rng.standard_normal((T, K)) * 2.0 ** -14).astype(np.float32)
    x[:, 0] = 2.0 ** (span - 14) * (1 + rng.random(T))
    tok = np.arange(T, dtype=np.int32)
    H = pkg.w4a16_gemm_grouped_swiglu(*on(dev, x, tok, off, qw, sc))
    want, tol = oracle.experts_swiglu(x, tok, off, qw, sc, "fp32")
    close(H, want, tol, f"swiglu 2^{span} {per}")
    w = rng.standard_normal((per, 2)).astype(np.float32)
    slots = np.stack([np.arange(per), per + np.arange(per)], 1).astype(np.int32)
    Y = pkg.w4a16_gemm_grouped_combine(*on(dev, x, off, qw, sc, slots, w))
    want, tol = oracle.experts_combine(x, off, qw, sc, slots, w, "fp32")
    close(Y, want, tol, f"combine 2^{span} {per}")


@pytest.mark.parametrize("per", [1, 6, 20, 40, 90])
@pytest.mark.parametrize("span", [20, 28, 34])
def test_bf16_rows_of_wide_span(dev, span, per):
    """bf16 rows of the same kind.  The tile kernel takes them as fp16 numbers of up to
    2^15, whose last place is 2^-24 or half of it off: 2^-39 of the row's largest for
    every other entry."""
    E, N, K = 2, 40, 160
    rng = np.random.default_rng(span)
    T = 2 * per
    off = np.array([0, per, T], np.int32)
    qw = codes_of(rng, E, N, K)
    qw[..., 0] = (qw[..., 0] & ~15) | 8  # nibble 8 of k = 0: weight 0
    sc = (2.0 ** 14 * (0.5 + rng.random((E, N, K // 32)))).astype(np.float32)
    x = rng.standard_normal((T, K)) * 2.0 ** -14
    x[:, 0] = 2.0 ** (span - 14) * (1 + rng.random(T))
    X = torch.from_numpy(x).bfloat16()
    xv = X.float().numpy()
    w = rng.standard_normal((per, 2)).astype(np.float32)
    slots = np.stack([np.arange(per), per + np.arange(per)], 1).astype(np.int32)
    tile = big_kernel(T, E, "bf16")
    Y = pkg.w4a16_gemm_grouped_combine(X.to(dev), *on(dev, off, qw, sc, slots, w))
    want, tol = oracle.experts_combine(xv, off, qw, sc, slots, w, "bf16", tile)
    if tile:
        lost = 2.0 ** -39 * np.abs(xv).max(1)  # of every entry of a row
        for t in range(per):
            for j in range(2):
                W = np.abs(oracle.unpack(qw[j]).astype(np.float64) - 8.0)
                sums = (W * np.repeat(np.abs(sc[j]).astype(np.float64), 32, axis=1)).sum(1)
                tol[t] += 1.01 * abs(w[t, j]) * lost[slots[t, j]] * sums
    close(Y, want, tol, f"bf16 2^{span} {per}")
