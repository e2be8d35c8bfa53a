"""fp32 rows whose magnitudes lie far apart in the experts' products."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from moe_cases import PER, close, codes_of, device, on  # noqa: E402


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
