"""A slot's result of the skinny kernel is its own: the same bits whatever else the batch holds."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from w8a8_cases import TYPES, codes_of, device, on, ref, same, scales_of  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    return device()


# experts' slots: of the last but one, 3 that are compared; in the first list nobody else has any
COUNTS = [(0, 0, 0, 0, 3, 0), (1, 0, 0, 0, 3, 0), (3, 2, 0, 1, 3, 5), (0, 17, 0, 0, 3, 9),
          (16, 1, 1, 1, 3, 2), (0, 0, 0, 0, 19, 0), (1, 1, 1, 1, 35, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K", [400, 4096, 8192, 12288])
@pytest.mark.parametrize("N", [2080, 200])
def test_other_slots_change_nothing(dev, N, K, dtype):
    rng = np.random.default_rng(N + K)
    E, mine = 6, 4
    w, ws = codes_of(rng, E, N, K), scales_of(rng, E, ref.blocks(N), ref.blocks(K))
    rows = 40
    x, xs = codes_of(rng, rows, K), scales_of(rng, rows, ref.blocks(K)) * np.float32(2.0 ** -16)
    X, XS, W, WS = on(dev, x, xs, w, ws)
    first = None
    for counts in COUNTS:
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        R = int(off[-1])
        assert pkg.w8a8_kernel(R, E) == pkg.W8A8_KERNEL_SKINNY
        index = rng.integers(0, rows, R).astype(np.int32)
        at = off[mine] + counts[mine] - 3  # the last 3 of the expert's slots: tokens 7, 0, 7
        index[at:at + 3] = (7, 0, 7)
        I, O = on(dev, index, off)
        got = pkg.w8a8_gemm_grouped(X, XS, I, O, W, WS, dtype=TYPES[dtype])[at:at + 3]
        assert same(got[0], got[2])
        if first is None:
            first = got
        assert same(got, first), counts


@pytest.mark.parametrize("K", [400, 4096, 8192])
def test_other_rows_change_nothing(dev, K):
    """Dense products of 1 to 4 rows."""
    rng = np.random.default_rng(K)
    N = 2080
    X, XS, W, WS = on(dev, codes_of(rng, 4, K), scales_of(rng, 4, ref.blocks(K)),
                      codes_of(rng, N, K), scales_of(rng, ref.blocks(N), ref.blocks(K)))
    all_ = pkg.w8a8_gemm(X, XS, W, WS, dtype=torch.float32)
    for m in range(4):
        one = slice(m, m + 1)
        assert same(pkg.w8a8_gemm(X[one], XS[one], W, WS, dtype=torch.float32), all_[one])
