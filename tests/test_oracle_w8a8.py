"""The oracle of the 8-bit operators: e4m3 against PyTorch's conversion of its own, the
quantizers by their properties."""

import numpy as np
import pytest

import oracle

ref = oracle.w8a8
torch = pytest.importorskip("torch")


def test_codes_are_those_of_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.E4M3, want.astype(np.float64), equal_nan=True)
    # back, but for NaN
    ok = (codes & 0x7F) != 0x7F
    assert np.array_equal(ref.e4m3_codes(ref.E4M3[ok]), codes[ok])


def test_rounding_is_to_nearest_even():
    rng = np.random.default_rng(0)
    mags = ref.E4M3[:127]
    ties = (mags[:-1] + mags[1:]) / 2
    q = np.concatenate([ties, -ties, rng.uniform(-448, 448, 4000),
                        rng.uniform(-0.02, 0.02, 4000)]).astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_codes(q), want)
    assert np.array_equal(ref.e4m3_codes([449.0, -1e9]), [0x7E, 0xFE])


@pytest.mark.parametrize("N,K", [(1, 16), (130, 272), (256, 128)])
def test_weights_come_back_within_half_a_step(N, K):
    rng = np.random.default_rng(N)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    W[:, :16] *= 0
    codes, scales = ref.quantize_weights(W)
    assert codes.shape == (N, K) and scales.shape == (ref.blocks(N), ref.blocks(K))
    s = np.repeat(ref.wide(scales, K), 128, 0)[:N]
    off = np.abs(ref.weight_values(codes, scales) - W)
    assert np.all(off <= s * (ref.e4m3_step(W / np.where(s > 0, s, 1)) / 2 * (1 + 2.0 ** -20)))


def test_products_of_whole_numbers():
    rng = np.random.default_rng(3)
    x, w = rng.integers(-8, 9, (5, 144)), rng.integers(-8, 9, (130, 144))
    xs, ws = np.array([[1.0, 2.0]] * 5), np.array([[1.0, 0.5], [4.0, 1.0]])
    y, mag = ref.gemm(ref.e4m3_codes(x), xs, ref.e4m3_codes(w), ws)
    X = x * np.where(np.arange(144) < 128, 1, 2)
    Wd = w * np.where(np.arange(130)[:, None] < 128, np.where(np.arange(144) < 128, 1, 0.5),
                      np.where(np.arange(144) < 128, 4, 1))
    assert np.array_equal(y, X @ Wd.T) and np.array_equal(mag, np.abs(X) @ np.abs(Wd).T)
    y2, _ = ref.grouped(ref.e4m3_codes(x), xs, [4, 0, 0], [0, 2, 2],
                        np.stack([ref.e4m3_codes(w)] * 2), np.stack([ws] * 2), 3)
    assert np.array_equal(y2[:2], (X @ Wd.T)[[4, 0]]) and not y2[2].any()
