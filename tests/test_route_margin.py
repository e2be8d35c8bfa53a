"""The routing kernel's test for groups that fp32 keys cannot tell apart, emulated in
NumPy (CPU only): a token it lets pass keeps the groups that 64-bit keys keep, however
large the biases and whatever their signs."""

import numpy as np
import pytest

UNIT = 2.0 ** -24


def kept(worth, limit):
    """The `limit` groups of the largest worth, ties to the lowest index."""
    best = np.argsort(-worth, axis=1, kind="stable")[:, :limit]
    mask = np.zeros(worth.shape, bool)
    np.put_along_axis(mask, best, True, 1)
    return mask


def worth(key, top):
    """(worth of every group, sum of the magnitudes it was added from)"""
    best = np.sort(key, -1)[..., -top:]
    return best.sum(-1, dtype=key.dtype), np.abs(best).sum(-1)


def tokens(bias, top, groups, seed, size=4, T=20000):
    """Keys of T tokens in fp32 (scores off by up to 5 units) and in 64 bits: one
    expert of each group favoured by `bias`, the others disfavoured by it."""
    rng = np.random.default_rng(seed)
    E = groups * size
    s = 1 / (1 + np.exp(-1.5 * rng.standard_normal((T, E))))
    b = np.where(np.arange(E) % size == 0, bias, -bias) + 0.1 * rng.standard_normal(E)
    b = b.astype(np.float32)
    off = s + UNIT * rng.uniform(-4, 4, s.shape)  # and at most one more by its own rounding
    shape = (T, groups, size)
    return ((off.astype(np.float32) + b).reshape(shape),
            (s + b.astype(np.float64)).reshape(shape))


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("groups,limit", [(8, 4), (32, 9)])
@pytest.mark.parametrize("bias", [0.0, 1.0, 64.0, 1e3, 1e4, 1e5, 1e6, -1e4])
def test_tokens_let_pass_keep_the_groups_of_64_bit_keys(bias, top, groups, limit):
    k32, k64 = tokens(bias, top, groups, int(abs(bias)) + groups)
    w32, size = worth(k32, top)
    mine, right = kept(w32, limit), kept(worth(k64, top)[0], limit)
    # each of the `top` keys is off by 5 units and its rounding, the sum by its own
    error = UNIT * (6 * top + 3 * size.astype(np.float64))
    low = np.where(mine, w32 - error, np.inf).min(1)
    high = np.where(mine, -np.inf, w32 + error).max(1)
    sure = low > high
    assert np.array_equal(mine[sure], right[sure])
    if abs(bias) <= 1e3:  # and little is done twice at ordinary sizes
        assert sure.mean() > 0.9
