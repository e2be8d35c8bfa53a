"""What w8a8_gemm_grouped writes and what it leaves: rows behind the last slot, lists that are
malformed and lists that overlap, for every type of output, rows that are whole vectors and odd
ones, and tiles of every size."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from w8a8_cases import TYPES, codes_of, device, on, ref, scales_of  # noqa: E402

K = 144
GUARD = 64  # elements around Y


@pytest.fixture(scope="module")
def dev():
    return device()


class Case:
    """Operands of E experts, the products of every expert with any rows in fp64 (on the device),
    and a Y of 7s with 7s around it."""

    def __init__(self, dev, E, R, N, dtype, seed):
        rng = np.random.default_rng(seed)
        x, xs = codes_of(rng, R, K), scales_of(rng, R, 2) * np.float32(2.0 ** -9)
        w, ws = codes_of(rng, E, N, K), scales_of(rng, E, ref.blocks(N), 2) * np.float32(2.0 ** -2)
        self.X, self.xs, self.W, self.ws = on(dev, x, xs, w, ws)
        table = torch.from_numpy(np.nan_to_num(ref.E4M3)).to(dev)
        self.x = table[self.X.long()] * self.xs.double().repeat_interleave(128, -1)[:, :K]
        self.w = table[self.W.long()] * self.ws.double().repeat_interleave(128, -1)[..., :K] \
            .repeat_interleave(128, -2)[:, :N]
        self.window = pkg.w8a8_kernel(R, E) != pkg.W8A8_KERNEL_SKINNY and dtype != "fp32"
        self.dtype = dtype
        self.room = torch.full((R * N + 2 * GUARD,), 7.0, dtype=TYPES[dtype], device=dev)
        self.Y = self.room[GUARD:GUARD + R * N].view(R, N)

    def run(self, off, index=None):
        dev = self.X.device
        off = torch.tensor(np.asarray(off, np.int64).astype(np.int32), device=dev)
        if index is not None:
            index = torch.from_numpy(np.asarray(index, np.int32)).to(dev)
        pkg.w8a8_gemm_grouped(self.X, self.xs, index, off, self.W, self.ws, self.Y)
        assert bool((self.room[:GUARD] == 7).all()) and bool((self.room[-GUARD:] == 7).all())

    def near(self, rows, e, got):
        """elementwise: `got` is rows `rows` of X times expert e's weights"""
        want, mag = self.x[rows] @ self.w[e].t(), self.x[rows].abs() @ self.w[e].abs().t()
        tol = (2 * 128 + 2 + 4) * ref.U * mag + (ref.WINDOW * mag if self.window else 0.0)
        tol = tol + ref.HALF_STEP[self.dtype] * (want.abs() + tol) + ref.SMALLEST[self.dtype]
        return (got.double() - want).abs() <= tol


# E, slots per expert, N: the skinny kernel, then tiles from 16 x 32 to 256 x 256
SIZES = [(3, 3, 1040), (3, 3, 1039), (3, 15, 1040), (3, 15, 1037), (3, 40, 1032), (3, 120, 2056),
         (3, 120, 2053), (3, 400, 2056), (16, 60, 2056), (4, 250, 4104), (4, 700, 4104), (4, 700, 4099),
         (8, 1100, 4104), (8, 1100, 4101)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,per,N", SIZES)
def test_rows_behind_the_last_slot(dev, E, per, N, dtype):
    R = E * per + 5
    c = Case(dev, E, R, N, dtype, per + N)
    off = np.arange(E + 1) * per
    off[1], off[2] = per, per  # the second has none
    off[2:] -= np.arange(len(off[2:])) % 2  # and not all the same
    c.run(off)
    assert bool((c.Y[off[-1]:] == 7).all())
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        assert bool(c.near(s, e, c.Y[s]).all()), e


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,per,N", SIZES)
def test_malformed_lists(dev, E, per, N, dtype):
    """Offsets and indices out of range are clamped: the first expert's slots are in order, the
    next takes all that are left, with tokens clamped into range, the others none."""
    R = E * per + 5
    c = Case(dev, E, R, N, dtype, per + N)
    rng = np.random.default_rng(per)
    index = rng.integers(0, R, R)
    index[per:] = rng.choice([-5, R, 2 ** 31 - 1, -2 ** 31], R - per)
    off = np.array([0, per, 2 ** 31 - 1] + [5, -7] * E)[:E + 1]
    off[3:] = -7
    c.run(off, index)
    clamped = torch.from_numpy(np.clip(index, 0, R - 1)).to(dev)
    assert bool(c.near(clamped[:per], 0, c.Y[:per]).all())
    assert bool(c.near(clamped[per:], 1, c.Y[per:]).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,per,N", SIZES)
def test_overlapping_lists(dev, E, per, N, dtype):
    """Experts that claim the same slots: every element is the result of one that claims it, or as
    it was (there are more items than workgroups for them)."""
    R = E * per + 5
    c = Case(dev, E, R, N, dtype, per + N)
    off = np.array([0, R] * E)[:E + 1]
    c.run(off)
    right = c.Y == 7
    assert not bool(right.all())
    for e in range(0, E, 2):
        if off[e + 1] > off[e]:
            right |= c.near(slice(0, R), e, c.Y)
    assert bool(right.all())
