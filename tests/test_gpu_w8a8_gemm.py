"""w8a8_gemm and w8a8_gemm_grouped against the oracle."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from w8a8_cases import TYPES, close, codes_of, device, on, ref, same, scales_of  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    return device()


def window(R, E, dtype):
    """whether the call's kernel adds up in the fp8 instructions' window"""
    return pkg.w8a8_kernel(R, E) != pkg.W8A8_KERNEL_SKINNY and dtype != "fp32"


def operands(rng, M, N, K, E=None):
    lead = () if E is None else (E,)
    return (codes_of(rng, M, K), scales_of(rng, M, ref.blocks(K)), codes_of(rng, *lead, N, K),
            scales_of(rng, *lead, ref.blocks(N), ref.blocks(K)))


# rows of every kernel and of its edges, outputs and features that are no whole tiles
SHAPES = [(1, 1, 16), (1, 130, 272), (2, 4096, 128), (3, 7, 2064), (16, 300, 384), (17, 129, 144),
          (33, 257, 1040), (61, 512, 896), (64, 64, 4112), (65, 200, 256), (100, 1000, 640),
          (128, 128, 128), (129, 385, 400), (200, 640, 1168), (256, 256, 512), (300, 515, 2080),
          (513, 777, 272), (1000, 300, 1024),
          # every tile that the library chooses from, more than 64 blocks of features among them
          (16, 300, 8464), (200, 640, 8336), (40, 7168, 400), (250, 4096, 1296), (256, 700, 16400),
          (500, 2100, 400), (500, 4100, 272), (1030, 4100, 656), (2050, 4100, 272),
          (600, 1500, 8336)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(dev, M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    x, xs, w, ws = operands(rng, M, N, K)
    want, mag = ref.gemm(x, xs, w, ws)
    if dtype == "fp16":  # into its range
        k = np.float32(2.0 ** -np.ceil(np.log2(np.abs(want).max() / 2 ** 14)))
        xs, want, mag = xs * k, want * k, mag * k
    got = pkg.w8a8_gemm(*on(dev, x, xs, w, ws), dtype=TYPES[dtype])
    close(got, want, ref.bound(mag, want, K, dtype, window(M, 0, dtype)), f"{M} {N} {K}")


def routed(rng, T, E, R, empty=()):
    """token_index [R] and expert_offsets [E + 1] of R slots, none for the experts in `empty`"""
    share = rng.random(E) + 0.1
    share[list(empty)] = 0
    counts = rng.multinomial(R, share / share.sum())
    return (rng.integers(0, T, R).astype(np.int32),
            np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,R,N,K", [
    (1, 1, 1, 16, 16), (1, 8, 3, 130, 272), (16, 32, 64, 257, 384), (7, 5, 100, 96, 1040),
    (60, 60, 240, 200, 208), (90, 2, 180, 129, 256), (100, 3, 700, 300, 528),
    (300, 2, 1100, 520, 144), (64, 130, 300, 64, 128), (90, 60, 700, 200, 8336),
    (500, 3, 700, 300, 1168), (800, 2, 2000, 1000, 272), (900, 4, 3000, 2000, 400),
    (2000, 8, 9000, 2100, 144)])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(dev, T, E, R, N, K, gather, dtype):
    rng = np.random.default_rng(T + E + R)
    rows = T if gather else R
    x, xs, w, ws = operands(rng, rows, N, K, E)
    index, offsets = routed(rng, T, E, R, empty=[0] if E > 2 else [])
    index = index if gather else None
    want, mag = ref.grouped(x, xs, index, offsets, w, ws, R)
    if dtype == "fp16":
        k = np.float32(2.0 ** -np.ceil(np.log2(np.abs(want).max() / 2 ** 14)))
        xs, want, mag = xs * k, want * k, mag * k
    X, XS, W, WS, off = on(dev, x, xs, w, ws, offsets)
    got = pkg.w8a8_gemm_grouped(X, XS, on(dev, index)[0] if gather else None, off, W, WS,
                                dtype=TYPES[dtype])
    close(got, want, ref.bound(mag, want, K, dtype, window(R, E, dtype)), f"{T} {E} {R}")


# rows per expert: the kernels on both sides of their choice
PER = [1, 3, 20, 50, 120, 400]


@pytest.mark.parametrize("per", PER)
def test_rows_behind_the_last_slot_stay(dev, per):
    rng = np.random.default_rng(per)
    E, N, K, R = 3, 140, 272, 3 * per + 5
    x, xs, w, ws = operands(rng, R, N, K, E)
    off = np.array([0, per, per, 2 * per], np.int32)
    Y = torch.full((R, N), 7.0, device=dev)
    X, XS, W, WS, O = on(dev, x, xs, w, ws, off)
    pkg.w8a8_gemm_grouped(X, XS, None, O, W, WS, Y)
    want, mag = ref.grouped(x, xs, None, off, w, ws, R)
    used = slice(0, 2 * per)
    close(Y[used], want[used], ref.bound(mag, want, K, "fp32", False)[used], "used")
    assert torch.all(Y[2 * per:] == 7.0)


@pytest.mark.parametrize("per", PER)
def test_malformed_lists_stay_in_bounds(dev, per):
    """Indices and offsets out of range are clamped; the slots that are in order are right."""
    rng = np.random.default_rng(per)
    E, N, K, R, T = 4, 140, 272, 4 * per, 2 * per
    x, xs, w, ws = operands(rng, T, N, K, E)
    index = rng.integers(0, T, R).astype(np.int32)
    index[per:] = rng.choice([-5, T, 2 ** 31 - 1, -2 ** 31], R - per)
    off = np.array([0, per, 2 ** 31 - 1, 5, -7], np.int32)
    X, XS, W, WS, I, O = on(dev, x, xs, w, ws, index, off)
    got = pkg.w8a8_gemm_grouped(X, XS, I, O, W, WS, dtype=torch.float32)
    torch.cuda.synchronize()
    want, mag = ref.gemm(x[index[:per]], xs[index[:per]], w[0], ws[0])
    close(got[:per], want, ref.bound(mag, want, K, "fp32", False), "in order")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_nan_stays_where_it_enters(dev, M, dtype):
    rng = np.random.default_rng(M)
    N, K = 300, 528
    x, xs, w, ws = operands(rng, M, N, K)
    x[0, 5] = 0x7F
    w[131, 520], w[7, 3] = 0xFF, 0x7F
    if M > 1:
        xs[M - 1, 4] = np.nan
    got = pkg.w8a8_gemm(*on(dev, x, xs, w, ws), dtype=TYPES[dtype]).float().cpu().numpy()
    nan = np.isnan(got)
    assert nan[0].all() and nan[M - 1].all() and nan[:, 131].all() and nan[:, 7].all()
    nan[0] = nan[M - 1] = True
    nan[:, [7, 131]] = False
    assert not nan[1:M - 1].any()


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_zero_scales_and_weights(dev, M):
    rng = np.random.default_rng(M)
    N, K = 200, 400
    x, xs, w, ws = operands(rng, M, N, K)
    xs[:] = 0
    got = pkg.w8a8_gemm(*on(dev, x, xs, w, ws))
    assert not got.any()


@pytest.mark.parametrize("M,N,K", [(1, 300, 640), (40, 129, 272), (70, 200, 256), (400, 520, 1168)])
def test_offset_buffers(dev, M, N, K):
    """Y at an address that its vector stores cannot take, codes at any 16 bytes."""
    rng = np.random.default_rng(M)
    x, xs, w, ws = on(dev, *operands(rng, M, N, K))
    want = pkg.w8a8_gemm(x, xs, w, ws)
    room = torch.zeros(M * N + 3, dtype=torch.bfloat16, device=dev)
    for at in (1, 2, 3):
        Y = room[at:at + M * N].view(M, N)
        pkg.w8a8_gemm(x, xs, w, ws, Y)
        assert same(Y, want)
    far = torch.zeros(x.numel() + 48, dtype=torch.uint8, device=dev)
    far[48:] = x.flatten()
    assert same(pkg.w8a8_gemm(far[48:].view(M, K), xs, w, ws), want)


def test_repeated_calls_are_the_same(dev):
    rng = np.random.default_rng(5)
    for M, N, K in [(1, 512, 2064), (64, 300, 1024), (300, 512, 640)]:
        a = on(dev, *operands(rng, M, N, K))
        first = pkg.w8a8_gemm(*a)
        for _ in range(3):
            assert same(pkg.w8a8_gemm(*a), first)


def test_nothing_to_do_and_refusals(dev):
    x, xs, w, ws = on(dev, *operands(np.random.default_rng(0), 4, 130, 256))
    assert pkg.w8a8_gemm(x[:0], xs[:0], w, ws).shape == (0, 130)
    assert pkg.w8a8_gemm(x, xs, w[:0], ws[:0]).shape == (4, 0)
    off = torch.zeros(2, dtype=torch.int32, device=dev)
    index = torch.zeros(0, dtype=torch.int32, device=dev)
    assert pkg.w8a8_gemm_grouped(x, xs, index, off, w[None], ws[None]).shape == (0, 130)
    for call, error in [
            (lambda: pkg.w8a8_gemm(x, xs[:, :1], w, ws), ValueError),
            (lambda: pkg.w8a8_gemm(x, xs, w[:, :128], ws), ValueError),
            (lambda: pkg.w8a8_gemm(x, xs, w[:, :128].contiguous(), ws), ValueError),
            (lambda: pkg.w8a8_gemm(x, xs, w, ws[:1]), ValueError),
            (lambda: pkg.w8a8_gemm(x, xs, w, ws, dtype=torch.float64), TypeError),
            (lambda: pkg.w8a8_gemm(x.float(), xs, w, ws), TypeError),
            (lambda: pkg.w8a8_gemm(x, xs, w, ws, torch.zeros(4, 4, device=dev)), ValueError),
            (lambda: pkg.w8a8_gemm_grouped(x, xs, None, off, w, ws), ValueError),
            (lambda: pkg.w8a8_gemm_grouped(x, xs, None, off[:1], w[None], ws[None]), ValueError),
            (lambda: pkg.w8a8_gemm_grouped(x, xs, off.long(), off, w[None], ws[None]), TypeError)]:
        with pytest.raises(error):
            call()


def test_codes_of_torch(dev):
    """torch.float8_e4m3fn and uint8 are the same codes."""
    x, xs, w, ws = on(dev, *operands(np.random.default_rng(2), 9, 200, 400))
    f8 = torch.float8_e4m3fn
    assert same(pkg.w8a8_gemm(x.view(f8), xs, w.view(f8), ws), pkg.w8a8_gemm(x, xs, w, ws))


def test_other_streams_and_two_at_once(dev):
    rng = np.random.default_rng(8)
    calls = [on(dev, *operands(rng, M, 512, 1024)) for M in (1, 70, 600, 40)]
    want = [pkg.w8a8_gemm(*a) for a in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(5):
        got.append([pkg.w8a8_gemm(*a, stream=s) for a, s in zip(calls, streams)])
    torch.cuda.synchronize()
    for each in got:
        assert all(same(a, b) for a, b in zip(each, want))
