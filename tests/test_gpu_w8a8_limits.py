"""The 8-bit products at the ends of their ranges: buffers past 2^31 and 2^32, many
experts, the longest rows, lists that hold nothing."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from w8a8_cases import TYPES, close, codes_of, device, on, ref, same, scales_of  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    return device()


def random_codes(dev, *shape):
    """codes of every value but NaN, made on the device"""
    c = torch.randint(0, 254, shape, dtype=torch.uint8, device=dev)
    return c + (c >= 127).to(torch.uint8)


@pytest.mark.parametrize("R", [5, 700])
def test_weights_past_2_32_bytes(dev, R):
    """Experts whose weights begin past 2^32 bytes."""
    E, N, K = 40, 4096, 32768
    W = torch.zeros(E, N, K, dtype=torch.uint8, device=dev)
    W[-1] = random_codes(dev, N, K)
    ws = torch.rand(E, 32, 256, device=dev)
    X, xs = random_codes(dev, R, K), torch.rand(R, 256, device=dev)
    off = torch.full((E + 1,), R, dtype=torch.int32, device=dev)
    off[:E] = 0
    got = pkg.w8a8_gemm_grouped(X, xs, None, off, W, ws, dtype=torch.float32)
    one = torch.tensor([0, R], dtype=torch.int32, device=dev)
    # the same slots of one expert that owns all (the kernels may differ: to their tolerance)
    want = pkg.w8a8_gemm_grouped(X, xs, None, one, W[-1:], ws[-1:], dtype=torch.float32)
    assert torch.isfinite(got).all() and want.any()
    x, w = xs.abs().amax().item() * 448, ws.abs().amax().item() * 448
    assert (got - want).abs().max().item() <= 2 * (2 * 128 + 256 + 4) * ref.U * K * x * w


@pytest.mark.parametrize("M", [3, 40, 300])
def test_activations_past_2_32_bytes(dev, M):
    """Tokens whose rows begin past 2^32 bytes, read through the index."""
    T, N, K = 33000, 200, 131072
    X = torch.zeros(T, K, dtype=torch.uint8, device=dev)
    X[-M:] = random_codes(dev, M, K)
    xs = torch.rand(T, 1024, device=dev)
    W, ws = random_codes(dev, 1, N, K), torch.rand(1, 2, 1024, device=dev)
    index = torch.arange(T - M, T, dtype=torch.int32, device=dev)
    off = torch.tensor([0, M], dtype=torch.int32, device=dev)
    got = pkg.w8a8_gemm_grouped(X, xs, index, off, W, ws, dtype=torch.float32)
    want = pkg.w8a8_gemm_grouped(X[-M:].contiguous(), xs[-M:].contiguous(), None, off, W, ws,
                                 dtype=torch.float32)
    assert same(got, want) and want.any()


def test_outputs_past_2_32_bytes(dev):
    """Y of more than 2^31 elements: its last rows are those of a call of their own."""
    M, N, K = 66000, 33000, 144
    X, xs = random_codes(dev, M, K), torch.rand(M, 2, device=dev)
    W, ws = random_codes(dev, N, K), torch.rand(258, 2, device=dev)
    Y = pkg.w8a8_gemm(X, xs, W, ws)
    last = slice(M - 256, M)
    own = pkg.w8a8_gemm(X[last].contiguous(), xs[last].contiguous(), W, ws, dtype=torch.float32)
    # both are within a rounding of 2^-8 and the fp8 instructions' window of the same sum
    values = torch.arange(256, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn).float()
    mag = (values[X[last].long()].abs() * xs[last].repeat_interleave(128, 1)[:, :K]) @ \
        (values[W.long()].abs() * ws.repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]).t()
    tol = 2.0 ** -8 * own.abs() + (ref.WINDOW + 2 * 262 * ref.U) * mag * 1.01
    assert bool(((Y[last].float() - own).abs() <= tol).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N,K", [(1030, 4096, 7168), (4100, 4100, 3600), (3000, 7168, 2048)])
def test_rows_behind_whole_rounds(dev, M, N, K, dtype):
    """Sizes whose last rows a launch of their own may take."""
    table = torch.from_numpy(np.nan_to_num(ref.E4M3)).to(dev)
    X, W = random_codes(dev, M, K), random_codes(dev, N, K)
    xs = torch.rand(M, ref.blocks(K), device=dev) * 2.0 ** -10
    ws = torch.rand(ref.blocks(N), ref.blocks(K), device=dev) * 2.0 ** -10

    def wide(scales):
        return scales.double().repeat_interleave(128, -1)[..., :K]

    x = table[X.long()] * wide(xs)
    w = table[W.long()] * wide(ws).repeat_interleave(128, 0)[:N]
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    got = pkg.w8a8_gemm(X, xs, W, ws, dtype=TYPES[dtype])
    tol = (2 * 128 + ref.blocks(K) + 4) * ref.U * mag
    if dtype != "fp32":
        tol += ref.WINDOW * mag
    tol += ref.HALF_STEP[dtype] * (want.abs() + tol) + ref.SMALLEST[dtype]
    err = (got.double() - want).abs()
    print(f"  max err/bound {(err / tol).max().item():.3e}", flush=True)
    assert bool((err <= tol).all())


@pytest.mark.parametrize("dtype", list(TYPES))
def test_part_filled_tiles(dev, dtype):
    """Experts whose last tiles hold few slots, a quarter, half, three quarters of them and one
    more, and all but one."""
    N, K = 4104, 272
    last = (1, 16, 63, 64, 65, 128, 129, 192, 193, 255)
    off = np.concatenate([[0], np.cumsum([1024 + n for n in last])]).astype(np.int32)
    E, R = len(last), int(off[-1])
    table = torch.from_numpy(np.nan_to_num(ref.E4M3)).to(dev)
    X, W = random_codes(dev, R, K), random_codes(dev, E, N, K)
    xs = torch.rand(R, ref.blocks(K), device=dev) * 2.0 ** -10
    ws = torch.rand(E, ref.blocks(N), ref.blocks(K), device=dev) * 2.0 ** -10
    got = pkg.w8a8_gemm_grouped(X, xs, None, torch.from_numpy(off).to(dev), W, ws,
                                dtype=TYPES[dtype])
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        x = table[X[rows].long()] * xs[rows].double().repeat_interleave(128, -1)[:, :K]
        w = table[W[e].long()] * ws[e].double().repeat_interleave(128, -1)[:, :K] \
            .repeat_interleave(128, 0)[:N]
        want, mag = x @ w.t(), x.abs() @ w.abs().t()
        tol = (2 * 128 + ref.blocks(K) + 4) * ref.U * mag
        if dtype != "fp32":
            tol += ref.WINDOW * mag
        tol += ref.HALF_STEP[dtype] * (want.abs() + tol) + ref.SMALLEST[dtype]
        err = (got[rows].double() - want).abs()
        print(f"  {last[e]} behind the last whole tile: max err/bound "
              f"{(err / tol).max().item():.3e}", flush=True)
        assert bool((err <= tol).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N", [(20, 4097), (64, 7169), (130, 4099), (300, 4103), (900, 4101),
                                 (2049, 4095), (4097, 4111)])
def test_odd_rows_of_outputs(dev, M, N, dtype):
    """Outputs whose rows begin anywhere, at any start: bit for bit those of whole vectors (the
    same product with rows of W more), and nothing around them is touched."""
    K = 400
    X, W = random_codes(dev, M, K), random_codes(dev, N, K)
    xs = torch.rand(M, ref.blocks(K), device=dev) * 2.0 ** -10
    ws = torch.rand(ref.blocks(N), ref.blocks(K), device=dev) * 2.0 ** -10
    more = -N % 8  # in N's last block, or the 8 rows would need scales of their own
    want = pkg.w8a8_gemm(X, xs, torch.cat([W, W[:more]]), ws if ref.blocks(N + more) == len(ws)
                         else torch.cat([ws, ws[:1]]), dtype=TYPES[dtype])[:, :N]
    for at in (0, 1, 5):
        room = torch.full((M * N + 32,), 7.0, dtype=TYPES[dtype], device=dev)
        Y = room[at + 8:at + 8 + M * N].view(M, N)
        pkg.w8a8_gemm(X, xs, W, ws, Y)
        assert same(Y, want.contiguous())
        assert bool((room[:at + 8] == 7).all()) and bool((room[at + 8 + M * N:] == 7).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_whole_rounds_and_rest_in_a_graph(dev, dtype):
    """Such a product captured, on inputs that change: bit for bit the eager one's, and nothing
    of the rows around its output is touched."""
    M, N, K = 1030, 4096, 7168
    W = random_codes(dev, N, K)
    X, xs = random_codes(dev, M, K), torch.rand(M, ref.blocks(K), device=dev) * 2.0 ** -10
    ws = torch.rand(ref.blocks(N), ref.blocks(K), device=dev) * 2.0 ** -10
    around = torch.full((M + 16, N), 7.0, dtype=TYPES[dtype], device=dev)
    Y = around[8:M + 8]
    pkg.w8a8_gemm(X, xs, W, ws, Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.w8a8_gemm(X, xs, W, ws, Y)
    for _ in range(3):
        X.copy_(random_codes(dev, M, K))
        xs.copy_(torch.rand_like(xs) * 2.0 ** -10)
        Y.fill_(7.0)
        graph.replay()
        got = Y.clone()
        assert same(got, pkg.w8a8_gemm(X, xs, W, ws, dtype=TYPES[dtype]))
    assert bool((around[:8] == 7).all()) and bool((around[M + 8:] == 7).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [1, 30, 130])
def test_longest_rows(dev, M, dtype):
    rng = np.random.default_rng(M)
    N, K = 70, 131072
    x, xs, w, ws = codes_of(rng, M, K), scales_of(rng, M, 1024), codes_of(rng, N, K), \
        scales_of(rng, 1, 1024)
    want, mag = ref.gemm(x, xs, w, ws)
    if dtype == "fp16":
        k = np.float32(2.0 ** -np.ceil(np.log2(np.abs(want).max() / 2 ** 14)))
        xs, want, mag = xs * k, want * k, mag * k
    got = pkg.w8a8_gemm(*on(dev, x, xs, w, ws), dtype=TYPES[dtype])
    window = pkg.w8a8_kernel(M) == pkg.W8A8_KERNEL_TILE and dtype != "fp32"
    close(got, want, ref.bound(mag, want, K, dtype, window), f"{M} rows")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 700, 8192), (2, 33, 12288)])
def test_rows_of_whole_pages(dev, M, N, K, dtype):
    """Few rows at lengths where workgroups begin at blocks of their own, dense and by expert; a
    NaN in any block reaches its outputs and no others."""
    rng = np.random.default_rng(N)
    E, R = 3, 3 * M
    x, xs = codes_of(rng, R, K), scales_of(rng, R, K // 128) * np.float32(2.0 ** -12)
    w, ws = codes_of(rng, E, N, K), scales_of(rng, E, -(-N // 128), K // 128) * np.float32(2.0 ** -12)
    off = np.array([0, 0, 2 * M, R], np.int32)
    X, XS, W, WS, O = on(dev, x, xs, w, ws, off)
    assert pkg.w8a8_kernel(R, E) == pkg.W8A8_KERNEL_SKINNY
    want, mag = ref.grouped(x, xs, None, off, w, ws, R)
    got = pkg.w8a8_gemm_grouped(X, XS, None, O, W, WS, dtype=TYPES[dtype])
    close(got, want, ref.bound(mag, want, K, dtype, False), f"by expert {M} {N} {K}")
    want, mag = ref.gemm(x[:M], xs[:M], w[0], ws[0])
    got = pkg.w8a8_gemm(X[:M], XS[:M], W[0], WS[0], dtype=TYPES[dtype])
    close(got, want, ref.bound(mag, want, K, dtype, False), f"{M} {N} {K}")
    for block in (0, 15, K // 128 - 1):
        bad = W[0].clone()
        bad[N - 1, 128 * block + 77] = 0x7F
        nan = pkg.w8a8_gemm(X[:M], XS[:M], bad, WS[0], dtype=TYPES[dtype]).isnan()
        assert bool(nan[:, N - 1].all()) and int(nan.sum()) == M


@pytest.mark.parametrize("E,R", [(65535, 100), (3000, 31000), (1025, 2000)])
def test_many_experts(dev, E, R):
    rng = np.random.default_rng(E)
    N, K = 24, 48
    x, xs = codes_of(rng, R, K), scales_of(rng, R, 1)
    w, ws = codes_of(rng, E, N, K), scales_of(rng, E, 1, 1)
    off = np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32)
    off[0], off[-1] = 0, R
    want, mag = ref.grouped(x, xs, None, off, w, ws, R)
    X, XS, O, W, WS = on(dev, x, xs, off, w, ws)
    got = pkg.w8a8_gemm_grouped(X, XS, None, O, W, WS, dtype=torch.float32)
    close(got, want, ref.bound(mag, want, K, "fp32", False), f"{E} experts")


@pytest.mark.parametrize("R", [6, 200, 3000])
def test_lists_that_hold_nothing(dev, R):
    """Every expert empty: nothing is written."""
    rng = np.random.default_rng(R)
    x, xs, w, ws = on(dev, codes_of(rng, R, 64), scales_of(rng, R, 1), codes_of(rng, 3, 40, 64),
                      scales_of(rng, 3, 1, 1))
    Y = torch.full((R, 40), 7.0, device=dev)
    for off in ([0, 0, 0, 0], [R, R, R, R], [-5, -5, -5, -5], [9, 8, 7, 6]):
        pkg.w8a8_gemm_grouped(x, xs, None, torch.tensor(off, dtype=torch.int32, device=dev), w, ws, Y)
    assert torch.all(Y == 7.0)


@pytest.mark.parametrize("per", [2, 40, 300])
def test_lists_that_overlap(dev, per):
    """Experts that claim each other's slots: some expert's result, and no access out of
    bounds."""
    rng = np.random.default_rng(per)
    E, R, N, K = 8, 4 * per, 40, 64
    x, xs, w, ws = on(dev, codes_of(rng, R, K), scales_of(rng, R, 1), codes_of(rng, E, N, K),
                      scales_of(rng, E, 1, 1))
    off = torch.tensor([0, R] * (E // 2) + [0], dtype=torch.int32, device=dev)
    got = pkg.w8a8_gemm_grouped(x, xs, None, off, w, ws, dtype=torch.float32)
    torch.cuda.synchronize()
    assert got.shape == (R, N)
