"""Accuracy of the experts' products of bf16 prompts, whose kernel takes scales and
scaled weights in fp16: the bound, element by element, and the root mean square."""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402
from moe_cases import big_kernel, close, codes_of, device, on  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    return device()


@pytest.mark.parametrize("K", [2048, 7168])
def test_bf16_prompt_products_within_the_bound(dev, K):
    """The tile kernel on long rows, element by element."""
    E, N, per = 2, 96, 65
    rng = np.random.default_rng(K)
    T = E * per
    off = np.array([0, per, T], np.int32)
    tok = rng.permutation(T).astype(np.int32)
    assert big_kernel(T, E, "bf16")
    qw = codes_of(rng, E, 2 * N, K)
    sc = (0.002 * 2.0 ** rng.random((E, 2 * N, K // 32))).astype(np.float32)
    X = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    H = pkg.w4a16_gemm_grouped_swiglu(X.to(dev), *on(dev, tok, off, qw, sc))
    want, tol = oracle.experts_swiglu(X.float().numpy(), tok, off, qw, sc, "bf16", True)
    close(H, want, tol, f"swiglu {K}")
    w = np.ones((T, 1), np.float32)
    slots = np.arange(T, dtype=np.int32)[:, None]
    Y = pkg.w4a16_gemm_grouped_combine(X.to(dev), *on(dev, off, qw, sc, slots, w))
    want, tol = oracle.experts_combine(X.float().numpy(), off, qw, sc, slots, w, "bf16", True)
    close(Y, want, tol, f"combine {K}")


@pytest.mark.parametrize("K", [32, 2048, 7168])
def test_bf16_prompt_products_root_mean_square(dev, K):
    """The tile kernel rounds a scale and a scaled weight to fp16, each by a relative
    error of mean square 2^-20 / 12 * E[1/m^2] over mantissas m in [1, 2), 0.541 on a
    log scale: 2^-24.47, and independent.  The mean square of a sum's error is that
    times the sum of the squared group sums (the scales') plus the sum of the squared
    products (the weights', none where the code is a power of two); 2^-24 of both leaves
    a third for the sample.

    The stored result is rounded far more coarsely, so the sum is seen as a
    difference: expert 1 has expert 0's codes and scales that fp16 takes exactly with
    every code (8 bits), at most 2^-8 apart from expert 0's, and a token subtracts its
    product with one from that with the other.  What is left is the rounding of a
    difference 2^-9 of the sum, and fp32's."""
    N, T = 512, 64
    rng = np.random.default_rng(K)
    G = K // 32
    codes = codes_of(rng, 1, N, K)
    near = 0.002 * 2.0 ** rng.random((1, N, G))
    exact = torch.from_numpy(near).bfloat16().double().numpy()
    apart = exact * (1 + 2.0 ** -8 * rng.random((1, N, G)))
    qw = np.concatenate([codes, codes])
    sc = np.concatenate([apart, exact]).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    off = np.array([0, T, 2 * T], np.int32)
    assert big_kernel(2 * T, 2, "bf16")
    slots = np.stack([np.arange(T), T + np.arange(T)], 1).astype(np.int32)
    w = np.tile(np.float32([1.0, -1.0]), (T, 1))
    Y = pkg.w4a16_gemm_grouped_combine(torch.cat([x, x]).to(dev), *on(dev, off, qw, sc, slots, w))

    xv = x.double().numpy()
    W = (oracle.unpack(codes[0]).astype(np.float64) - 8.0).reshape(N, G, 32)
    s0, s1 = sc.astype(np.float64)
    sums = np.einsum("tgk,ngk->tng", xv.reshape(T, G, 32), W)
    want = (sums * (s0 - s1)).sum(-1)
    terms = ((sums * s0) ** 2).sum(-1)
    terms += np.einsum("tgk,ngk->tn", xv.reshape(T, G, 32) ** 2, (W * s0[..., None]) ** 2)
    err = Y.double().cpu().numpy() - want
    # the difference's own rounding, and two fp32 sums (2^-21 of their terms' root sum)
    other = (2.0 ** -8 * want) ** 2 / 3 + 2 * 2.0 ** -42 * terms
    share = np.sqrt(np.mean(err ** 2) / np.mean(terms))
    print(f"  {K}: root mean square {share * 2 ** 12:.3f} * 2^-12 of the terms", flush=True)
    assert np.mean(err ** 2) <= np.mean(2.0 ** -24 * terms + other)


def test_bf16_codes_are_exact_up_to_52_slots(dev):
    """Sums to fp32's accuracy in the tile kernel, too: seen as in the test above, by
    tokens that take the difference of two nearly equal products."""
    N, T, K = 256, 52, 1024
    rng = np.random.default_rng(52)
    codes = codes_of(rng, 1, N, K)
    s1 = (0.002 * 2.0 ** rng.random((1, N, K // 32))).astype(np.float32)
    s0 = (s1 * (1 + 2.0 ** -8 * rng.random((1, N, K // 32)))).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16()
    off = np.array([0, T, 2 * T], np.int32)
    assert big_kernel(2 * T, 2, "bf16")
    slots = np.stack([np.arange(T), T + np.arange(T)], 1).astype(np.int32)
    w = np.tile(np.float32([1.0, -1.0]), (T, 1))
    args = (off, np.concatenate([codes, codes]), np.concatenate([s0, s1]), slots, w)
    Y = pkg.w4a16_gemm_grouped_combine(torch.cat([x, x]).to(dev), *on(dev, *args))
    xv = torch.cat([x, x]).float().numpy()
    want, tol = oracle.experts_combine(xv, *args, "fp32")
    close(Y, want, tol + 2.0 ** -8 * (np.abs(want) + tol), "52 slots")


@pytest.mark.parametrize("per", [32, 60])
def test_bf16_prompt_weights_past_4_gib(dev, per):
    E, F, K, T = 300, 1024, 14336, 40
    gen = torch.Generator(dev).manual_seed(per)
    qw = torch.randint(-(2 ** 31), 2 ** 31, (E, 2 * F, K // 8), dtype=torch.int32, device=dev,
                       generator=gen)
    sc = 0.003 + 0.002 * torch.rand(E, 2 * F, K // 32, device=dev, generator=gen)
    X = torch.randn(T, K, device=dev, generator=gen).bfloat16()
    tok = torch.randint(0, T, (E * per,), dtype=torch.int32, device=dev, generator=gen)
    off = torch.arange(0, E * per + 1, per, dtype=torch.int32, device=dev)
    assert big_kernel(E * per, E, "bf16")
    H = pkg.w4a16_gemm_grouped_swiglu(X, tok, off, qw, sc)
    for e in (0, 146, E - 1):
        one = slice(e * per, (e + 1) * per)
        want, tol = oracle.experts_swiglu(X.float().cpu().numpy(), tok[one].cpu().numpy(),
                                          np.array([0, per], np.int32), qw[e:e + 1].cpu().numpy(),
                                          sc[e:e + 1].cpu().numpy(), "bf16", True)
        close(H[one], want, tol, f"expert {e}")

