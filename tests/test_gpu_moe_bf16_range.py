"""bf16 activations up to the type's largest number in the experts' products."""

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
@pytest.mark.parametrize("big", [1e33, 5e36, 1e38, 3.3e38])
def test_bf16_activations_up_to_the_largest(dev, big, per):
    """Finite where the definition is: activations up to bf16's largest number, the
    scales so small that the sums are of ordinary size."""
    E, N, K = 2, 48, 160
    rng = np.random.default_rng(per)
    T = 2 * per
    off = np.array([0, per, T], np.int32)
    qw = codes_of(rng, E, 2 * N, K)
    sc = ((0.003 + 0.002 * rng.random((E, 2 * N, K // 32))) * (2.0 ** 17 / big)).astype(np.float32)
    x = rng.uniform(-1, 1, (T, K)) * big
    x[0, :32] = big  # one sign throughout: the offset's largest sums
    X = torch.from_numpy(x.astype(np.float32)).bfloat16()
    assert torch.isfinite(X).all()
    xv, tok = X.float().numpy(), np.arange(T, dtype=np.int32)
    H = pkg.w4a16_gemm_grouped_swiglu(X.to(dev), *on(dev, tok, off, qw, sc))
    tile = big_kernel(T, E, "bf16")
    want, tol = oracle.experts_swiglu(xv, tok, off, qw, sc, "bf16", tile)
    close(H, want, tol, f"swiglu {big} {per}")

    w = rng.standard_normal((per, 2)).astype(np.float32)
    slots = np.stack([np.arange(per), per + np.arange(per)], 1).astype(np.int32)
    Y = pkg.w4a16_gemm_grouped_combine(X.to(dev), *on(dev, off, qw, sc, slots, w))
    want, tol = oracle.experts_combine(xv, off, qw, sc, slots, w, "bf16", tile)
    close(Y, want, tol, f"combine {big} {per}")
