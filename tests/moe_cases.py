"""Inputs and comparisons shared by the GPU tests of the experts' products."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import int4_weight_only_03_amd as pkg  # noqa: E402

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}

# slots of each of two experts: one token, the skinny kernel's items, the tile kernel
PER = [1, 2, 6, 20, 90]


def device():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    pkg.load()
    return torch.device("cuda:0")


def codes_of(rng, E, rows, K):
    """qweight int32 [E][rows][K/8] of random nibbles"""
    return rng.integers(-(2 ** 31), 2 ** 31, (E, rows, K // 8), dtype=np.int64).astype(np.int32)


def on(dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got)), f"{what}: {np.sum(~np.isfinite(got))} not finite"
    err = np.abs(got - want)
    print(f"  {what}: max err/bound {np.max(err / tol):.3e}", flush=True)
    assert np.all(err <= tol)


def big_kernel(R, E, dtype):
    return pkg.w4a16_experts_kernel(R, E, TYPES[dtype]) == pkg.W4A16_EXPERTS_TILE
