"""Routing with biases of opposite signs inside a group, whose two largest keys cancel:
the groups and experts are those of 64-bit keys."""

import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    pkg.load()
    return torch.device("cuda:0")


def choices(x, bias, topk, score, groups, limit):
    """ids [T][topk] by 64-bit keys, groups valued by their two largest"""
    x = x.astype(np.float64)
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-x))
    else:
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    key = s + bias.astype(np.float64)
    T, E = key.shape
    part = np.sort(key.reshape(T, groups, -1), -1)
    worth = part[..., -1] + part[..., -2]
    best = np.argsort(-worth, axis=1, kind="stable")[:, :limit]
    open_ = np.zeros((T, groups), bool)
    np.put_along_axis(open_, best, True, 1)
    key = np.where(np.repeat(open_, E // groups, 1), key, -np.inf)
    return np.argsort(-key, axis=1, kind="stable")[:, :topk].astype(np.int32)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,limit,topk", [
    (40000, 32, 8, 4, 8),     # 16 lanes a token
    (20000, 128, 32, 9, 12),  # a wave a token
    (64, 160, 8, 3, 6), (16, 64, 8, 4, 8),
])
def test_groups_whose_keys_cancel(dev, T, E, groups, limit, topk, score):
    wrong = {}
    for size in (1.0, 1e4, 1e5, 1e6, -1e4):
        rng = np.random.default_rng(T + int(abs(size)))
        x = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
        bias = np.where(np.arange(E) % (E // groups) == 0, size, -size)
        bias = (bias + 0.1 * rng.standard_normal(E)).astype(np.float32)
        r = pkg.w4a16_moe_route(torch.from_numpy(x).to(dev), topk,
                                bias=torch.from_numpy(bias).to(dev), score=score, groups=groups,
                                group_limit=limit, group_top=2)
        want = choices(x, bias, topk, score, groups, limit)
        wrong[size] = int((r.ids.cpu().numpy() != want).any(1).sum())
        print("  tokens of", T, score, size, "otherwise:", wrong[size], flush=True)
    sys.stdout.flush()
    assert not any(wrong.values()), wrong


@pytest.mark.parametrize("T", [1, 40, 5000])
def test_groups_masked_by_the_lowest_number(dev, T):
    """Biases of fp32's lowest and largest numbers: sums of two overflow in fp32."""
    E, groups, limit, topk = 32, 8, 3, 6
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, E)).astype(np.float32)
    most = np.finfo(np.float32).max
    for big in ([0, 1, 2, 3], [4, 5, 6, 9, 10, 11], list(range(8, 30))):
        for sign in (-1, 1):
            bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
            bias[big] = sign * most * rng.choice([1.0, 0.75, 0.5], len(big)).astype(np.float32)
            r = pkg.w4a16_moe_route(torch.from_numpy(x).to(dev), topk,
                                    bias=torch.from_numpy(bias).to(dev), score="sigmoid",
                                    groups=groups, group_limit=limit, group_top=2)
            want = choices(x, bias, topk, "sigmoid", groups, limit)
            assert np.array_equal(r.ids.cpu().numpy(), want), (big, sign)
