"""Argument checks and workspace queries of the mixture-of-experts entry points
(no GPU is touched: the addresses are fakes that are never dereferenced)."""

import inspect

import numpy as np
import pytest

import int4_weight_only_03_amd as pkg
from int4_weight_only_03_amd import binding

OK, ARG, SHAPE, ALIGN = 0, 1, 2, 3
BASE = 1 << 40


def at(i):
    return BASE + (i << 33)


def route(lib, **change):
    a = dict(logits=at(0), bias=at(1), num=at(2), ids=at(3), weights=at(4), slots=at(5),
             token_index=at(6), offsets=at(7), T=100, E=64, topk=8, score=0, groups=8,
             group_limit=4, group_top=2, renormalize=1, scale=1.0, dtype=0, ws=at(8),
             ws_bytes=1 << 20, stream=None)
    a.update(change)
    return lib.w4a16_moe_route(*a.values())


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(topk=0), ARG), (dict(topk=65), ARG),
    (dict(E=1032), SHAPE), (dict(topk=33), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(T=1 << 62), SHAPE), (dict(T=(1 << 25) + 1, topk=1), SHAPE),
    (dict(score=2), ARG), (dict(dtype=3), ARG), (dict(dtype=-1), ARG), (dict(groups=0), ARG),
    (dict(groups=7), ARG), (dict(groups=128, E=256), SHAPE), (dict(group_limit=0), ARG),
    (dict(group_limit=9), ARG), (dict(group_top=0), ARG), (dict(group_top=3), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(logits=None), ARG), (dict(ids=None), ARG), (dict(weights=None), ARG),
    (dict(slots=None), ARG), (dict(token_index=None), ARG), (dict(offsets=None), ARG),
    (dict(logits=at(0) + 2), ALIGN), (dict(bias=at(1) + 1), ALIGN), (dict(num=at(2) + 2), ALIGN),
    (dict(ids=at(3) + 2), ALIGN), (dict(offsets=at(7) + 1), ALIGN),
    (dict(logits=at(0) + 1, dtype=2), ALIGN),
    (dict(ws=None), ARG), (dict(ws=at(8) + 128), ARG), (dict(ws_bytes=64), ARG),
    (dict(ws=at(0)), ARG), (dict(slots=at(3)), ARG), (dict(ids=at(0) + 64), ARG),
    (dict(token_index=at(2)), ARG), (dict(offsets=at(1)), ARG), (dict(weights=at(8)), ARG),
])
def test_route_refusals(lib, change, want):
    assert route(lib, **change) == want


def test_route_workspace(lib):
    f = binding.load().w4a16_moe_route_workspace_bytes
    assert [f(T, 256, 8) for T in (0, 1, 16)] == [0, 0, 0]
    assert f(17, 256, 8) == 2 * 256 * 4             # counts of blocks of 16 tokens
    assert f(4097, 1000, 8) == 257 * 1000 * 4
    assert f((1 << 25) + 1, 64, 8) == f(100, 2000, 8) == f(100, 64, 65) == f(-1, 64, 8) == 0


def swiglu(lib, **change):
    a = dict(X=at(0), token_index=at(1), offsets=at(2), qweight=at(3), scales=at(4), H=at(5), T=10,
             R=40, E=8, F=96, K=64, group=32, dtype=2, ws=None, ws_bytes=0, stream=None)
    a.update(change)
    return lib.w4a16_gemm_grouped_swiglu(*a.values())


EXPERTS = [
    (dict(group=16), ARG), (dict(dtype=7), ARG), (dict(E=0), ARG), (dict(K=0), ARG),
    (dict(K=48), SHAPE), (dict(E=65536), SHAPE), (dict(K=(1 << 17) + 32), SHAPE),
    (dict(T=-1), ARG), (dict(qweight=None), ARG), (dict(scales=None), ARG),
    (dict(offsets=None), ARG), (dict(qweight=at(3) + 8), ALIGN), (dict(scales=at(4) + 2), ALIGN),
    (dict(offsets=at(2) + 2), ALIGN),
]


@pytest.mark.parametrize("change,want", EXPERTS + [
    (dict(R=0), OK), (dict(F=0), OK), (dict(R=-1), ARG), (dict(F=-1), ARG), (dict(T=0), ARG),
    (dict(F=1 << 31), SHAPE), (dict(R=1 << 31), SHAPE), (dict(R=1 << 30, F=1 << 20), SHAPE),
    (dict(X=None), ARG), (dict(token_index=None), ARG), (dict(H=None), ARG),
    (dict(X=at(0) + 8), ALIGN), (dict(H=at(5) + 1), ALIGN), (dict(H=at(5) + 2, dtype=0), ALIGN),
    (dict(token_index=at(1) + 1), ALIGN),
    (dict(H=at(0) + 128), ARG), (dict(H=at(3)), ARG), (dict(H=at(4)), ARG), (dict(H=at(2)), ARG),
    (dict(H=at(1)), ARG),
    # more workgroups than a launch takes
    (dict(R=65535, E=65535, F=40000, K=32, qweight=at(100), scales=at(200), H=at(300)), SHAPE),
    # 128 slots per expert: the tile kernel's limbs
    (dict(R=1024), ARG), (dict(R=1024, ws=at(6), ws_bytes=10), ARG),
    (dict(R=1024, ws=at(6) + 16, ws_bytes=1 << 30), ARG),
    (dict(R=1024, ws=at(0), ws_bytes=1 << 30), ARG), (dict(R=1024, ws=at(5), ws_bytes=1 << 30), ARG),
])
def test_swiglu_refusals(lib, change, want):
    assert swiglu(lib, **change) == want


def combine(lib, **change):
    a = dict(H=at(0), offsets=at(2), qweight=at(3), scales=at(4), slots=at(5), weights=at(6),
             Y=at(7), T=10, topk=4, E=8, N=96, K=64, group=32, dtype=1, ws=at(8),
             ws_bytes=1 << 30, stream=None)
    a.update(change)
    return lib.w4a16_gemm_grouped_combine(*a.values())


@pytest.mark.parametrize("change,want", EXPERTS + [
    (dict(T=0), OK), (dict(N=0), OK), (dict(topk=0), ARG), (dict(N=-1), ARG),
    (dict(T=1 << 30, topk=4), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(H=None), ARG), (dict(slots=None), ARG), (dict(weights=None), ARG), (dict(Y=None), ARG),
    (dict(H=at(0) + 4), ALIGN), (dict(Y=at(7) + 1), ALIGN), (dict(slots=at(5) + 2), ALIGN),
    (dict(weights=at(6) + 2), ALIGN),
    (dict(Y=at(0)), ARG), (dict(Y=at(5)), ARG), (dict(Y=at(6)), ARG), (dict(Y=at(8)), ARG),
    (dict(ws=None), ARG), (dict(ws_bytes=100), ARG), (dict(ws=at(8) + 64), ARG),
    (dict(ws=at(3)), ARG),
])
def test_combine_refusals(lib, change, want):
    assert combine(lib, **change) == want


def test_experts_workspaces(lib):
    import torch
    rows = 40 * 96 * 4
    f = pkg.w4a16_grouped_combine_workspace_bytes
    assert f(10, 4, 8, 96, 64, torch.float16) == rows
    assert f(10, 4, 8, 93, 64, torch.float16) == rows      # rows padded to 4 values
    assert f(10, 4, 8, 96, 64, torch.float32) == rows + 40 * 64 * 4 + 256  # and limbs
    assert f(0, 4, 8, 96, 64, torch.float16) == f(10, 0, 8, 96, 64, torch.float16) == 0
    g = pkg.w4a16_grouped_swiglu_workspace_bytes
    assert g(10, 40, 8, 96, 64, torch.bfloat16) == g(10, 40, 8, 96, 64, torch.float16) == 0
    kernel = pkg.w4a16_experts_kernel
    for dtype, most in ((torch.float32, 10), (torch.float16, 28), (torch.bfloat16, 28)):
        assert kernel(8 * most, 8, dtype) == pkg.W4A16_EXPERTS_SKINNY
        assert kernel(8 * most + 1, 8, dtype) == pkg.W4A16_EXPERTS_TILE
        assert kernel(3, 8, dtype) == pkg.W4A16_EXPERTS_SKINNY
        assert kernel(0, 8, dtype) == kernel(8, 0, dtype) == 0
    assert binding.load().w4a16_experts_kernel(8, 8, 3) == 0
    # limbs of rows padded to 64 features (two for fp32), one factor per row
    assert g(64, 40, 8, 96, 96, torch.float32) == 64 * 128 * 4 + 64 * 4
    assert g(1024, 4096, 8, 96, 96, torch.bfloat16) == 1024 * 128 * 2 + 1024 * 4
    assert g(1024, 4096, 8, 96, 96, torch.float32) == 1024 * 128 * 4 + 1024 * 4
    with pytest.raises(TypeError):
        g(10, 40, 8, 96, 64, torch.float64)


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        pkg.w4a16_moe_route(x, 2)
    with pytest.raises(TypeError):
        pkg.w4a16_gemm_grouped_swiglu(x, x, x, x, x)
    with pytest.raises(TypeError):
        pkg.w4a16_gemm_grouped_combine(x, x, x, x, x, x)
    with pytest.raises(TypeError):
        pkg.w4a16_moe_route(np.zeros((4, 64)), 2)


def test_every_entry_point_has_a_binding():
    declared = {n for n in binding.header_functions() if "moe" in n or "experts_kernel" in n or
                "grouped_swiglu" in n or "grouped_combine" in n}
    assert len(declared) == 7
    for name in declared:
        assert inspect.isfunction(getattr(pkg, name)), name
        assert name in binding._SIGS
