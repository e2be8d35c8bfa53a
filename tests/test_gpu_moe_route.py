"""GPU parity of the routing of tokens to experts (w4a16_moe_route): choices and
slot lists equal to the oracle's, weights within their rounding."""

import sys

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import int4_weight_only_03_amd as pkg  # noqa: E402

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm device")
    pkg.load()
    return torch.device("cuda:0")


def check(r, logits, topk, E, bias=None, num_tokens=None, **options):
    """r against the oracle on the logits' values.  Each weight is a quotient of two
    64-bit numbers whose inputs are exact, but for the fp32 terms (2 ulp each) of a
    softmax sum; it is rounded once: 3 * 2^-23 covers both."""
    ids, w = oracle.route(logits, topk, bias=bias, num_tokens=num_tokens, **options)
    slots, tok, off = oracle.slot_lists(ids, E)
    torch.cuda.synchronize()
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.expert_offsets.cpu().numpy(), off)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.array_equal(r.token_index.cpu().numpy(), tok)
    got = r.weights.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w) <= 3 * 2.0 ** -23 * np.abs(w) + 2.0 ** -149)
    return ids


def run(dev, logits, topk, dtype="fp32", bias=None, num_tokens=None, **options):
    """(result, the logits as the type holds them)"""
    x = torch.from_numpy(np.ascontiguousarray(logits)).float().to(TYPES[dtype])
    b = None if bias is None else torch.tensor(bias, dtype=torch.float32, device=dev)
    n = None if num_tokens is None else torch.tensor([num_tokens], dtype=torch.int32, device=dev)
    r = pkg.w4a16_moe_route(x.to(dev), topk, bias=b, num_tokens=n, **options)
    return r, x.float().numpy()


def case(T, E, topk, dtype="fp32", bias=False, n=None, **options):
    return pytest.param(T, E, topk, dtype, bias, n, options,
                        id=f"{T}x{E}k{topk}{dtype}{'b' if bias else ''}" +
                        "".join(str(v) for v in options.values()))


SHAPES = [
    case(1, 1, 1), case(1, 2, 1, "bf16"), case(1, 256, 8, bias=True, score="sigmoid", groups=8,
                                               group_limit=4, group_top=2, scale=2.5),
    case(3, 5, 5, "fp16", score="sigmoid"), case(16, 32, 4), case(17, 63, 6, "bf16", bias=True),
    case(64, 64, 32), case(64, 65, 3, "fp16", renormalize=False),
    case(64, 160, 6, "bf16", groups=8, group_limit=3, renormalize=False, scale=16.0),
    case(65, 128, 8, groups=4, group_limit=2), case(66, 129, 1, bias=True),
    case(100, 257, 10, bias=True, score="sigmoid", renormalize=False),
    case(100, 511, 8, "bf16", groups=7, group_limit=3, group_top=2),
    case(130, 512, 8, groups=64, group_limit=5, group_top=2, bias=True),
    case(70, 1000, 16, groups=8, group_limit=8, bias=True),
    case(33, 1024, 32, groups=32, group_limit=4, group_top=2, bias=True, score="sigmoid"),
    case(1000, 1024, 4, "fp16", bias=True), case(4097, 60, 4, "bf16"),
    case(5000, 8, 2, bias=True, score="sigmoid"), case(333, 66, 6, groups=22, group_limit=9),
    case(64, 48, 5, n=61), case(64, 48, 5, n=0), case(300, 48, 5, "bf16", n=129, bias=True),
    case(300, 48, 5, n=1000), case(300, 48, 5, n=-7),
]


@pytest.mark.parametrize("T,E,topk,dtype,bias,n,options", SHAPES)
def test_route_shapes(dev, T, E, topk, dtype, bias, n, options):
    say("route", T, E, topk, dtype, bias, n, options)
    rng = np.random.default_rng(T * 7 + E)
    logits = 1.5 * rng.standard_normal((T, E))
    b = 0.1 * rng.standard_normal(E) if bias else None
    b = None if b is None else b.astype(np.float32)
    r, x = run(dev, logits, topk, dtype, b, n, **options)
    check(r, x, topk, E, b, n, **options)


@pytest.mark.parametrize("T", [9, 130])
@pytest.mark.parametrize("options", [dict(), dict(score="sigmoid"),
                                     dict(groups=6, group_limit=2),
                                     dict(groups=6, group_limit=4, group_top=2, score="sigmoid")])
@pytest.mark.parametrize("bias", [None, 0.0, 0.25])
def test_route_ties(dev, T, options, bias):
    """Few distinct logits: equal keys go to the lowest index, equal groups too."""
    rng = np.random.default_rng(T)
    logits = rng.integers(0, 3, (T, 72)).astype(np.float32)
    logits[0] = 0.0
    b = None if bias is None else np.full(72, bias, np.float32)
    r, x = run(dev, logits, 7, bias=b, **options)
    check(r, x, 7, 72, b, **options)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_keys_next_to_each_other(dev, score):
    """Keys that differ by far less than fp32 tells apart: the logits of each token
    differ, and the bias undoes the differences of token 0's scores to fp32."""
    rng = np.random.default_rng(5)
    T, E, topk = 200, 96, 8
    base = rng.standard_normal(E)
    logits = np.tile(base, (T, 1)).astype(np.float32)
    logits += rng.integers(-3, 4, (T, E)) * np.float32(2.0 ** -22)
    x = logits[0].astype(np.float64)
    s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x) / np.exp(x).sum()
    b = (0.75 - s).astype(np.float32)
    for options in (dict(), dict(groups=8, group_limit=3, group_top=2)):
        r, xv = run(dev, logits, topk, bias=b, score=score, **options)
        check(r, xv, topk, E, b, score=score, **options)


@pytest.mark.parametrize("T", [6, 80])
def test_route_masked_experts(dev, T):
    """-inf and NaN logits and biases, rows with too few experts or none, +inf."""
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(8)
    logits = rng.standard_normal((T, 24)).astype(np.float32)
    logits[0] = -inf
    logits[1] = nan
    logits[2, 2:] = -inf
    logits[3, :20] = nan
    logits[4, [3, 9]] = inf
    logits[5, 6:12] = -inf
    b = (0.1 * rng.standard_normal(24)).astype(np.float32)
    bm = b.copy()
    bm[[0, 7, 8]] = [-inf, nan, inf]
    for bias in (None, b, bm):
        for options in (dict(), dict(score="sigmoid", renormalize=False),
                        dict(groups=4, group_limit=2, group_top=2),
                        dict(score="sigmoid", groups=4, group_limit=1)):
            say("masked", T, bias is not None, options)
            r, x = run(dev, logits, 5, bias=bias, **options)
            check(r, x, 5, 24, bias, **options)


def test_route_far_logits(dev):
    """Logits that reach far: scores underflow fp32 and 64 bits."""
    rng = np.random.default_rng(9)
    logits = (rng.standard_normal((40, 50)) * 10.0 ** rng.integers(0, 5, (40, 1))).astype(np.float32)
    for options in (dict(), dict(renormalize=False), dict(score="sigmoid"),
                    dict(score="sigmoid", renormalize=False)):
        r, x = run(dev, logits, 6, **options)
        check(r, x, 6, 50, **options)


def test_route_nothing(dev):
    r = pkg.w4a16_moe_route(torch.empty(0, 8, device=dev), 2)
    torch.cuda.synchronize()
    assert r.expert_offsets.tolist() == [0] * 9 and r.ids.shape == (0, 2)


@pytest.mark.parametrize("T", [13, 700])
def test_route_writes_its_outputs_only(dev, T):
    """Every buffer between guard words; twice the same bits."""
    E, topk, pad = 40, 3, 64
    sizes = [T * topk] * 4 + [E + 1]
    need = pkg.w4a16_moe_route_workspace_bytes(T, E, topk)
    x = torch.randn(T, E, device=dev)
    got = []
    for _ in range(2):
        raw = [torch.full((n + 2 * pad,), 0x7FC0DEAD, dtype=torch.int32, device=dev) for n in sizes]
        ws = torch.full((need // 4 + 2 * pad,), 0x7FC0DEAD, dtype=torch.int32, device=dev)
        v = [b[pad:pad + n] for b, n in zip(raw, sizes)]
        out = pkg.W4A16Routing(v[0].view(T, topk), v[1].view(torch.float32).view(T, topk),
                               v[2].view(T, topk), v[3], v[4])
        r = pkg.w4a16_moe_route(x, topk, out=out,
                                workspace=ws[pad:pad + need // 4].view(torch.uint8))
        torch.cuda.synchronize()
        assert r is out
        for b in raw + [ws]:
            assert torch.all(b[:pad] == 0x7FC0DEAD) and torch.all(b[-pad:] == 0x7FC0DEAD)
        got.append([b.clone() for b in raw])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    check(r, x.cpu().numpy(), topk, E)


@pytest.mark.parametrize("T", [64, 300])
def test_route_in_a_graph_and_on_another_stream(dev, T):
    """Replays with new logits and another number of tokens, eager work between."""
    E, topk = 64, 6
    x = torch.randn(T, E, device=dev)
    n = torch.tensor([T], dtype=torch.int32, device=dev)
    ws = torch.empty(max(pkg.w4a16_moe_route_workspace_bytes(T, E, topk), 1), dtype=torch.uint8,
                     device=dev)
    out = pkg.w4a16_moe_routing(T, E, topk, dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = pkg.w4a16_moe_route(x, topk, num_tokens=n, stream=side)
    side.synchronize()
    check(r, x.cpu().numpy(), topk, E)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.w4a16_moe_route(x, topk, num_tokens=n, out=out, workspace=ws)
    for i in range(3):
        x.copy_(torch.randn(T, E, device=dev))
        n.fill_(T - 7 * i)
        pkg.w4a16_moe_route(x, 3)
        g.replay()
        torch.cuda.synchronize()
        check(out, x.cpu().numpy(), topk, E, num_tokens=T - 7 * i)
