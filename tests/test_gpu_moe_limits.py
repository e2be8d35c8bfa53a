"""The mixture-of-experts entry points at the ends of their ranges: non-finite and
subnormal activations, buffers past 2^31 elements, single and many tokens, two
calls at once."""

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


def weights_of(rng, E, rows, K):
    qw = rng.integers(-(2 ** 31), 2 ** 31, (E, rows, K // 8), dtype=np.int64).astype(np.int32)
    return qw, (0.003 + 0.002 * rng.random((E, rows, K // 32))).astype(np.float32)


def on(dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def close(got, want, tol, what):
    err = np.abs(got.double().cpu().numpy() - want)
    say(f"  {what}: max err/bound {np.max(err / tol):.3e}")
    assert np.all(err <= tol)


def tile(R, E, dtype):
    return pkg.w4a16_experts_kernel(R, E, TYPES[dtype]) == pkg.W4A16_EXPERTS_TILE


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [6, 90])
def test_non_finite_rows_stay_in_their_rows(dev, T, dtype):
    """A row with an infinity or NaN makes its own slots non-finite and no others."""
    E, F, K = 2, 40, 160
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, K)).astype(np.float32)
    bad = [1, 3, T - 1]
    x[1, 5], x[3, 159], x[T - 1, 64] = np.inf, np.nan, -np.inf
    X = torch.from_numpy(x).to(TYPES[dtype])
    good = X.float().numpy().copy()
    good[bad] = 0.0
    tok = np.concatenate([np.arange(T), np.arange(T)]).astype(np.int32)
    off = np.array([0, T, 2 * T], np.int32)
    gq, gs = weights_of(rng, E, 2 * F, K)
    say("non-finite", T, dtype, "tile", tile(2 * T, E, dtype))
    H = pkg.w4a16_gemm_grouped_swiglu(X.to(dev), *on(dev, tok, off, gq, gs))
    want, tol = oracle.experts_swiglu(good, tok, off, gq, gs, dtype, tile(2 * T, E, dtype))
    rows = np.isin(tok, bad)
    assert not torch.isfinite(H[torch.from_numpy(rows).to(dev)]).any()
    close(H[torch.from_numpy(~rows).to(dev)], want[~rows], tol[~rows], "swiglu")

    dq, ds = weights_of(rng, E, F, K)
    slots = np.stack([np.arange(T), T + np.arange(T)], 1).astype(np.int32)
    w = rng.random((T, 2)).astype(np.float32) - 0.5
    Hx = torch.cat([X, X.roll(2, 0)]).to(dev)
    Hg = np.concatenate([good, np.roll(good, 2, 0)])
    Y = pkg.w4a16_gemm_grouped_combine(Hx, *on(dev, off, dq, ds, slots, w))
    want, tol = oracle.experts_combine(Hg, off, dq, ds, slots, w, dtype, tile(2 * T, E, dtype))
    hit = ~np.isfinite(Hx.float().cpu().numpy()).all(1)[slots]
    hit = hit.any(1)
    assert hit.any() and (~hit).any()
    assert not torch.isfinite(Y[torch.from_numpy(hit).to(dev)]).any()
    close(Y[torch.from_numpy(~hit).to(dev)], want[~hit], tol[~hit], "combine")


@pytest.mark.parametrize("dtype,down,up", [("fp32", -130, 80), ("bf16", -130, 80), ("fp16", -18, 18)])
@pytest.mark.parametrize("T", [6, 90])
def test_subnormal_activations(dev, T, dtype, down, up):
    """Rows of subnormal numbers: powers of two pass through every product exactly, so
    the result is that of the same digits at ordinary size."""
    E, N, K = 2, 40, 160
    rng = np.random.default_rng(T + up)
    x = np.ldexp(rng.standard_normal((2 * T, K)), down)
    X = torch.from_numpy(x).to(TYPES[dtype])
    digits = np.ldexp(X.double().numpy(), -down).astype(np.float32)
    off = np.array([0, T, 2 * T], np.int32)
    qw, sc = weights_of(rng, E, N, K)
    slots = np.stack([np.arange(T), T + np.arange(T)], 1).astype(np.int32)
    w = rng.standard_normal((T, 2)).astype(np.float32)
    big = tile(2 * T, E, dtype)
    say("subnormal", T, dtype, "tile", big)
    Y = pkg.w4a16_gemm_grouped_combine(X.to(dev),
                                       *on(dev, off, qw, np.ldexp(sc, up), slots, w))
    want, tol = oracle.experts_combine(digits, off, qw, sc, slots, w, dtype, big)
    close(Y.double() * 2.0 ** -(down + up), want, tol, "combine")


@pytest.mark.parametrize("dtype,per", [("bf16", 1), ("fp16", 32), ("fp32", 12)])
def test_weights_past_4_gib(dev, dtype, per):
    E, F, K = 300, 1024, 14336
    T = 40
    gen = torch.Generator(dev).manual_seed(per)
    qw = torch.randint(-(2 ** 31), 2 ** 31, (E, 2 * F, K // 8), dtype=torch.int32, device=dev,
                       generator=gen)
    sc = 0.003 + 0.002 * torch.rand(E, 2 * F, K // 32, device=dev, generator=gen)
    X = torch.randn(T, K, device=dev, generator=gen).to(TYPES[dtype])
    tok = torch.randint(0, T, (E * per,), dtype=torch.int32, device=dev, generator=gen)
    off = torch.arange(0, E * per + 1, per, dtype=torch.int32, device=dev)
    say("4 GiB", dtype, per, qw.numel() * 4)
    H = pkg.w4a16_gemm_grouped_swiglu(X, tok, off, qw, sc)
    for e in (0, 146, E - 1):
        one = slice(e * per, (e + 1) * per)
        want, tol = oracle.experts_swiglu(X.float().cpu().numpy(), tok[one].cpu().numpy(),
                                          np.array([0, per], np.int32), qw[e:e + 1].cpu().numpy(),
                                          sc[e:e + 1].cpu().numpy(), dtype, tile(E * per, E, dtype))
        close(H[one], want, tol, f"expert {e}")


def test_more_than_2_31_outputs(dev):
    T, N, K, E = 600000, 4096, 32, 2
    rng = np.random.default_rng(1)
    x = torch.randn(T, K, device=dev).bfloat16()
    tok = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=dev)
    off = np.array([0, 250001, T], np.int32)
    gq, gs = weights_of(rng, E, 2 * N, K)
    say("outputs", T * N)
    H = pkg.w4a16_gemm_grouped_swiglu(x, tok, *on(dev, off, gq, gs))
    pick = [0, 1, 250000, 250001, 524287, 524288, T - 1]
    xs = x.float().cpu().numpy()
    for r in pick:
        e = int(r >= off[1])
        want, tol = oracle.experts_swiglu(xs, np.array([T - 1 - r], np.int32),
                                          np.array([0, 1], np.int32), gq[e:e + 1], gs[e:e + 1],
                                          "bf16", True)
        close(H[r:r + 1], want, tol, f"row {r}")
    del H
    dq, ds = weights_of(rng, E, N, K)
    slots = torch.arange(T, dtype=torch.int32, device=dev).view(T, 1).roll(7, 0).contiguous()
    w = torch.rand(T, 1, device=dev)
    Y = pkg.w4a16_gemm_grouped_combine(x, *on(dev, off, dq, ds), slots, w)
    for t in pick + [T - 8]:
        r = int(slots[t])
        e = int(r >= off[1])
        want, tol = oracle.experts_combine(xs[r:r + 1], np.array([0, 1], np.int32), dq[e:e + 1],
                                           ds[e:e + 1], np.zeros((1, 1), np.int32),
                                           w[t:t + 1].cpu().numpy(), "bf16", True)
        close(Y[t:t + 1], want, tol, f"token {t}")


def lists_agree(r, E, topk):
    """slots, token_index and expert_offsets against a stable sort of the choices"""
    ids = r.ids.flatten().long()
    order = torch.sort(ids, dim=-1, stable=True).indices
    assert torch.equal(r.token_index.long(), order // topk)
    assert torch.equal(r.slots.flatten().long()[order], torch.arange(len(ids), device=ids.device))
    counts = torch.bincount(ids, minlength=E)
    assert torch.equal(r.expert_offsets[1:].long(), counts.cumsum(0)) and r.expert_offsets[0] == 0


@pytest.mark.parametrize("T,E,topk,dtype,options", [
    (2200000, 1024, 2, "bf16", dict()),  # more than 2^31 logits
    (70001, 4, 1, "fp32", dict(score="sigmoid")),
    (40000, 192, 6, "fp16", dict(groups=8, group_limit=3, group_top=2)),
    (17001, 256, 16, "bf16", dict(groups=16, group_limit=4)),
    (4200, 250, 8, "fp32", dict(score="sigmoid", bias=0.1, groups=10, group_limit=4, group_top=2)),
    (4200, 150, 8, "fp32", dict(bias=0.01)),
])
def test_route_many_tokens(dev, T, E, topk, dtype, options):
    x = torch.randn(T, E, dtype=TYPES[dtype], device=dev)
    say("route", T, E, topk, dtype, options)
    bias = options.get("bias")
    if bias is not None:
        bias = bias * torch.randn(E, device=dev)
    r = pkg.w4a16_moe_route(x, topk, **dict(options, bias=bias))
    options = dict(options, bias=None if bias is None else bias.cpu().numpy())
    lists_agree(r, E, topk)
    for part in (slice(0, 200), slice(T // 2, T // 2 + 200), slice(T - 200, T)):
        ids, w = oracle.route(x[part].float().cpu().numpy(), topk, **options)
        assert np.array_equal(r.ids[part].cpu().numpy(), ids)
        assert np.allclose(r.weights[part].cpu().numpy(), w, rtol=3 * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 18, 63, 64, 65])
@pytest.mark.parametrize("E,topk,groups", [(193, 3, 1), (256, 8, 8), (256, 17, 4), (40, 2, 20),
                                           (1, 1, 1), (1024, 32, 64)])
@pytest.mark.parametrize("live", [None, 0, 1])
def test_route_few_tokens(dev, T, E, topk, groups, live):
    """Each lane layout on both sides of its bounds, with and without a bias."""
    rng = np.random.default_rng(T * E)
    x = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    limit = max(1, min(groups, -(-topk * groups // E)))
    n = None if live is None else torch.tensor([live], dtype=torch.int32, device=dev)
    for b in (None, bias):
        r = pkg.w4a16_moe_route(torch.from_numpy(x).to(dev), topk,
                                bias=None if b is None else torch.from_numpy(b).to(dev),
                                groups=groups, group_limit=limit, num_tokens=n)
        ids, w = oracle.route(x, topk, bias=b, groups=groups, group_limit=limit, num_tokens=live)
        slots, tok, off = oracle.slot_lists(ids, E)
        for got, want in zip((r.ids, r.slots, r.token_index, r.expert_offsets),
                             (ids, slots, tok, off)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.allclose(r.weights.cpu().numpy(), w, rtol=3 * 2.0 ** -23, atol=0)


def test_two_layers_at_once(dev):
    """Two streams, each with its own buffers, against the same calls one by one."""
    E, topk, F, K, N = 8, 2, 96, 256, 160
    rng = np.random.default_rng(4)
    gq, gs, dq, ds = on(dev, *weights_of(rng, E, 2 * F, K), *weights_of(rng, E, N, F))
    cases = [(300, torch.bfloat16), (24, torch.float32), (700, torch.float16), (1, torch.bfloat16)]
    inputs = [(torch.randn(T, E, device=dev), torch.randn(T, K, device=dev).to(t))
              for T, t in cases]

    def layer(logits, X, stream=None):
        r = pkg.w4a16_moe_route(logits, topk, stream=stream)
        H = pkg.w4a16_gemm_grouped_swiglu(X, r.token_index, r.expert_offsets, gq, gs,
                                          stream=stream)
        return pkg.w4a16_gemm_grouped_combine(H, r.expert_offsets, dq, ds, r.slots, r.weights,
                                              stream=stream)

    want = [layer(*i) for i in inputs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [layer(*i, stream=streams[j % 2]) for j, i in enumerate(inputs)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_share_a_workspace(dev):
    """Graphs of different batches on one workspace, replayed in turn with eager calls
    on the same workspace between them."""
    E, topk, F, K, N = 6, 2, 64, 160, 96
    rng = np.random.default_rng(11)
    gq, gs, dq, ds = on(dev, *weights_of(rng, E, 2 * F, K), *weights_of(rng, E, N, F))
    batches = [(40, torch.float32), (9, torch.float32), (300, torch.bfloat16)]
    need = max(max(pkg.w4a16_moe_route_workspace_bytes(T, E, topk),
                   pkg.w4a16_grouped_swiglu_workspace_bytes(T, T * topk, E, F, K, t),
                   pkg.w4a16_grouped_combine_workspace_bytes(T, topk, E, N, F, t))
               for T, t in batches)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    inputs = [(torch.randn(T, E, device=dev), torch.randn(T, K, device=dev).to(t))
              for T, t in batches]

    def layer(logits, X):
        r = pkg.w4a16_moe_route(logits, topk, workspace=ws)
        H = pkg.w4a16_gemm_grouped_swiglu(X, r.token_index, r.expert_offsets, gq, gs, workspace=ws)
        return pkg.w4a16_gemm_grouped_combine(H, r.expert_offsets, dq, ds, r.slots, r.weights,
                                              workspace=ws)

    graphs = []
    for i in inputs:
        layer(*i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, layer(*i)))
    for turn in range(3):
        for (T, t), i, (g, out) in zip(batches, inputs, graphs):
            i[0].copy_(torch.randn(T, E, device=dev))
            i[1].copy_(torch.randn(T, K, device=dev))
            out.zero_()
            g.replay()
            assert torch.equal(layer(*i), out)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("topk,E,N,K", [
    # waves of a slot: 4, 2 and 1, and K of fewer blocks than waves
    (1, 1, 1, 32), (1, 5, 33, 2080), (3, 9, 100, 2048), (4, 7, 31, 96), (8, 64, 65, 1056),
    (8, 130, 7168, 512), (5, 40, 97, 544), (16, 20, 300, 160), (9, 9, 64, 608),
    (17, 33, 70, 96),                      # more choices than a workgroup's waves
    (4, 6, 40, 8192), (16, 16, 64, 4096),  # workgroups too few for so much to read
])
def test_combine_of_one_token(dev, topk, E, N, K, dtype):
    """Slots in any order, one of them named twice, some without an expert."""
    rng = np.random.default_rng(topk * N + K)
    ids = rng.permutation(E)[:topk].astype(np.int32)[None]
    slots, _, off = oracle.slot_lists(ids, E)
    qw, sc = weights_of(rng, E, N, K)
    x = rng.standard_normal((topk, K)).astype(np.float32)
    X = torch.from_numpy(x).to(TYPES[dtype])
    say("one token", topk, E, N, K, dtype)
    for change in range(3):
        s, w = slots.copy(), rng.standard_normal((1, topk)).astype(np.float32)
        if change == 1:
            s[0, -1] = s[0, 0]
        elif change == 2:
            s[0, ::2], w[0, ::2] = -1, np.nan
        buf = torch.full((N + 128,), 77.0, dtype=TYPES[dtype], device=dev)
        Y = pkg.w4a16_gemm_grouped_combine(X.to(dev), *on(dev, off, qw, sc, s, w),
                                           Y=buf[64:64 + N].view(1, N))
        want, tol = oracle.experts_combine(X.float().numpy(), off, qw, sc, s, w, dtype, False)
        close(Y, want, tol, f"change {change}")
        assert torch.all(buf[:64] == 77) and torch.all(buf[64 + N:] == 77)


def test_malformed_lists_of_one_token_stay_in_bounds(dev):
    E, topk, N, K = 4, 6, 70, 96
    rng = np.random.default_rng(3)
    qw, sc = on(dev, *weights_of(rng, E, N, K))
    X = torch.randn(topk, K, device=dev).half()
    w = torch.rand(1, topk, device=dev)
    buf = torch.full((N + 128,), 77.0, dtype=torch.half, device=dev)
    for off in ([-3, 99, 1, 4, 70], [9, 9, 9, 9, 9], [0, 0, 0, 0, 0], [6, 5, 4, 3, 2]):
        slots = torch.tensor([[-9, 99, 5, 0, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=dev)
        pkg.w4a16_gemm_grouped_combine(X, torch.tensor(off, dtype=torch.int32, device=dev), qw, sc,
                                       slots, w, Y=buf[64:64 + N].view(1, N))
    torch.cuda.synchronize()
    assert torch.all(buf[:64] == 77) and torch.all(buf[64 + N:] == 77)
