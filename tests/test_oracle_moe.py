"""The oracle of the mixture-of-experts layer against hand-sized cases and
closed forms (CPU only)."""

import numpy as np
import pytest

import oracle
import workloads


def test_route_by_hand():
    # softmax of log-probabilities gives the probabilities back
    p = np.array([[0.1, 0.4, 0.2, 0.3]])
    ids, w = oracle.route(np.log(p), 2, renormalize=False)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[0.4, 0.3]], rtol=1e-14)
    ids, w = oracle.route(np.log(p), 2, scale=2.0)
    assert np.allclose(w, [[2 * 0.4 / 0.7, 2 * 0.3 / 0.7]], rtol=1e-14)
    # a bias changes the choice, not the weights
    ids, w = oracle.route(np.log(p), 2, bias=[1.0, 0.0, 0.0, 0.0], renormalize=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.1, 0.4]], rtol=1e-14)
    # sigmoid
    ids, w = oracle.route([[0.0, 1.0]], 1, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[1]] and np.isclose(w[0, 0], 1 / (1 + np.exp(-1.0)), rtol=1e-14)


def test_route_ties_groups_and_masks():
    assert oracle.route([[2.0, 2.0, 2.0]], 2)[0].tolist() == [[0, 1]]
    x = [[3.0, -9.0, 2.0, 2.5]]  # groups {0, 1} and {2, 3}
    assert oracle.route(x, 2, groups=2, group_limit=1, group_top=1)[0].tolist() == [[0, 1]]
    assert oracle.route(x, 2, score="sigmoid", groups=2, group_limit=1,
                        group_top=2)[0].tolist() == [[3, 2]]
    inf = np.inf
    ids, w = oracle.route([[-inf, np.nan, 1.0, -inf], [-inf] * 4, [0.0] * 4], 2, num_tokens=2)
    assert ids.tolist() == [[2, -1], [-1, -1], [-1, -1]]
    assert w.tolist() == [[1.0, 0.0], [0.0, 0.0], [0.0, 0.0]]
    ids, _ = oracle.route([[0.0, 1.0, 2.0, 3.0]], 2, bias=[0.0, 0.0, -inf, np.nan])
    assert ids.tolist() == [[1, 0]]
    # a group without an open expert is never entered
    ids, _ = oracle.route([[-inf, -inf, 1.0, 2.0]], 3, groups=2, group_limit=1)
    assert ids.tolist() == [[3, 2, -1]]
    # +inf: shared among the experts that have it
    ids, w = oracle.route([[inf, 0.0, inf]], 2, renormalize=False)
    assert ids.tolist() == [[0, 2]] and w.tolist() == [[0.5, 0.5]]


def test_slot_lists_by_hand():
    slots, tok, off = oracle.slot_lists(np.array([[2, 0], [-1, -1], [0, 2], [1, -1]]), 4)
    assert off.tolist() == [0, 2, 3, 5, 5]
    assert tok.tolist() == [0, 2, 3, 0, 2, -1, -1, -1]
    assert slots.tolist() == [[3, 0], [-1, -1], [1, 4], [2, -1]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_layer_against_dense_products(dtype):
    """Every token through its experts, written as a dense loop over tokens."""
    T, E, k, F, K, N = 5, 3, 2, 4, 64, 6
    rng = np.random.default_rng(1)
    X = rng.standard_normal((T, K)).astype(np.float32)
    ids, w = oracle.route(rng.standard_normal((T, E)), k)
    slots, tok, off = oracle.slot_lists(ids, E)
    gu = [oracle.quantize(workloads.random_case(1, 2 * F, K, e)[1]) for e in range(E)]
    H, tol = oracle.experts_swiglu(X, tok, off, np.stack([q for q, _ in gu]),
                                   np.stack([s for _, s in gu]), dtype)
    Hk = rng.standard_normal((T * k, 32)).astype(np.float32)
    dn = [oracle.quantize(workloads.random_case(1, N, 32, 9 + e)[1]) for e in range(E)]
    Y, _ = oracle.experts_combine(Hk, off, np.stack([q for q, _ in dn]),
                                  np.stack([s for _, s in dn]), slots, w, dtype)
    for t in range(T):
        y = np.zeros(N)
        for j in range(k):
            e = ids[t, j]
            W = oracle.dequantize(*gu[e]).astype(np.float64)
            g, u = W[:F] @ X[t], W[F:] @ X[t]
            assert np.allclose(H[slots[t, j]], g / (1 + np.exp(-g)) * u, rtol=1e-12)
            y += w[t, j] * (oracle.dequantize(*dn[e]).astype(np.float64) @ Hk[slots[t, j]])
        assert np.allclose(Y[t], y, rtol=1e-12)
    assert np.all(tol > 0)
