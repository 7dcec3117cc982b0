"""The draft operators' oracle on the CPU: small cases by hand, brute force, and the property that
verification exists for: what is emitted is distributed as the target says."""
import itertools

import numpy as np
import pytest

from draft_util import forest, random_parents, softmax
from oracle import attention_oracle as A
from oracle import draft_oracle as D


def test_ancestors_and_positions_by_hand():
    parents = [-1, 0, 0, 1, 2, 2, 5, 9]                # the last one's parent is no earlier node
    mask, pos = D.tree_mask(parents, [0, 8], 1, [20])
    want = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 2, 4}, {0, 2, 5}, {0, 2, 5, 6}, {7}]
    assert [int(m) for m in mask[:, 0]] == [sum(1 << j for j in s) for s in want]
    assert pos.tolist() == [12 + len(s) - 1 for s in want]


def test_a_chain_is_the_causal_mask():
    rng = np.random.default_rng(0)
    n, L, hq, d = 5, 40, 2, 64
    q = rng.standard_normal((n, hq, d))
    cache = [rng.integers(0, 256, (3, 1, 16, w)).astype(np.uint8) for w in (d // 2, d // 32)] * 2
    cache[1] = cache[3] = np.full((3, 1, 16, d // 32), 126, np.uint8)
    table = np.array([[2, 0, 1]])
    parents, starts = forest(rng, [n], "chain")
    mask, pos = D.tree_mask(parents, starts, 1, [L])
    for window in (0, 7):
        a = A.attention(q, *cache, table, [L], starts, 0.1, causal=True, window=window)
        if window:                                      # of the tree the mask alone takes
            mask = np.array([[sum(1 << j for j in range(max(0, i - window + 1), i + 1))] for i in range(n)], np.int32)
        b = D.attention(q, *cache, table, [L], starts, 0.1, mask, window, pos)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-13, atol=0)


@pytest.mark.parametrize("mode", ["drawn", "distinct", "chosen"])
def test_the_first_token_is_distributed_as_the_target(mode):
    # Exactly: all drafts of the root's two children, all outcomes of the two tests (each a rejection
    # with probability 1 - a, found by bisection on u), and the next token's distribution.
    rng = np.random.default_rng(1)
    V = 5
    for trial in range(4):
        p, q = softmax(rng.standard_normal(V)), softmax(rng.standard_normal(V))
        got = np.zeros(V)
        for x, y in itertools.product(range(V), repeat=2):
            if mode == "distinct":
                if x == y:
                    continue
                weight = q[x] * q[y] / (1 - q[x])
            elif mode == "drawn":
                weight = q[x] * q[y]
            else:
                order = np.argsort(-q)
                weight = float((x, y) == (order[0], order[1]))
            if weight == 0:
                continue
            rows = np.stack([p, p, p])
            drafts = None if mode == "chosen" else np.stack([q, q, q])

            def walk(u1, u2, s):
                return D.verify_one(rows, drafts, [0, x, y], [-1, 0, 0], [0, u1, u2], s, 2, mode == "drawn")

            def threshold(accepts):
                lo, hi = 0.0, 1.0
                if accepts(1.0 - 2.0 ** -40):
                    return 1.0
                for _ in range(50):
                    m = (lo + hi) / 2
                    lo, hi = (m, hi) if accepts(m) else (lo, m)
                return lo

            a1 = threshold(lambda u: walk(u, 1.0, 0.5)[0] == [0, 1])
            got[x] += weight * a1
            a2 = threshold(lambda u: walk(1.0, u, 0.5)[0] == [0, 2]) if a1 < 1 else 0.0
            got[y] += weight * (1 - a1) * a2
            left = weight * (1 - a1) * (1 - a2)
            if left > 1e-12:
                edges = np.linspace(0, 1, 4001)[:-1] + 1 / 8000
                told = np.bincount([walk(1.0, 1.0, s)[1][0] for s in edges], minlength=V) / 4000
                got += left * told
        # the last draw is integrated on a grid of 4000 points: each bin's edge is off by 1/4000 at most
        assert np.abs(got - p).max() < 2 / 4000, (mode, trial, got, p)


def test_edges_by_hand():
    one = np.array([[0.25, 0.5, 0.25, 0.0]] * 3)
    run = lambda **k: D.verify_one(**{**dict(target=one, draft=one, tokens=[0, 1, 2], parents=[-1, 0, 1],
                                             accept_u=[0, .9, .9], sample_u=0.0, width=3, replacement=True), **k})
    assert run() == ([0, 1, 2], [1, 2, 0])                       # p = q: everything stands
    assert run(width=2) == ([0, 1], [1, 0])                      # no place for the second
    assert run(tokens=[0, 9, 2]) == ([0], [0])                   # no such token; nothing is left of p - q: p
    assert run(tokens=[0, 3, 2], draft=None) == ([0], [0])
    assert run(sample_u=0.25) == ([0, 1, 2], [1, 2, 1])          # the sum has to exceed
    assert run(sample_u=1.0) == ([0, 1, 2], [1, 2, 2])           # the last that is there
    assert run(target=0 * one) == ([0], [-1])
    assert run(draft=None, tokens=[0, 1, 1], parents=[-1, 0, 0], accept_u=[0, .6, 0.0], sample_u=.5) == ([0], [2])


def test_accept_by_hand():
    cache = [np.arange(4 * 16, dtype=np.uint8).reshape(4, 1, 16, 1).copy() for _ in range(4)]
    table = np.array([[3, 1]])
    after, lens = D.accept(cache, table, [20], [0, 6], np.array([[0, 2, 5, -1]]), [3])
    assert lens.tolist() == [17]
    want = cache[0].copy()
    want[3, 0, 15], want[1, 0, 0] = cache[0][1, 0, 0], cache[0][1, 0, 3]      # 15 <- 16, 16 <- 19
    assert all(np.array_equal(a, want) for a in after)


def test_random_trees_are_trees():
    rng = np.random.default_rng(3)
    for n in (1, 2, 33, 200):
        p = random_parents(rng, n)
        assert len(p) == n and p[0] == -1 and all(0 <= p[i] < i for i in range(1, n))
