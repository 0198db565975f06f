"""The oracle of speculative steps against what fixes it: enumeration of all outcomes, the
decode attention's oracle node by node, and worked examples."""
import itertools

import numpy as np
import pytest

import oracle
from oracle import tree


def test_depths_and_ancestors():
    par = [-1, 0, 0, 1, 3, 2, -1, 6]
    assert tree.depths(par) == [0, 1, 1, 2, 3, 2, 0, 1]
    m = tree.ancestors(par)
    assert [np.flatnonzero(r).tolist() for r in m] == [
        [0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4], [0, 2, 5], [6], [6, 7]]


@pytest.mark.parametrize("window", [0, 3, 6])
def test_a_node_attends_like_a_sequence_of_its_path(window):
    """Each node's output is the decode attention of the context and its path alone."""
    rng = np.random.default_rng(1)
    Hq, Hkv, D, ps, ctx = 4, 2, 8, 4, 9
    par = [-1, 0, 0, 2, 1, 3]
    n = len(par)
    table = np.array([[0] * 6, [3, 1, 5, 2, -1, -1]])
    kc, vc = rng.standard_normal((2, Hkv, 6 * ps, D))
    q = rng.standard_normal((n, Hq, D))
    out = tree.tree_attention(q, kc, vc, table, [1], [ctx], [0, n], par, window, 0.3, ps)
    for t in range(n):
        path = np.flatnonzero(tree.ancestors(par)[t])
        rows = [tree.cache_row(table, 1, j, ps) for j in list(range(ctx)) + list(ctx + path)]
        ident = np.array([np.arange(1), [0]])
        want = oracle.decode_attention(
            q[t:t + 1], kc[:, rows], vc[:, rows], ident.repeat(1, 1), np.array([1]),
            np.array([len(rows)]), window, 0.3, len(rows))
        assert np.allclose(out[t], want[0], atol=1e-12)


def _outcomes(target, draft, parents, V, sampled):
    """Distribution of the first new token over all drafts, by enumeration of the tokens and
    integration over the uniform numbers (a grid fine enough to be exact for these p, q)."""
    kids = [i for i, p in enumerate(parents) if p == 0]
    total = np.zeros(V)
    grid = (np.arange(16) + 0.5) / 16
    picks = (np.arange(64) + 0.5) / 64
    for toks in itertools.product(range(V), repeat=len(kids)):
        pr = (np.prod([draft[0, t] for t in toks]) if sampled
              else float(toks == tuple(range(len(kids)))))
        if pr == 0:
            continue
        tokens = np.zeros(len(parents), int)
        tokens[kids] = toks
        for us in itertools.product(grid, repeat=len(kids)):
            u = np.zeros(len(parents))
            u[kids] = us
            acc, path, _ = tree.tree_verify(target, draft if sampled else None, tokens,
                                            [0, len(parents)], parents, u, [0.5], len(parents))
            w = pr / len(grid) ** len(kids)
            if acc[0]:
                total[tokens[path[0, 1]]] += w
                continue
            for x in picks:
                _, _, nxt = tree.tree_verify(target, draft if sampled else None, tokens,
                                             [0, len(parents)], parents, u, [x], len(parents))
                total[nxt[0]] += w / len(picks)
    return total


@pytest.mark.parametrize("sampled", [True, False])
def test_the_targets_distribution_is_kept(sampled):
    """Two siblings: whatever the draft, the token after node 0 is distributed as the target
    says. Thresholds u q S < w fall between the grid's points up to 1/16 of each test and 1/64
    of each pick, so the total is within their sum."""
    p = np.array([[0.5, 0.25, 0.25], [0.2, 0.3, 0.5], [0.1, 0.1, 0.8]])
    q = np.array([[0.25, 0.25, 0.5], [0.4, 0.3, 0.3], [0.3, 0.3, 0.4]])
    got = _outcomes(p, q, [-1, 0, 0], 3, sampled)
    assert abs(got.sum() - 1) < 1e-9
    assert np.abs(got - p[0]).max() < 1 / 16 / 2 + 1 / 64, got


def test_residual_by_its_single_number():
    """w_k = max(p - a_k q, 0), a_k+1 = a_k + S_k equals the normalised residual."""
    rng = np.random.default_rng(2)
    for _ in range(50):
        p, q = rng.dirichlet(np.full(9, 0.5), 2)
        dist, a, s = p, 0.0, 1.0
        for _ in range(3):
            a += s
            w = np.maximum(p - a * q, 0)
            s = w.sum()
            dist = np.maximum(dist - q, 0)
            if dist.sum() < 1e-9:
                break
            dist /= dist.sum()
            assert np.allclose(w / s, dist, atol=1e-9)


def test_worked_example_of_a_walk():
    p = np.array([[0.5, 0.5, 0, 0], [0, 0, 1.0, 0], [0.25] * 4, [0, 0, 0, 1.0]])
    tokens, parents = [7, 1, 2, 0], [-1, 0, 1, 0]
    acc, path, nxt = tree.tree_verify(p, None, tokens, [0, 4], parents, [0, .4, .9, 0], [.6], 4)
    assert acc[0] == 2 and path[0].tolist() == [0, 1, 2, -1] and nxt[0] == 2
    acc, path, nxt = tree.tree_verify(p, None, tokens, [0, 4], parents, [0, .6, .9, .3], [.6], 4)
    assert acc[0] == 1 and path[0].tolist() == [0, 3, -1, -1] and nxt[0] == 3


def test_keep_path_moves_in_order():
    table = np.array([[0, 0], [2, 1]])
    cache = np.arange(12.0).reshape(1, 12, 1)
    tree.keep_path(cache, table, [1], [1], [2], [[0, 2, 3, -1]], 4)
    # tokens 1 + (2, 3) -> 1 + (1, 2): rows 8 + 3, 4 -> 8 + 2, 8 + 3
    assert cache[0, :, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 4]
