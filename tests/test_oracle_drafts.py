"""Pins of the oracle that the calls on drafted tokens are tested with: what a
node sees, and that the walk's tokens are distributed as the target's."""

import numpy as np
import pytest

from oracle import drafts as D


def test_lines_and_what_a_node_sees():
    parent = [-1, 0, 0, 1, 1, 3, 2]
    assert D.line(parent, 5) == [0, 1, 3, 5] and D.line(parent, 6) == [0, 2, 6] and D.line(parent, 0) == [0]
    assert D.sees(parent, 5, 10) == list(range(10)) + [10, 11, 13, 15]
    assert D.sees(parent, 6, 0) == [0, 2, 6]
    # positions: node 5 is at row0 + 3
    assert D.sees(parent, 5, 10, 8) == [8, 9, 10, 11, 13, 15]
    assert D.sees(parent, 5, 10, 12) == [13, 15] and D.sees(parent, 5, 10, 13) == [15] and D.sees(parent, 5, 10, 14) == []
    # a chain is causal
    chain = D.tree(None, 5, "chain")
    for j in range(5):
        assert D.sees(chain, j, 7) == list(range(8 + j))


def outcomes(parent, target, draft, tokens, weight, n_u=400):
    """The distribution of the first new token over uniform random numbers on a
    grid's middles (exact as all probabilities are multiples of its step)."""
    V = target.shape[1]
    got = np.zeros(V)
    grid = (np.arange(n_u) + 0.5) / n_u
    kids = [j for j in range(1, len(parent)) if parent[j] == 0]
    for u in np.stack(np.meshgrid(*[grid] * len(kids), indexing="ij"), -1).reshape(-1, len(kids)) if kids else [()]:
        un = np.full(len(parent), 0.25)
        un[kids] = u
        path, out, _ = D.verify(parent, tokens, target, draft, un)
        if len(path) > 1:
            got[out[0]] += 1
        else:
            # the last draw's distribution: what is left, by its own numbers
            for u0 in grid:
                un[0] = u0
                got[D.verify(parent, tokens, target, draft, un)[1][0]] += 1 / n_u
    return weight * got / n_u ** len(kids)


def test_a_sampled_draft_gives_the_target():
    """One child drawn from q: sum over draws of q(x) times the outcome is p."""
    p = np.array([[0.5, 0.25, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25]])
    q = np.array([[0.25, 0.5, 0.125, 0.125], [1, 0, 0, 0]])
    total = sum(outcomes([-1, 0], p, q, [0, x], q[0, x], n_u=64) for x in range(4))
    assert np.allclose(total, p[0], atol=1 / 64)


def test_two_sampled_siblings_give_the_target():
    p = np.array([[0.5, 0.25, 0.25], [1, 0, 0], [1, 0, 0]])
    q = np.array([[0.25, 0.5, 0.25], [1, 0, 0], [1, 0, 0]])
    total = sum(outcomes([-1, 0, 0], p, q, [0, x, y], q[0, x] * q[0, y], n_u=24) for x in range(3) for y in range(3))
    assert np.allclose(total, p[0], atol=2 / 24)


@pytest.mark.parametrize("tokens", [[0, 1, 2], [0, 3, 3], [0, 0, 1]])
def test_chosen_siblings_give_the_target(tokens):
    """Without the draft's probabilities, whatever was drafted."""
    p = np.array([[0.5, 0.25, 0.125, 0.125], [1, 0, 0, 0], [1, 0, 0, 0]])
    assert np.allclose(outcomes([-1, 0, 0], p, None, tokens, 1.0, n_u=32), p[0], atol=2 / 32)


def test_the_walk_by_hand():
    p = np.array([[0.1, 0.6, 0.3], [0.2, 0.0, 0.8], [0.5, 0.5, 0.0]])
    # 0 -> 1 (token 1), 1 -> 2 (token 2): both accepted, then 0 from [0.5, 0.5, 0]
    assert D.verify([-1, 0, 1], [0, 1, 2], p, None, [0.3, 0.59, 0.79])[:2] == ([0, 1, 2], [1, 2, 0])
    # the second rejected: from [0.2, 0, 0] there is only token 0
    assert D.verify([-1, 0, 1], [0, 1, 2], p, None, [0.99, 0.59, 0.81])[:2] == ([0, 1], [1, 0])
    # q: p / q = 0.75 for token 1, then max(p - q, 0) = [0, 0, 0.2]
    q = np.array([[0.1, 0.8, 0.1]] * 3)
    assert D.verify([-1, 0, 1], [0, 1, 2], p, q, [0.99, 0.76, 0.0])[:2] == ([0], [2])
    assert D.verify([-1, 0, -1], [0, 1, 2], p, q, [0.3, 0.74, 0.0])[:2] == ([0, 1], [1, 2])


def test_keep_moves_rows_together():
    assert D.keep(list("abcdefgh"), 2, [0, 2, 5]) == list("abcehfgh")
    assert D.keep(list("abc"), 0, []) == list("abc")
