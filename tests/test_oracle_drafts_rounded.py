"""Pins of the walk where rounded probabilities leave nothing after a rejection."""

import numpy as np
import pytest

from oracle import drafts as D


def bf16(p):
    u = np.asarray(p, dtype=np.float32).view(np.uint32)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)


P, Q = bf16([0.9995, 0.0002, 0.0002, 0.0001]), bf16([0.9985, 0.0006, 0.0005, 0.0004])


def test_the_last_token_is_the_targets_own():
    """Both rows hold 1 at token 0 and the draft more elsewhere, so nothing is
    left of p - q: the last token is drawn from p."""
    assert P[0] == Q[0] == 1 and np.all(P[1:] < Q[1:])
    # (P sums to about 1.0005: 0.99975 of that is 1.00025, past token 1's 1.0002)
    for u0, token in ((0.0, 0), (0.9, 0), (1 - 2.0 ** -24, 3), (0.99975, 2)):
        assert D.verify([-1, 0], [0, 1], [P, P], [Q, Q], [u0, 0.9])[:2] == ([0], [token])
    assert D.verify([-1, 0, 0, 0], [0, 1, 1, 2], [P] * 4, [Q] * 4, [0.5, 0.9, 0.9, 0.0])[:2] == ([0], [0])
    # an accepted sibling has it that the rows are not needed
    assert D.verify([-1, 0], [0, 1], [P, P], [Q, Q], [0.5, 0.1])[:2] == ([0, 1], [1, 0])


def test_without_the_drafts_probabilities():
    """All of the target's tokens tried and rejected, by less than is missing to 1."""
    p = np.array([[0.5, 0.25, 0.0, 0.0]] * 3)
    assert D.verify([-1, 0, 0], [0, 0, 1], p, None, [0.1, 0.6, 0.7])[:2] == ([0], [0])
    assert D.verify([-1, 0, 0], [0, 0, 1], p, None, [0.7, 0.6, 0.7])[:2] == ([0], [1])


def test_the_distribution_is_the_targets_to_what_rounding_moves():
    """A child drawn from q, by enumeration over draws, u and the last draw's u: p within the rows'
    rounding (half a step of bf16 is 2^-8 of each probability)."""
    n = 512
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(4)
    for x in range(4):
        taken = np.mean([len(D.verify([-1, 0], [0, x], [P, P], [Q, Q], [0.5, u])[0]) > 1 for u in grid])
        got[x] += Q[x] * taken
        if taken < 1:  # what is left does not depend on which u it was that rejected
            for u0 in grid:
                token = D.verify([-1, 0], [0, x], [P, P], [Q, Q], [u0, grid[-1]])[1][0]
                assert token >= 0
                got[token] += Q[x] * (1 - taken) / n
    assert np.abs(got / Q.sum() - P / P.sum()).max() < 2.0 ** -8


@pytest.mark.parametrize("draft", [[1.0, 1.0, 0.0, 0.0], [2.0, 0.0, 0.5, 0.0]])
def test_a_draft_that_is_no_distribution(draft):
    """Its sum is twice the target's or more: nothing is left, and no token."""
    p = np.array([[1.0, 0.0, 0.0, 0.0]] * 2)
    assert D.verify([-1, 0], [0, 2], p, [draft] * 2, [0.3, 0.9])[:2] == ([0], [-1])


def test_a_target_of_zeros_has_no_token():
    z = np.zeros((2, 4))
    for draft in (None, [Q, Q], z):
        assert D.verify([-1, 0], [0, 1], z, draft, [0.3, 0.0])[:2] == ([0], [-1])
