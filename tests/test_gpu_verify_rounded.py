"""ds4x_verify_drafts where rounded probabilities leave nothing after a
rejection: the last token is drawn from the target's row, and nothing is flagged."""

import numpy as np
import pytest

from gpu_path import require_gpu
from oracle import drafts as D
from test_gpu_verify import expect, probabilities, run, to_bf16, widen

pytestmark = pytest.mark.gpu


def sure(rng, n, vocab, top, tail):
    """Rows that give one token `top` and up to `tail` others the rest, in bf16."""
    p = np.zeros((n, vocab))
    p[:, 1] = top
    at = 2 + np.arange(tail) * ((vocab - 2) // tail)
    w = rng.random((n, tail))
    p[:, at] = (1 - top) * w / w.sum(axis=1, keepdims=True)
    return widen(to_bf16(p.astype(np.float32)))


def nothing_left(trees, tokens, target, draft, u):
    """How many walks end where nothing is left and the target's row is drawn from."""
    count, at = 0, 0
    for parent in trees:
        s = slice(at, at + len(parent))
        path = D.verify(parent, tokens[s], target[s], None if draft is None else draft[s], u[s])[0]
        cur, kids = path[-1], [j for j in range(len(parent)) if parent[j] == path[-1]]
        if kids:
            p, mass = target[s][cur].astype(np.float64), 1.0
            for j in kids:
                if draft is None:
                    p[tokens[s][j]] = 0
                else:
                    p = np.maximum(p - mass * draft[s][cur], 0.0)
                    mass = p.sum()
            count += not p.any()
        at += len(parent)
    return count


@pytest.mark.parametrize("vocab", [30, 1000, 20011, 131072])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", ["star", "chain"])
def test_a_sure_target_and_a_sure_draft(vocab, dtype, shape):
    """The draft a little less sure, its tail sampled: where both round to 1 and
    the draft is larger elsewhere the rest of p is zero everywhere."""
    require_gpu()
    rng = np.random.default_rng(120 + vocab)
    trees = [D.tree(rng, 4, shape) for _ in range(48)]
    n = 4 * 48
    target, draft = sure(rng, n, vocab, 0.9999, 9), sure(rng, n, vocab, 0.9995, 9)
    tokens = (2 + rng.integers(0, 9, n) * ((vocab - 2) // 9)).astype(np.int32)
    u = rng.random(n).astype(np.float32)
    u[::8] = 0.9999  # (some last draws from the tail)
    args = (trees, tokens, target, draft, u)
    want = expect(*args)
    assert nothing_left(*args) >= 4
    assert min(want[1][::4]) >= 0
    assert run(*args, dtype=dtype) == want


@pytest.mark.parametrize("vocab", [30, 20011])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_the_drafts_probabilities(vocab, dtype):
    """A target cut to its likeliest tokens and rounded below 1, all of them tried."""
    require_gpu()
    rng = np.random.default_rng(121 + vocab)
    trees = [D.tree(rng, 4, "star") for _ in range(40)]
    n = 4 * 40
    target = np.zeros((n, vocab))
    target[:, [2, 9, 17]] = [0.5, 0.25, 0.125]
    target = target.astype(np.float32)
    tokens = np.tile(np.array([0, 9, 2, 17], dtype=np.int32), 40)
    u = rng.random(n).astype(np.float32)
    u[rng.random(n) < 0.7] = 0.97
    args = (trees, tokens, target, None, u)
    want = expect(*args)
    rejected = [s for s in range(40) if want[2][s] == 1]
    assert len(rejected) >= 4 and nothing_left(*args) >= 4
    assert run(*args, dtype=dtype) == want


def test_neighbours_of_a_row_that_is_none():
    """A target of zeros, a draft that sums to three times the target's: no token, flagged;
    the sequences beside them as ever."""
    require_gpu()
    rng = np.random.default_rng(122)
    vocab = 3000
    trees = [D.tree(rng, 3, "star") for _ in range(4)]
    target, draft = (sure(rng, 12, vocab, t, 5) for t in (0.9999, 0.9995))
    tokens = np.full(12, 2, dtype=np.int32)
    u = np.full(12, 0.99, dtype=np.float32)
    target[3:6] = 0.0
    draft[6:9] = 3 * target[6:9]
    args = (trees, tokens, target, draft, u)
    want = expect(*args)
    assert [want[1][s] for s in (0, 3, 6, 9)].count(-1) == 2
    assert run(*args, status=-7) == want


def test_exact_rows_are_as_before():
    """Rows in f32 whose difference is not zero go on to be drawn from it."""
    require_gpu()
    rng = np.random.default_rng(123)
    trees = [D.tree(rng, 5, "star") for _ in range(20)]
    target, draft = probabilities(rng, 100, 4001), probabilities(rng, 100, 4001)
    tokens = rng.integers(0, 4001, 100).astype(np.int32)
    u = rng.random(100).astype(np.float32)
    args = (trees, tokens, target, draft, u)
    assert nothing_left(*args) == 0 and run(*args) == expect(*args)
