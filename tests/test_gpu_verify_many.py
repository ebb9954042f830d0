"""ds4x_verify_drafts with many sequences and real vocabularies: the form with
more blocks an SM, clusters that swap their sums, several chunks a warp, tried
tokens anywhere in a chunk; against the float64 walk, whole."""

import numpy as np
import pytest

from oracle import drafts as D
from test_gpu_verify import expect, probabilities, run, to_bf16, widen

pytestmark = pytest.mark.gpu

# sequences, tokens: by the rule of csrc/verify.cu 8, 4, 2, 1 and 1 blocks a sequence on 152 SMs
SIZES = [(61, 50257), (120, 20011), (256, 20011), (400, 3000), (400, 20011)]


def siblings(rng, seqs):
    """Stars of 3 to 6 nodes, some nodes with children of their own."""
    return [[-1] + [0] * int(rng.integers(2, 5)) + [1] * int(rng.integers(0, 2)) for _ in range(seqs)]


def u_of(rng, n):
    """Half of them such that most drafts are rejected."""
    u = rng.random(n).astype(np.float32)
    high = rng.random(n) < 0.5
    u[high] = (1 - rng.random(int(high.sum())) / 64).astype(np.float32)
    return np.minimum(u, np.float32(1 - 2.0 ** -24))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, vocab", SIZES)
def test_sampled_siblings(seqs, vocab, dtype):
    rng = np.random.default_rng(190 + seqs + vocab)
    trees = siblings(rng, seqs)
    n = sum(map(len, trees))
    target = probabilities(rng, n, vocab)
    draft = target * rng.random((n, vocab), dtype=np.float32) + 0.3 * probabilities(rng, n, vocab)
    draft /= draft.sum(axis=1, keepdims=True)
    if dtype == "bf16":
        target, draft = widen(to_bf16(target)), widen(to_bf16(draft))
    tokens, at = [], 0
    for parent in trees:
        for p in parent:
            c = np.cumsum(draft[at + max(p, 0)], dtype=np.float64)
            tokens.append(int(min(np.searchsorted(c, rng.random() * c[-1], side="right"), vocab - 1)))
        at += len(parent)
    args = (trees, np.array(tokens, dtype=np.int32), target, draft, u_of(rng, n))
    want = expect(*args)
    assert want[2].count(1) > seqs // 16 and sum(c > 1 for c in want[2]) > seqs // 16
    assert run(*args, dtype=dtype) == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, vocab", SIZES)
def test_chosen_siblings(seqs, vocab, dtype):
    """Likely tokens, all in one chunk of 1024 or spread over the vocabulary, in
    every part of a chunk, rejected and left out of the last draw."""
    rng = np.random.default_rng(191 + seqs + vocab)
    trees = siblings(rng, seqs)
    n = sum(map(len, trees))
    target = probabilities(rng, n, vocab, peak=0.5)
    tokens, at = np.zeros(n, dtype=np.int32), 0
    for s, parent in enumerate(trees):
        base = 1024 * int(rng.integers(0, (vocab - 1) // 1024 + 1)) if s % 2 else 0
        room = min(1024, vocab - base) if s % 2 else vocab
        tokens[at:at + len(parent)] = base + rng.choice(room, len(parent), replace=False)
        for j, p in enumerate(parent):  # an eighth each
            target[at + max(p, 0), tokens[at + j]] = 0.125 if p >= 0 else 0.0
        at += len(parent)
    rest = 1 - 0.125 * np.array([sum(p == j for p in t) for t in trees for j in range(len(t))])
    drafted = np.zeros_like(target, dtype=bool)
    drafted[target == 0.125] = True
    others = np.where(drafted, 0, target)
    target = np.where(drafted, target, others / others.sum(axis=1, keepdims=True) * rest[:, None]).astype(np.float32)
    if dtype == "bf16":
        target = widen(to_bf16(target))
    u = rng.random(n).astype(np.float32)
    args = (trees, tokens, target, None, u)
    want = expect(*args)
    assert want[2].count(1) > seqs // 16 and sum(c > 1 for c in want[2]) > seqs // 16
    assert run(*args, dtype=dtype) == want
