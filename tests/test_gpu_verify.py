"""ds4x_verify_drafts against the float64 walk of the oracle: the same nodes and
tokens, whole.

The kernel's comparisons are good to 2^-40 of what is compared (pairs of floats
throughout, about 2^-44 a sum).  The oracle says how near each walk's decisions came to their borders;
inputs are seeded, and every compared walk keeps 2^-36 from its borders (which
a sum's rounding cannot cross), save those of exact powers of two, whose sums
are exact on both sides."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, dev, new_ws, require_gpu
from oracle import drafts as D

pytestmark = pytest.mark.gpu
FAR = 2.0 ** -36


def probabilities(rng, n, vocab, peak=2.0, zeros=0.0):
    p = rng.random((n, vocab)) ** -peak
    p[rng.random((n, vocab)) < zeros] = 0.0
    p[:, rng.integers(vocab)] += 1e-3
    return (p / p.sum(axis=1, keepdims=True)).astype(np.float32)


def to_bf16(p):
    u = p.view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def widen(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def drafted(rng, trees, target, draft, likely):
    """Tokens: draws from the parent's draft, or its likeliest ones."""
    tokens, at = [], 0
    for parent in trees:
        for j, p in enumerate(parent):
            row = (draft if draft is not None else target)[at + max(p, 0)].astype(np.float64)
            if likely:
                tokens.append(int(np.argsort(-row, kind="stable")[min(parent[:j].count(p), len(row) - 1)]))
            else:
                tokens.append(int(rng.choice(len(row), p=row / row.sum())))
        at += len(parent)
    return np.array(tokens, dtype=np.int32)


def run(trees, tokens, target, draft, u, dtype="f32", pad=0, stream=None, extra=0, status=0, wide=0):
    """Rows padded by `pad` elements of NaN, `extra` padding tokens, integer
    arrays beginning `wide` elements into their storage."""
    B = require_gpu()
    n, V = target.shape
    S = len(trees)

    def rows(p):
        if p is None:
            return None
        t = bf16_dev(to_bf16(p)) if dtype == "bf16" else dev(p)
        w = torch.full((n + extra, -(-V // 8) * 8 + pad), float("nan"), dtype=t.dtype, device="cuda")
        w[:n, :V] = t
        return w[:, :V]

    def ints(v, count, fill):
        t = torch.full((count + wide,), fill, dtype=torch.int32, device="cuda")[wide:]
        t[:len(v)] = torch.tensor(np.asarray(v, dtype=np.int32))
        return t

    cu = ints(np.concatenate([[0], np.cumsum([len(t) for t in trees])]), S + 1, 0)
    parent, tok = ints([p for t in trees for p in t], n + extra, 77), ints(tokens, n + extra, -5)
    un = torch.zeros(n + extra + wide, device="cuda")[wide:]
    un[:n] = torch.tensor(np.asarray(u, dtype=np.float32))
    path, out, count = ints([], n + extra, 99), ints([], n + extra, 99), ints([], S, 99)
    ws = new_ws(256)
    torch.cuda.synchronize()
    B.ds4x_verify_drafts(cu, parent, tok, rows(target), rows(draft), un, path, out, count, ws, stream=stream)
    torch.cuda.synchronize()
    assert B.ds4x_workspace_status(ws) == status
    assert torch.all(path[n:] == 99) and torch.all(out[n:] == 99)
    return path[:n].tolist(), out[:n].tolist(), count.tolist()


def expect(trees, tokens, target, draft, u, far=FAR):
    path, out, count, at = [], [], [], 0
    for parent in trees:
        n = len(parent)
        if n == 0:
            count.append(0)
            continue
        s = slice(at, at + n)
        p, o, near = D.verify(parent, tokens[s], target[s], None if draft is None else draft[s], u[s])
        assert near > far, f"a decision lies {near} from its border"
        path += p + [-1] * (n - len(p))
        out += o + [-1] * (n - len(o))
        count.append(len(p))
        at += n
    return path, out, count


@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 128, 1000, 1023, 1025, 4097, 50257, 131072])
@pytest.mark.parametrize("dtype, sampled, shape", [("f32", True, "chain"), ("f32", True, "level"), ("f32", False, "level"),
                                                   ("bf16", True, "random"), ("bf16", False, "star")])
def test_walks(vocab, dtype, sampled, shape):
    rng = np.random.default_rng(vocab * 10 + len(shape))
    nodes = [1, 6, 13, 0, 9, 2, 24] if vocab < 40000 else [6, 1, 9]
    trees = [D.tree(rng, n, shape) if n else [] for n in nodes]
    n = sum(nodes)
    target, draft = probabilities(rng, n, vocab), None
    if sampled:
        mixed = target * rng.random((n, vocab)).astype(np.float32) + 0.3 * probabilities(rng, n, vocab)
        draft = (mixed / mixed.sum(axis=1, keepdims=True)).astype(np.float32)
    if dtype == "bf16":
        target, draft = widen(to_bf16(target)), None if draft is None else widen(to_bf16(draft))
    tokens = drafted(rng, trees, target, draft, not sampled)
    u = rng.random(n).astype(np.float32)
    args = (trees, tokens, target, draft, u)
    want = expect(*args)
    assert run(*args, dtype=dtype) == want
    assert run(*args, dtype=dtype, pad=16, extra=5, wide=1) == want


@pytest.mark.parametrize("sampled", [True, False])
def test_many_siblings_and_zeros(sampled):
    """Probabilities that are mostly zero, as a top-p sampler leaves them; many
    children a node, the same token among them several times; long chains of
    rejections."""
    rng = np.random.default_rng(80)
    trees = [D.tree(rng, n, s) for n, s in [(40, "star"), (33, "level"), (60, "random"), (12, "chain"), (5, "forest")]]
    n, V = sum(map(len, trees)), 3000
    target, draft = probabilities(rng, n, V, zeros=0.97), probabilities(rng, n, V, zeros=0.9)
    both = 0.2 * target + 0.8 * draft
    draft = (both / both.sum(axis=1, keepdims=True)).astype(np.float32)
    tokens = drafted(rng, trees, target, draft, False)
    tokens[10:14] = tokens[9]
    u = rng.random(n).astype(np.float32)
    args = (trees, tokens, target, draft if sampled else None, u)
    assert run(*args) == expect(*args)


def test_borders_of_equal_probabilities():
    """Powers of two: every sum is exact, so u on a border is decided by the
    definition (the sum must pass u; acceptance needs u q C < w)."""
    V = 1024
    target = np.full((3, V), 2.0 ** -10, dtype=np.float32)
    for u0 in (0.0, 2.0 ** -10, 0.5, 511 / 1024, 512 / 1024, 1023 / 1024, 1 - 2.0 ** -24):
        for dtype in ("f32", "bf16"):
            _, out, _ = run([[-1]], np.zeros(1, np.int32), target[:1], None, np.array([u0]), dtype=dtype)
            assert out == [int(u0 * 1024)]
    # u q C = w is not accepted, one step below is; the rest's tokens leave out the tried one
    draft = np.full((3, V), 2.0 ** -9, dtype=np.float32)
    draft[:, V // 2:] = 0
    tok = np.array([0, 3, 0], dtype=np.int32)
    for u1, took in ((0.5, False), (np.nextafter(np.float32(0.5), np.float32(0)), True)):
        path, out, count = run([[-1, 0, -1]], tok, target, draft, np.array([0.25, u1, 0]))
        # what is left of 2^-10 each when 2^-9 is taken off the lower half: the upper half
        assert (path, out, count) == (([0, 1, -1], [3, 256, -1], [2]) if took else ([0, -1, -1], [V // 2 + 128, -1, -1], [1]))
    for u1, took in ((2.0 ** -10, False), (np.nextafter(np.float32(2.0 ** -10), np.float32(0)), True)):
        path, out, count = run([[-1, 0, -1]], tok, target, None, np.array([3.5 / 1023, u1, 0]))
        assert out[:count[0]] == ([3, 3] if took else [4])


def test_what_is_left_when_the_draft_is_the_target():
    """p = q: the first child is accepted whatever u is; siblings behind a
    rejection that cannot be are never looked at."""
    rng = np.random.default_rng(81)
    target = probabilities(rng, 8, 500)
    trees = [D.tree(rng, 8, "chain")]
    tokens = drafted(rng, trees, target, target, False)
    u = np.full(8, 1 - 2.0 ** -24, dtype=np.float32)
    path, out, count = run(trees, tokens, target, target, u)
    assert path == list(range(8)) and count == [8] and out[:7] == tokens[1:].tolist()


def test_nothing_left_is_minus_one_and_flagged():
    V = 300
    target = np.zeros((2, V), dtype=np.float32)
    path, out, count = run([[-1, 0]], np.array([0, 5], np.int32), target, None, np.array([0.3, 0.0]), status=-7)
    assert (path, out, count) == ([0, -1], [-1, -1], [1])
    target[0, 7] = 1.0  # all of it on a token that u rejects by a hair: no, u = 1 is none; the draft's is tried and gone
    draft = np.zeros((2, V), dtype=np.float32)
    draft[0, 7] = 1.0
    draft[0, 9] = 1.0
    path, out, count = run([[-1, 0]], np.array([0, 9], np.int32), target, draft, np.array([0.3, 0.0]), status=-7)
    assert (path, out, count) == ([0, -1], [-1, -1], [1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_negative_and_nan_count_as_zero(dtype):
    rng = np.random.default_rng(82)
    trees = [D.tree(rng, 9, "level"), D.tree(rng, 4, "chain")]
    target, draft = widen(to_bf16(probabilities(rng, 13, 2000))), widen(to_bf16(probabilities(rng, 13, 2000)))
    tokens = drafted(rng, trees, target, draft, False)
    for a in (target, draft):
        a[:, ::3] = np.nan
        a[:, 1::7] *= -1
    u = rng.random(13).astype(np.float32)
    for q in (draft, None):
        args = (trees, tokens, target, q, u)
        assert run(*args, dtype=dtype) == expect(*args)


def test_tokens_outside_the_vocabulary():
    rng = np.random.default_rng(83)
    target = probabilities(rng, 4, 100)
    for draft in (None, probabilities(rng, 4, 100)):
        tokens = np.array([-9, 100, -1, 1 << 30], dtype=np.int32)
        trees, u = [[-1, 0, 0, 0]], np.array([0.4, 0.0, 0.0, 0.0], dtype=np.float32)
        assert run(trees, tokens, target, draft, u, status=-7) == expect(trees, tokens, target, draft, u)


def test_parents_that_are_none():
    """Counted as roots: the walk does not reach them."""
    rng = np.random.default_rng(84)
    target = probabilities(rng, 6, 64)
    tokens = np.argmax(target[0]) * np.ones(6, dtype=np.int32)
    u = np.zeros(6, dtype=np.float32)
    got = run([[-1, 5, -3, 3, 1 << 20, 0]], tokens, target, None, u, status=-7)
    assert got == expect([[-1, -1, -1, -1, -1, 0]], tokens, target, None, u)
    assert got[0][:2] == [0, 5]


def test_largest_drafts():
    rng = np.random.default_rng(85)
    trees = [D.tree(rng, 1024, "chain"), D.tree(rng, 1024, "star"), D.tree(rng, 1024, "random")]
    n, V = 3 * 1024, 64
    target = probabilities(rng, n, V, peak=0.2)
    tokens = drafted(rng, trees, target, target, False)
    u = rng.random(n).astype(np.float32)
    u[:700] = 0.01
    want = expect(trees, tokens, target, target, u)
    assert run(trees, tokens, target, target, u) == want
    tokens2 = rng.integers(0, V, n).astype(np.int32)
    want = expect(trees, tokens2, target, None, u)
    assert run(trees, tokens2, target, None, u) == want
    # one node more: nothing for that sequence, its neighbour as ever
    trees = [D.tree(rng, 1025, "chain"), D.tree(rng, 5, "chain")]
    target = probabilities(rng, 1030, V, peak=0.2)
    u = rng.random(1030).astype(np.float32)
    tokens = rng.integers(0, V, 1030).astype(np.int32)
    path, out, count = run(trees, tokens, target, None, u, status=-7)
    one = expect(trees[1:], tokens[1025:], target[1025:], None, u[1025:])
    assert count == [0] + one[2] and path == [-1] * 1025 + one[0] and out == [-1] * 1025 + one[1]


def test_many_sequences():
    rng = np.random.default_rng(86)
    trees = [D.tree(rng, int(n), "level") if n else [] for n in rng.integers(0, 5, 2000)]
    n, V = sum(map(len, trees)), 333
    target, draft = probabilities(rng, n, V), probabilities(rng, n, V, zeros=0.3)
    draft = ((target + draft) / 2).astype(np.float32)
    tokens = drafted(rng, trees, target, draft, False)
    u = rng.random(n).astype(np.float32)
    args = (trees, tokens, target, draft, u)
    want = expect(*args)
    assert sum(c > 1 for c in want[2]) > 200  # many accept some
    assert run(*args) == want


def test_a_large_vocabulary_and_nearly_equal_rows():
    """2^20 tokens, flat, the draft near the target: what is left is small beside
    what it is the difference of."""
    rng = np.random.default_rng(87)
    V = 1 << 20
    trees = [[-1, 0, 0, 1]]
    target = probabilities(rng, 4, V, peak=0.3)
    draft = (target * (1 + 1e-4 * rng.standard_normal((4, V)))).astype(np.float32)
    draft /= draft.sum(axis=1, keepdims=True, dtype=np.float64).astype(np.float32)
    low = int(np.argmin(target[0] / draft[0]))
    tokens = np.array([0, low, low, 7], dtype=np.int32)
    for u0 in (0.1, 0.55, 0.93):
        u = np.array([u0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.5], dtype=np.float32)
        args = (trees, tokens, target, draft, u)
        want = expect(*args, far=2.0 ** -26)  # (what is left is 2^-14 of what it is the difference of)
        assert want[2] == [1] and run(*args) == want


def test_captured_on_another_stream_and_again():
    B = require_gpu()
    rng = np.random.default_rng(88)
    n, V = 12, 5003
    wide = -(-V // 8) * 8
    target, draft = (torch.zeros((n, wide), device="cuda")[:, :V] for _ in range(2))
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    parent, tokens, path, out = torch.zeros((4, n), dtype=torch.int32, device="cuda")
    u, count = torch.zeros(n, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = new_ws(256)
    call = lambda st=None: B.ds4x_verify_drafts(cu, parent, tokens, target, draft, u, path, out, count, ws, stream=st)  # noqa: E731
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    ws.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for nodes in ([4, 8, 0], [1, 1, 10], [12, 0, 0]):
        trees = [D.tree(rng, m, "level") if m else [] for m in nodes]
        t, d = probabilities(rng, n, V), probabilities(rng, n, V)
        d = ((t + d) / 2).astype(np.float32)
        tok, un = drafted(rng, trees, t, d, False), rng.random(n).astype(np.float32)
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)))
        parent.copy_(torch.tensor([p for tr in trees for p in tr], dtype=torch.int32))
        tokens.copy_(torch.tensor(tok))
        target.copy_(torch.tensor(t))
        draft.copy_(torch.tensor(d))
        u.copy_(torch.tensor(un))
        want = expect(trees, tok, t, d, un)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert (path.tolist(), out.tolist(), count.tolist()) == want
    assert B.ds4x_workspace_status(ws) == 0
