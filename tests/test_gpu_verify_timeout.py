"""Verification's bounded wait: when a sum of its blocks never comes, every block
gives up after its time limit (0.5 s of the GPU's global timer), all its warps
alike, writes nothing and leaves with its cluster; the workspace status word reads
DS4X_ETIMEOUT and the context stays usable.  The wait is made to run out without
any fault: the workspace header's extra-arrivals word is set, so the barriers wait
for more bytes than the blocks give."""

import time

import numpy as np
import pytest
import torch

from gpu_path import dev, new_ws, require_gpu
from oracle import drafts as D
from test_gpu_verify import drafted, expect, probabilities, run

pytestmark = pytest.mark.gpu
ETIMEOUT = -6


@pytest.mark.parametrize("trees_of, vocab, sampled", [([1], 100, False), ([6], 50000, True), ([9, 6, 4], 131072, True),
                                                      ([6, 1, 0, 7], 20000, False)])
def test_wait_runs_out_and_recovers(trees_of, vocab, sampled):
    """One block a sequence and clusters of up to 16; walks that end at once and
    walks that would make several passes."""
    B = require_gpu()
    rng = np.random.default_rng(110 + vocab)
    trees = [D.tree(rng, n, "star") if n else [] for n in trees_of]
    n, S = sum(trees_of), len(trees)
    target = probabilities(rng, n, vocab)
    draft = ((target + probabilities(rng, n, vocab)) / 2).astype(np.float32) if sampled else None
    tokens = drafted(rng, trees, target, draft, not sampled)
    u = np.full(n, 1 - 2.0 ** -24, dtype=np.float32)
    u[0] = 0.4
    wide = -(-vocab // 8) * 8
    rows = lambda p: None if p is None else dev(np.pad(p, ((0, 0), (0, wide - vocab))))[:, :vocab]  # noqa: E731
    cu = dev(np.concatenate([[0], np.cumsum(trees_of)]).astype(np.int32))
    parent = dev(np.array([p for t in trees for p in t], dtype=np.int32))
    path, out, count = (torch.full((k,), 99, dtype=torch.int32, device="cuda") for k in (n, n, S))
    ws = new_ws(256)
    ws[12:16].view(torch.int32).fill_(1)  # a sum that never comes
    args = (cu, parent, dev(tokens), rows(target), rows(draft), dev(u), path, out, count, ws)
    torch.cuda.synchronize()
    t0 = time.time()
    B.ds4x_verify_drafts(*args)
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    assert B.ds4x_workspace_status(ws) == ETIMEOUT
    assert 0.3 < elapsed < 30.0, elapsed
    assert torch.all(path == 99) and torch.all(out == 99)  # a block that gave up writes nothing
    # the context is still usable and a fresh workspace gives the exact result
    assert run(trees, tokens, target, draft, u) == expect(trees, tokens, target, draft, u)
