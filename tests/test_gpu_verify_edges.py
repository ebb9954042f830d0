"""ds4x_verify_drafts at its edges: what is flagged, whatever the random numbers are."""

import numpy as np
import pytest

from oracle import drafts as D
from test_gpu_verify import expect, probabilities, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("bad", [-1, 100, 1 << 30, -(1 << 31)])
def test_a_bad_token_on_a_node_that_is_never_tried_is_flagged(sampled, bad):
    """Behind an accepted sibling, and on a root that the walk does not reach;
    node 0's is not looked at."""
    rng = np.random.default_rng(130)
    target = probabilities(rng, 7, 100)
    draft = probabilities(rng, 7, 100) if sampled else None
    trees = [[-1, 0, 0, 1], [-1, -1, 1]]
    u = np.array([0.4, 0.0, 0.0, 0.0, 0.3, 0.5, 0.5], dtype=np.float32)
    good = np.array([5, 7, 8, 9, 3, 2, 1], dtype=np.int32)
    want = expect(trees, good, target, draft, u)
    assert want[0][:4] == [0, 1, 3, -1]
    for node in range(7):
        tokens = good.copy()
        tokens[node] = bad
        if node in (1, 3):  # (the walk comes to these)
            assert run(trees, tokens, target, draft, u, status=-7) == expect(trees, tokens, target, draft, u)
        else:
            assert run(trees, tokens, target, draft, u, status=0 if node in (0, 4) else -7) == want
