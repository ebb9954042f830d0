"""ds4x_paged_tree_attn at its edges: nodes that share a unit with others."""

import numpy as np
import pytest

from oracle import codecs as C
from oracle import drafts as D
from paged_path import Pool, check_token
from test_gpu_tree_attn import SCALE, queries, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 3, 5, 9, 12, 20, 30])
@pytest.mark.parametrize("row0", [3, 150])
def test_nodes_past_the_largest_draft_beside_the_last_of_it(heads, row0):
    """1024 is no multiple of the nodes that share a unit for 3, 5, 9, 12 and 20
    heads: those behind it are zeros all the same, those before are as ever."""
    rng = np.random.default_rng(140 + heads)
    n = 1045
    big = D.tree(rng, n, "random")
    pool = Pool([row0 + n], 64, 141)
    q, qv = queries(n, heads, 142)
    got, lse = run(pool, [big], [row0], q, status=-7)
    out = C.bf16_decode(got).astype(np.float64)
    assert np.all(out[1024:] == 0) and np.all(np.isneginf(lse[1024:]))
    for j in [0, 1, 500] + list(range(1000, 1024)):
        check_token(out[j], lse[j].astype(np.float64), pool.values(0, D.sees(big, j, row0)), qv[j], SCALE)
