"""Host checks of the paged attentions at their edges.  Each call here is refused at
the last for its workspace, so none reaches a GPU."""

import pytest

from test_paged_host import ATTN, FAKE, SPARSE, call, lib  # noqa: F401

VEC = 2 * 64 * 512  # bytes of a token's queries


@pytest.mark.parametrize("fn, args", [("ds4x_paged_attn", ATTN), ("ds4x_paged_sparse_attn", SPARSE)])
@pytest.mark.parametrize("gap, q_stride, out_stride, n, ok", [
    (VEC, 2, 2, 3, True),             # a token's queries, then its outputs
    (-VEC, 2, 2, 3, True),            # the other way round
    (5 * VEC, 2, 2, 3, True),         # some tokens on
    (-3 * VEC, 2, 2, 3, True),
    (VEC, 3, 3, 5, True),
    (2 * VEC, 3, 3, 5, True),
    (3 * VEC, 3, 3, 5, False),        # the next token's queries
    (VEC - 16, 2, 2, 3, False),       # 16 bytes of its own queries
    (VEC + 16, 2, 2, 3, False),       # 16 bytes of the next one's
    (-VEC - 16, 2, 2, 3, False),
    (VEC, 2, 3, 3, False),            # of different strides: only apart
    (6 * VEC, 2, 3, 3, True),
    (VEC, 1, 1, 1, True),
    (VEC - 16, 1, 1, 1, False),
    (0, 1, 1, 3, False),
])
def test_queries_and_outputs_may_interleave_but_not_overlap(lib, fn, args, gap, q_stride, out_stride, n, ok):  # noqa: F811
    base = FAKE << 12
    a = dict(args, n=n, q=base, q_stride=q_stride * 64 * 512, out=base + gap, out_stride=out_stride * 64 * 512, nws=0)
    assert call(lib, fn, a) == (-3 if ok else -1)
