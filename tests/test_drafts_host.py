"""The host checks of the calls on drafted tokens: a bad call is refused before
any CUDA call, so these run without a GPU."""

import os

import pytest

from test_paged_host import BAD_CACHE, BAD_QO, BAD_ROWS, CACHE, FAKE, FAR


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_sparse_csa_gb300 import build as B

    if not os.path.exists(B.LIB_PATH):
        B.build()
    from compressed_kv_sparse_csa_gb300 import binding

    return binding.lib()


TREE = dict(CACHE, row0=FAKE, parent=FAKE, begin=None, n=3, heads=64, q=FAKE, q_stride=64 * 512, scale=0.04, out=FAR,
            out_stride=64 * 512, lse=FAKE, ws=FAKE, nws=None)
KEEP = dict(CACHE, row0=FAKE, path=FAKE, n_path=FAKE, n=3, ws=FAKE, nws=256)
P, T, N = FAR, FAR + 0x1000, FAR + 0x2000  # outputs
VERIFY = dict(cu=FAKE, n_seqs=2, n=3, parent=FAKE, tokens=FAKE, target=FAKE, target_stride=1000, draft=FAKE,
              draft_stride=1000, type=0, vocab=1000, u=FAKE, path=P, out=T, n_path=N, ws=FAKE, nws=256)
BAD_TREE = BAD_QO + [dict(row0=None), dict(row0=FAKE + 4), dict(parent=None), dict(parent=FAKE + 2), dict(begin=FAKE + 4)]
BAD_KEEP = BAD_ROWS + [dict(path=None), dict(path=FAKE + 2), dict(n_path=None), dict(n_path=FAKE + 1)]
BAD_VERIFY = [dict({k: None}) for k in ("cu", "parent", "tokens", "target", "u", "path", "out", "n_path", "ws")] + [
    dict({k: FAKE + 2}) for k in ("cu", "parent", "tokens", "u", "path", "out", "n_path")] + [
    dict(target=FAKE + 8), dict(draft=FAKE + 4), dict(ws=FAKE + 8), dict(n_seqs=0), dict(n_seqs=-1),
    dict(n_seqs=2 ** 31 - 1), dict(n=0), dict(n=1 << 31), dict(vocab=0), dict(vocab=(1 << 20) + 1, target_stride=1 << 21),
    dict(type=2), dict(type=-1), dict(target_stride=996), dict(target_stride=1002), dict(draft_stride=999),
    dict(type=1, target_stride=1004), dict(draft_stride=1 << 41),
    # outputs on one another and on inputs
    dict(out=P), dict(out=P + 8), dict(n_path=P + 8), dict(n_path=T), dict(path=FAKE), dict(out=FAKE + 8),
    dict(n_path=FAKE), dict(target=P - 2 * 4000), dict(draft=T - 16), dict(ws=N - 128)]


def call(lib, fn, args):
    if args["nws"] is None:
        args = dict(args, nws=lib.ds4x_paged_attn_workspace())
    return getattr(lib, fn)(*args.values(), None)


@pytest.mark.parametrize("fn, good, bad", [("ds4x_paged_tree_attn", TREE, BAD_CACHE + BAD_TREE),
                                           ("ds4x_paged_keep", KEEP, BAD_CACHE + BAD_KEEP),
                                           ("ds4x_verify_drafts", VERIFY, BAD_VERIFY)])
def test_refusals(lib, fn, good, bad):
    for b in bad:
        assert call(lib, fn, dict(good, **b)) == -1, b
    nws = lib.ds4x_paged_attn_workspace() if good["nws"] is None else good["nws"]
    assert call(lib, fn, dict(good, nws=nws - 1)) == -3


def test_binding_refuses_what_it_can_see():
    """CPU tensors: ValueError before the library is called."""
    import torch

    from compressed_kv_sparse_csa_gb300 import binding as B

    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        B.ds4x_verify_drafts(i, i, i, torch.zeros((2, 8)), None, torch.zeros(2), i, i, i[:1], torch.zeros(256, dtype=torch.uint8))
    t = torch.zeros(64 * 368, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.ds4x_paged_keep(t, 64, torch.zeros((1, 1), dtype=torch.int32), i, torch.zeros(1, dtype=torch.int64), i, i[:1], t)
