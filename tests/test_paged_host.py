"""The paged calls' host checks: a bad call is refused before any CUDA call,
so these run without a GPU."""

import ctypes
import os

import pytest

FAKE, FAR = 0x10000, 0x7F0000000000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_sparse_csa_gb300 import build as B

    if not os.path.exists(B.LIB_PATH):
        B.build()
    from compressed_kv_sparse_csa_gb300 import binding

    return binding.lib()


CACHE = dict(pages=FAKE, n_pages=10, page_rows=64, table=FAKE, n_seqs=2, seq_pages=4, table_stride=4, cu=FAKE)
APPEND = dict(CACHE, row0=FAKE, kv_in=FAKE, in_type=0, in_stride=512, n=3, pos=FAKE, freq=FAKE, style=0, ws=FAKE, nws=256)
GATHER = dict(CACHE, row0=FAKE, out=FAKE, out_type=1, out_stride=512, n=3, ws=FAKE, nws=256)
ATTN = dict(CACHE, begin=None, end=FAKE, n=3, heads=64, q=FAKE, q_stride=64 * 512, scale=0.04, out=FAR,
            out_stride=64 * 512, lse=FAKE, ws=FAKE, nws=None)
SPARSE = dict(CACHE, n_rows=FAKE, idx=FAKE, k=512, n=3, heads=64, q=FAKE, q_stride=64 * 512, scale=0.04, out=FAR,
              out_stride=64 * 512, lse=FAKE, ws=FAKE, nws=None)

BAD_CACHE = [dict(pages=None), dict(pages=FAKE + 8), dict(n_pages=0), dict(n_pages=1 << 31), dict(page_rows=0),
             dict(page_rows=8), dict(page_rows=48), dict(page_rows=512), dict(page_rows=-64), dict(table=None),
             dict(table=FAKE + 2), dict(n_seqs=0), dict(n_seqs=2 ** 31 - 1), dict(seq_pages=0), dict(table_stride=3),
             dict(seq_pages=1 << 26, table_stride=1 << 26), dict(cu=None), dict(cu=FAKE + 1), dict(ws=None),
             dict(ws=FAKE + 8)]
BAD_ROWS = [dict(row0=None), dict(row0=FAKE + 4), dict(n=0), dict(n=-1), dict(n=1 << 31)]
BAD_APPEND = BAD_ROWS + [dict(kv_in=None), dict(kv_in=FAKE + 4), dict(in_type=2), dict(in_type=-1), dict(in_stride=511),
                         dict(in_stride=514), dict(in_type=1, in_stride=516), dict(pos=FAKE + 4), dict(freq=FAKE + 2),
                         dict(style=2)]
BAD_GATHER = BAD_ROWS + [dict(out=None), dict(out=FAKE + 8), dict(out_type=2), dict(out_stride=508),
                         dict(out_stride=516)]
BAD_QO = [dict(n=0), dict(n=65536), dict(heads=0), dict(heads=129, q_stride=129 * 512, out_stride=129 * 512),
          dict(q=None), dict(q=FAKE + 2), dict(q_stride=64 * 512 - 8), dict(q_stride=64 * 512 + 4), dict(out=None),
          dict(out=FAR + 8), dict(out_stride=100), dict(lse=FAKE + 2), dict(out=FAKE), dict(out=FAKE + 2 * 64 * 512 * 3 - 16)]
BAD_ATTN = BAD_QO + [dict(end=None), dict(end=FAKE + 4), dict(begin=FAKE + 4)]
BAD_SPARSE = BAD_QO + [dict(n_rows=None), dict(n_rows=FAKE + 4), dict(idx=None), dict(idx=FAKE + 2), dict(k=0),
                       dict(k=8193)]


def call(lib, fn, args):
    if args["nws"] is None:
        args = dict(args, nws=lib.ds4x_paged_attn_workspace())
    return getattr(lib, fn)(*args.values(), None)


@pytest.mark.parametrize("fn, good, bad", [("ds4x_paged_append", APPEND, BAD_CACHE + BAD_APPEND),
                                           ("ds4x_paged_gather", GATHER, BAD_CACHE + BAD_GATHER),
                                           ("ds4x_paged_attn", ATTN, BAD_CACHE + BAD_ATTN),
                                           ("ds4x_paged_sparse_attn", SPARSE, BAD_CACHE + BAD_SPARSE)])
def test_refusals(lib, fn, good, bad):
    for b in bad:
        assert call(lib, fn, dict(good, **b)) == -1, b
    nws = 256 if "stride" in fn or fn in ("ds4x_paged_append", "ds4x_paged_gather") else lib.ds4x_paged_attn_workspace()
    assert call(lib, fn, dict(good, nws=nws - 1)) == -3


def test_workspace_size(lib):
    assert 256 <= lib.ds4x_paged_attn_workspace() <= 48 << 20


def test_header_constants_match_the_oracle():
    import re

    from conftest import ROOT
    from oracle import paged as O

    text = open(os.path.join(ROOT, "include", "ds4x.h")).read()
    assert int(re.search(r"DS4X_PAGED_ROW_BYTES = (\d+)", text).group(1)) == O.ROW_BYTES == 224 + 128 + 16
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_binding_refuses_what_it_can_see():
    """CPU tensors, shapes and types: ValueError before the library is called."""
    import torch

    from compressed_kv_sparse_csa_gb300 import binding as B

    t = torch.zeros(64 * 368, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.ds4x_paged_gather(t, 64, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                            torch.zeros(1, dtype=torch.int64), torch.zeros((1, 512)), t)
