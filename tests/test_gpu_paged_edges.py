"""Calls of the paged attentions whose result must not depend on what lies beside
them: another unit's queries, another session's or token's rows, what an earlier
kernel left on the chip, entries that are no row's."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, bf16_host_bits, dev, new_ws, require_gpu
from oracle import codecs as C
from oracle import paged as O
from paged_path import Pool, bf16, check_token
from test_gpu_paged_attn import SCALE, check, queries, run

pytestmark = pytest.mark.gpu


def same_bits(a, b):
    return torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def appended(x, page_rows):
    """Device rows x f32 [seqs, rows, 512] as `seqs` sequences of a pool, page after page: (pages, table)."""
    B = require_gpu()
    S, n, _ = x.shape
    per = -(-n // page_rows)
    pages = torch.zeros((S * per, page_rows * O.ROW_BYTES), dtype=torch.uint8, device="cuda")
    table = torch.arange(S * per, dtype=torch.int32, device="cuda").view(S, per)
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * n
    ws = new_ws(256)
    B.ds4x_paged_append(pages, page_rows, table, cu, torch.zeros(S, dtype=torch.int64, device="cuda"), x.reshape(S * n, 512), ws)
    assert B.ds4x_workspace_status(ws) == 0
    return pages, table


def attend(pages, page_rows, table, cu, end, q, ws, begin=None, scale=SCALE, status=0):
    B = require_gpu()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], device="cuda")
    B.ds4x_paged_attn(pages, page_rows, table, cu, end, q, scale, out, lse, ws, row_begin=begin)
    assert B.ds4x_workspace_status(ws) == status
    return out, lse


def test_what_an_earlier_call_left_does_not_show():
    """A call of 64 heads over bytes that were never rows (NaN in every product), then
    calls of few heads whose lists begin with tiles without a row and whose logits are
    far below zero."""
    rng = np.random.default_rng(15)
    n, T = 500, 400
    d = rng.standard_normal(512)
    d /= np.linalg.norm(d)
    x = (4.0 * d + 0.2 * rng.standard_normal((n, 512))).astype(np.float32)
    pool = Pool([n], 32, 16, x=[x], extra_pages=3)
    free = [p for p in range(pool.n_pages) if p not in pool.table[0, :16]]
    idx = np.full((T, 300), -1, dtype=np.int32)
    idx[:, 150:] = rng.integers(0, n, (T, 150))
    for heads in (1, 16, 40):
        qb, qv = bf16(np.tile(d * -900.0 / 4.0 / SCALE, (T, heads, 1)))
        old = pool.table.copy()
        pool.table[0, :16] = free[0]
        run(pool, [T], queries(T, 64, 17)[0], end=[n] * T)
        pool.table = old
        got, lse = run(pool, [T], qb, idx=idx, n_rows=[n])
        out = C.bf16_decode(got).astype(np.float64)
        for t in (0, 1, 2, 3, 77, 78, T - 1):
            check_token(out[t], lse[t].astype(np.float64), pool.values(0, idx[t, 150:]), qv[t], SCALE)
