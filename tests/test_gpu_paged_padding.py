"""Padding tokens of the paged calls: whatever their entries hold, nothing of theirs
counts, nothing is flagged and their outputs stay."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, dev, new_ws, require_gpu
from paged_path import Pool
from test_gpu_paged_attn import SCALE, queries

pytestmark = pytest.mark.gpu
LOW, HIGH = -(1 << 63), (1 << 63) - 1
TOKENS, ROWS = [2, 0, 5], [40, 7, 900]
N, PAD = 7, 50


def mixed(real, fills):
    """int64 [N + PAD]: the real entries, then the fills in turn."""
    return dev(np.concatenate([np.asarray(real, dtype=np.int64), np.resize(np.array(fills, dtype=np.int64), PAD)]))


def setup(heads):
    pool = Pool(ROWS, 16, 50)
    cu = dev(np.concatenate([[0], np.cumsum(TOKENS)]).astype(np.int32))
    bits, _ = queries(N + PAD, heads, 51)
    bits[N:] = np.resize(np.array([0x7FC0, 0x7F80, 0xFF80, 0x7F7F], dtype=np.uint16), bits[N:].shape)
    return pool, dev(pool.pages), dev(pool.table), cu, bf16_dev(bits)


@pytest.mark.parametrize("heads", [64, 8, 100])
@pytest.mark.parametrize("sparse", [False, True])
def test_attention(heads, sparse):
    B = require_gpu()
    _, pages, table, cu, q = setup(heads)
    n_rows = dev(np.array(ROWS, dtype=np.int64))
    end = [39, 40, 896, 897, 898, 899, 900]
    idx = np.random.default_rng(52).integers(0, 40, (N + PAD, 90)).astype(np.int32)
    idx[N:] = np.resize(np.array([-1, -2, 1 << 30, (1 << 31) - 1, -(1 << 31), 3], dtype=np.int32), (PAD, 90))
    res = []
    for n in (N, N + PAD):
        out = torch.full((n, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse, ws = torch.full((n, heads), 7.0, device="cuda"), new_ws(B.ds4x_paged_attn_workspace())
        if sparse:
            B.ds4x_paged_sparse_attn(pages, 16, table, cu, n_rows, dev(idx[:n]), q[:n], SCALE, out, lse, ws)
        else:
            B.ds4x_paged_attn(pages, 16, table, cu, mixed(end, [HIGH, LOW, 1 << 40, 900, 0])[:n], q[:n], SCALE, out, lse, ws,
                              row_begin=mixed([0, 3, 0, 0, 100, 0, 899], [LOW, HIGH, 0, 1 << 33, 5])[:n])
        assert B.ds4x_workspace_status(ws) == 0
        res.append((out, lse))
    (a, la), (b, lb) = res
    assert torch.all(b[N:] == 7.0) and torch.all(lb[N:] == 7.0)
    # (the tokens' rows may be cut otherwise among more tokens: equal to half a step of the output)
    assert torch.allclose(a.float(), b[:N].float(), rtol=2.0 ** -7, atol=2.0 ** -10) and torch.allclose(la, lb[:N], rtol=2.0 ** -18, atol=2.0 ** -16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_and_gather(dtype):
    B = require_gpu()
    pool, pages, table, cu, _ = setup(1)
    x = torch.randn((N + PAD, 512), device="cuda").to(dtype)
    x[N:] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").to(dtype).repeat(128)
    row0 = dev(np.array([38, 0, 895], dtype=np.int64))
    pos = mixed([1, 5, 1 << 20, 3, 4, 5, 6], [LOW, HIGH, -1])
    freq = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    res = []
    for n in (N, N + PAD):
        p, ws = pages.clone(), new_ws(256)
        out = torch.full((n, 512), 7.0, dtype=dtype, device="cuda")
        B.ds4x_paged_append(p, 16, table, cu, row0, x[:n], ws, pos=pos[:n], inv_freq=freq)
        B.ds4x_paged_gather(p, 16, table, cu, row0, out, ws)
        assert B.ds4x_workspace_status(ws) == 0
        res.append((p, out))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1][:N]) and torch.all(res[1][1][N:] == 7.0)
