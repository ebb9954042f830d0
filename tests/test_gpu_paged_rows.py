"""ds4x_paged_append and ds4x_paged_gather against the oracle.

Without rotation the whole pool is compared byte for byte (so rows that no
token names, the pages' other bytes and other pages are seen to stay).  With
rotation the codes and block scales are exact too; the RoPE values are off by
half an FP16 step plus the rotation's fp32 products and fp32 cos and sin
(2^-21 of the pair's size covers them)."""

import numpy as np
import pytest
import torch

from gpu_path import dev, new_ws, require_gpu
from oracle import paged as O
from paged_path import Pool, bf16

pytestmark = pytest.mark.gpu


def run_append(pool, tokens, row0, x, n=None, pos=None, freq=None, style=0, dtype=torch.float32, pad=0, status=0):
    """Appends tokens[s] rows to each sequence from row0[s]; x f32 [n, 512]
    with any tokens past the sequences' being padding.  Returns the pool's
    pages and the rows read back (f32 and bf16 bits)."""
    B = require_gpu()
    cu = dev(np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32))
    pages, table = dev(pool.pages), dev(pool.table)
    wide = torch.full((x.shape[0], 512 + pad), float("nan"), device="cuda", dtype=dtype)
    wide[:, :512] = dev(x).to(dtype)
    ws = new_ws(256)
    r0 = dev(np.asarray(row0, dtype=np.int64))
    B.ds4x_paged_append(pages, pool.R, table, cu, r0, wide[:, :512], ws,
                        pos=None if pos is None else dev(np.asarray(pos, dtype=np.int64)),
                        inv_freq=None if freq is None else dev(np.asarray(freq, dtype=np.float32)), rope_style=style)
    back = []
    for t in (torch.float32, torch.bfloat16):
        out = torch.full((x.shape[0], 512 + pad), 7.0, device="cuda", dtype=t)
        B.ds4x_paged_gather(pages, pool.R, table, cu, r0, out[:, :512], ws)
        torch.cuda.synchronize()
        assert torch.all(out[:, 512:] == 7.0)
        back.append(out[:, :512])
    assert B.ds4x_workspace_status(ws) == status
    return pages.cpu().numpy(), back[0].cpu().numpy(), back[1].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def places(pool, tokens, row0):
    """(sequence, row) of each token."""
    return [(s, r0 + j) for s, (t, r0) in enumerate(zip(tokens, row0)) for j in range(t)]


def expected(pool, tokens, row0, x):
    want = pool.pages.copy()
    sr = places(pool, tokens, row0)
    rows = np.array([r for _, r in sr])
    page = pool.table[[s for s, _ in sr], rows // pool.R]
    q = O.quantise(x[:len(sr)])
    O.write(want, pool.R, page, rows % pool.R, *q)
    return want, O.values(*q)


SPECIAL = np.array([0.0, -0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, -6.0, 0.2500001, 4.9999995,
                    2.0 ** -100, -2.0 ** -126, 2.0 ** 60, 65504.0, 1e-30, 3e38, -3e38, 6.0 * 2.0 ** 96], dtype=np.float32)


@pytest.mark.parametrize("page_rows", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens, row0, pad", [([1], [0], 0), ([1, 0, 1, 1], [255, 3, 0, 17], 8), ([33, 0, 200, 1], [0, 0, 61, 15], 24),
                                               ([0, 0, 5], [0, 0, 300], 0)])
def test_append_without_rotation_is_byte_exact(page_rows, dtype, tokens, row0, pad):
    pool = Pool([a + b for a, b in zip(tokens, row0)], page_rows, 11)
    n = sum(tokens)
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((n + 3, 512)) * 2.0 ** rng.integers(-8, 9, (n + 3, 1))).astype(np.float32)  # 3 padding tokens
    x[0, :len(SPECIAL)] = SPECIAL[:]
    x[n - 1, :64] = 0
    x[n - 1, 448:] = rng.choice(SPECIAL[:16], 64)
    x = bf16(x)[1].astype(np.float32) if dtype == torch.bfloat16 else x
    pages, back, back16 = run_append(pool, tokens, row0, x, dtype=dtype, pad=pad)
    want, vals = expected(pool, tokens, row0, x)
    assert np.array_equal(pages, want)
    assert np.array_equal(back[:n].astype(np.float64), vals) and np.all(back[n:] == 7.0)
    assert np.array_equal(back16[:n], bf16(vals)[0]) and np.all(back16[n:] == bf16(np.full(1, 7.0))[0])


def test_special_rows():
    """All zero, one value a row over the whole exponent range, ties."""
    x = np.zeros((1 + 24 * 8, 512), dtype=np.float32)
    for i in range(24 * 8):
        x[1 + i, (37 * i) % 512] = SPECIAL[i % 24] * (1 if i % 3 else -1)
    pool = Pool([len(x)], 64, 13)
    pages, back, _ = run_append(pool, [len(x)], [0], x)
    want, vals = expected(pool, [len(x)], [0], x)
    assert np.array_equal(pages, want) and np.array_equal(back.astype(np.float64), vals)


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("base, sign", [(0, 1), (1 << 20, 1), ((1 << 31) + 12345, 1), ((1 << 40) + 7, 1), (5000, -1), (-(1 << 22), 1)])
def test_rotation(style, base, sign):
    rng = np.random.default_rng(14)
    tokens, row0 = [40, 0, 57], [0, 0, 30]
    n = sum(tokens)
    x = rng.standard_normal((n, 512)).astype(np.float32)
    pos = base + rng.integers(0, 100, n)
    freq = sign * (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    freq[0], freq[5] = 7.5 * sign, 0.0  # more than a turn a position, and none
    pool = Pool([a + b for a, b in zip(tokens, row0)], 32, 15)
    pages, back, _ = run_append(pool, tokens, row0, x, pos=pos, freq=freq, style=style)
    want, _ = expected(pool, tokens, row0, x)
    sr = places(pool, tokens, row0)
    rows = np.array([r for _, r in sr])
    page = pool.table[[s for s, _ in sr], rows // 32]
    got, ref = O.read(pages, 32, page, rows % 32), O.read(want, 32, page, rows % 32)
    assert np.array_equal(got[:, :448], ref[:, :448])
    assert np.array_equal(got, back.astype(np.float64))
    turned = O.rotate(x, pos, freq, bool(style))[:, 448:]
    i = np.arange(32)
    a, b = (i, 32 + i) if style else (2 * i, 2 * i + 1)
    size = np.empty((n, 64))
    size[:, a] = size[:, b] = np.hypot(turned[:, a], turned[:, b])
    # the turn: pos 2^-63 of a turn, and its 32 bits as a float (2^-25 of half a turn)
    ang = 2 * np.pi * (np.abs(pos).max() * 2.0 ** -63 + 2.0 ** -26)
    tol = 2.0 ** -11 * np.abs(turned) + (2.0 ** -21 + ang) * size + 2.0 ** -24 * np.abs(x).max()
    assert np.all(np.abs(got[:, 448:] - turned) <= tol), np.abs(got[:, 448:] - turned).max()


def test_position_defaults_to_the_row_number():
    rng = np.random.default_rng(16)
    x = rng.standard_normal((9, 512)).astype(np.float32)
    freq = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    pool = Pool([1009, 3], 64, 17, fill=0)
    a = run_append(pool, [7, 2], [1000, 1], x, freq=freq)
    b = run_append(pool, [7, 2], [1000, 1], x, freq=freq, pos=list(range(1000, 1007)) + [1, 2])
    assert np.array_equal(a[0], b[0])


def test_rows_that_the_table_does_not_place_are_left_out_and_flagged():
    rng = np.random.default_rng(18)
    x = rng.standard_normal((12, 512)).astype(np.float32)
    pool = Pool([40, 20], 16, 19)
    # sequence 0: rows 38 .. 43 (its pages end at 48); sequence 1: rows -2 .. 3, of which the first two lie nowhere
    pages, back, _ = run_append(pool, [6, 6], [38, -2], x, status=-7)
    keep = [0, 1, 2, 3, 4, 5, 8, 9, 10, 11]
    sr = [p for p in places(pool, [6, 6], [38, -2])]
    want = pool.pages.copy()
    s, r = np.array([sr[k][0] for k in keep]), np.array([sr[k][1] for k in keep])
    O.write(want, 16, pool.table[s, r // 16], r % 16, *O.quantise(x[keep]))
    assert np.array_equal(pages, want) and np.all(back[6:8] == 0)
    # an entry outside the pool and one past the sequence's entries
    pool.table[0, 2], pool.table[1, 1] = pool.n_pages, -1
    pages, back, _ = run_append(pool, [6, 6], [38, 30], x, status=-7)
    assert np.array_equal(pages, pool.pages) is True and np.all(back == 0)
    pages, back, _ = run_append(pool, [6, 6], [pool.table.shape[1] * 16, 1 << 40], x, status=-7)
    assert np.array_equal(pages, pool.pages) and np.all(back == 0)


def test_many_sequences_find_their_tokens():
    """Sequences by the hundred, most without a token (the search over cu_tokens)."""
    rng = np.random.default_rng(20)
    for n_seqs in (31, 32, 33, 1024, 1025, 2500):
        tokens = rng.choice([0, 0, 0, 1, 2, 5], n_seqs)
        tokens[-1] = 1
        pool = Pool([int(t) for t in tokens], 16, 21, fill=0)
        n = int(tokens.sum())
        x = rng.standard_normal((n, 512)).astype(np.float32)
        pages, _, _ = run_append(pool, list(tokens), [0] * n_seqs, x)
        want, _ = expected(pool, list(tokens), [0] * n_seqs, x)
        assert np.array_equal(pages, want)


def test_captured_append_follows_its_inputs():
    """One graph replayed with other tokens, rows, positions and values, on a stream of its own."""
    B = require_gpu()
    rng = np.random.default_rng(22)
    pool = Pool([64, 64, 64], 32, 23, fill=0)
    pages, table, ws = dev(pool.pages), dev(pool.table), new_ws(256)
    cu, row0 = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    x = torch.zeros((6, 512), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.ds4x_paged_append(pages, 32, table, cu, row0, x, ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.ds4x_paged_append(pages, 32, table, cu, row0, x, ws)
    for tokens, r0 in (([1, 1, 1], [0, 5, 9]), ([0, 6, 0], [1, 30, 2]), ([0, 0, 0], [0, 0, 0]), ([2, 0, 3], [33, 0, 61])):
        xs = rng.standard_normal((6, 512)).astype(np.float32)
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum(tokens)]), dtype=torch.int32))
        row0.copy_(torch.tensor(r0))
        x.copy_(torch.from_numpy(xs))
        pool.pages = pages.cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        want = expected(pool, tokens, r0, xs)[0] if sum(tokens) else pool.pages
        assert np.array_equal(pages.cpu().numpy(), want)
    assert B.ds4x_workspace_status(ws) == 0


def test_pool_beyond_32_bit_offsets():
    """A pool of more than 4 GiB whose pages in use lie at its end."""
    B = require_gpu()
    R = 256
    n_pages = (5 << 30) // (R * 368)
    pages = torch.zeros((n_pages, R * 368), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(24)
    x = rng.standard_normal((300, 512)).astype(np.float32)
    cu, r0 = dev(np.array([0, 300], dtype=np.int32)), dev(np.array([100], dtype=np.int64))
    ws = new_ws(256)
    B.ds4x_paged_append(pages, R, table, cu, r0, dev(x), ws)
    out = torch.empty((300, 512), device="cuda")
    B.ds4x_paged_gather(pages, R, table, cu, r0, out, ws)
    assert B.ds4x_workspace_status(ws) == 0
    assert np.array_equal(out.cpu().numpy().astype(np.float64), O.values(*O.quantise(x)))
    last = pages[-2:].flip(0).cpu().numpy()
    rows = np.arange(100, 400)
    assert np.array_equal(O.read(last, R, rows // R, rows % R), O.values(*O.quantise(x)))
    assert int(pages[:-2].max()) == 0
