"""ds4x_paged_attn and ds4x_paged_sparse_attn against the float64 oracle, within
the bounds that paged_path derives; and the calls together with the cache's
writer and the indexer."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, bf16_host_bits, dev, new_ws, pack, require_gpu
from oracle import codecs as C
from oracle import paged as O
from paged_path import Pool, bf16, check_token

pytestmark = pytest.mark.gpu
SCALE = 512.0 ** -0.5


def run(pool, tokens, q, begin=None, end=None, idx=None, n_rows=None, scale=SCALE, status=0, lse=True, pad=0, ws=None):
    """q [n, heads, 512] bf16 bits; (out bits [n, heads, 512], lse)."""
    B = require_gpu()
    n, H = q.shape[:2]
    cu = dev(np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32))
    pages = pool.dev if hasattr(pool, "dev") else dev(pool.pages)
    table = dev(pool.table)
    wq = torch.zeros((n, H * 512 + pad), dtype=torch.bfloat16, device="cuda")
    wq[:, :H * 512] = bf16_dev(q).view(n, -1)
    wo = torch.full((n, H * 512 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    qd, od = wq[:, :H * 512].unflatten(1, (H, 512)), wo[:, :H * 512].unflatten(1, (H, 512))
    ls = torch.full((n, H), 7.0, device="cuda") if lse else None
    ws = new_ws(B.ds4x_paged_attn_workspace()) if ws is None else ws
    i64 = lambda a: None if a is None else dev(np.asarray(a, dtype=np.int64))  # noqa: E731
    if idx is None:
        B.ds4x_paged_attn(pages, pool.R, table, cu, i64(end), qd, scale, od, ls, ws, row_begin=i64(begin))
    else:
        B.ds4x_paged_sparse_attn(pages, pool.R, table, cu, i64(n_rows), dev(np.asarray(idx, dtype=np.int32)), qd, scale, od, ls, ws)
    torch.cuda.synchronize()
    assert B.ds4x_workspace_status(ws) == status
    assert torch.all(wo[:, H * 512:] == 7.0)
    return bf16_host_bits(od.contiguous()), ls.cpu().numpy() if lse else None


def check(pool, tokens, qv, rows_of, got, lse, scale=SCALE):
    """Every token's output against the oracle over rows rows_of(t, s); padding
    tokens untouched."""
    out = C.bf16_decode(got).astype(np.float64)
    t = 0
    for s, c in enumerate(tokens):
        for _ in range(c):
            check_token(out[t], None if lse is None else lse[t].astype(np.float64), pool.values(s, rows_of(t, s)), qv[t], scale)
            t += 1
    assert np.all(out[t:] == 7.0) and (lse is None or np.all(lse[t:] == 7.0))


def queries(n, heads, seed, size=1.0):
    return bf16(np.random.default_rng(seed).standard_normal((n, heads, 512)) * size)


@pytest.mark.parametrize("rows", [0, 1, 2, 63, 64, 65, 127, 128, 129, 500, 2049])
@pytest.mark.parametrize("page_rows, heads", [(16, 64), (64, 64), (256, 64), (32, 1), (128, 7), (64, 33), (64, 100), (16, 128)])
def test_one_token(rows, page_rows, heads):
    pool = Pool([rows], page_rows, 100 + rows)
    q, qv = queries(1, heads, rows)
    got, lse = run(pool, [1], q, end=[rows])
    check(pool, [1], qv, lambda t, s: np.arange(rows), got, lse)


@pytest.mark.parametrize("heads", [64, 20, 16])
def test_ragged_tokens_ranges_and_padding(heads):
    """Sequences with none, one and many tokens; each token its own range, some
    empty, some backwards; padding tokens behind the last sequence."""
    rng = np.random.default_rng(30)
    rows, tokens = [0, 700, 5, 1300, 64, 257], [2, 0, 3, 9, 1, 4]
    pool = Pool(rows, 32, 31)
    n = sum(tokens)
    seq = np.repeat(np.arange(6), tokens)
    end = np.array([rng.integers(0, rows[s] + 1) for s in seq])
    begin = np.array([rng.integers(0, e + 1) for e in end])
    begin[4], end[4] = 4, 2          # backwards: nothing
    begin[7], end[7] = 640, 1300     # from a tile's edge
    begin[8], end[8] = -5, 1         # a begin below the first row is the first row
    begin[9], end[9] = 1299, 1300
    q, qv = queries(n + 3, heads, 32)
    pad_b, pad_e = np.append(begin, [0, 0, 0]), np.append(end, [1 << 40, 9, 9])
    got, lse = run(pool, tokens, q, begin=pad_b, end=pad_e, pad=24)
    check(pool, tokens, qv, lambda t, s: np.arange(max(0, begin[t]), max(end[t], max(0, begin[t]))), got, lse)
    got2, none = run(pool, tokens, q, begin=pad_b, end=pad_e, lse=False)
    assert none is None and np.array_equal(got, got2)


def test_causal_chunk_and_window():
    pool = Pool([600], 64, 33)
    T = 200
    q, qv = queries(T, 64, 34)
    end = np.arange(400, 400 + T) + 1
    got, lse = run(pool, [T], q, end=end)
    check(pool, [T], qv, lambda t, s: np.arange(end[t]), got, lse)
    got, lse = run(pool, [T], q, begin=end - 130, end=end)
    check(pool, [T], qv, lambda t, s: np.arange(end[t] - 130, end[t]), got, lse)


@pytest.mark.parametrize("rows", [[20011], [9000, 130, 40000, 0, 77], [1] * 70, [3000] * 40])
def test_long_and_uneven_sequences(rows):
    """Lengths that are split over many workers beside ones that are not."""
    pool = Pool(rows, 128, 35)
    q, qv = queries(len(rows), 64, 36)
    got, lse = run(pool, [1] * len(rows), q, end=rows)
    check(pool, [1] * len(rows), qv, lambda t, s: np.arange(rows[s]), got, lse)
    again, lse2 = run(pool, [1] * len(rows), q, end=rows)
    assert np.array_equal(got, again) and np.array_equal(lse.view(np.uint32), lse2.view(np.uint32))


@pytest.mark.parametrize("order", ["rising", "falling", "spike"])
def test_logits_that_move_the_maximum(order):
    """Rows whose logits rise by far more than any lazy bound, tile after tile."""
    rng = np.random.default_rng(37)
    n = 900
    d = rng.standard_normal(512)
    a = np.linspace(-6, 6, n) if order != "spike" else np.where(np.arange(n) % 97 == 96, 8.0, -2.0)
    x = (a[:, None] * d + 0.3 * rng.standard_normal((n, 512))).astype(np.float32)
    pool = Pool([n], 64, 38, x=[x if order != "falling" else x[::-1].copy()])
    qb, qv = bf16(np.stack([d * f + 0.1 * rng.standard_normal(512) for f in rng.choice([-2, -0.5, 0.1, 1, 3], 64)])[None])
    got, lse = run(pool, [1], qb, end=[n])
    check(pool, [1], qv, lambda t, s: np.arange(n), got, lse)


@pytest.mark.parametrize("shift", [-900.0, -200.0, 200.0, 900.0])
def test_logits_far_from_zero(shift):
    """Every logit far below or above zero, in a list whose first tiles hold no row
    and in a whole range."""
    rng = np.random.default_rng(70)
    n = 500
    d = rng.standard_normal(512)
    d /= np.linalg.norm(d)
    x = (4.0 * d + 0.2 * rng.standard_normal((n, 512))).astype(np.float32)
    pool = Pool([n], 32, 71, x=[x])
    qb, qv = bf16((d * shift / 4.0 / SCALE + rng.standard_normal((1, 64, 512)) * 0.1))
    got, lse = run(pool, [1], qb, end=[n])
    check(pool, [1], qv, lambda t, s: np.arange(n), got, lse)
    idx = np.full((1, 700), -1, dtype=np.int32)
    idx[0, 200:] = rng.integers(0, n, 500)
    got, lse = run(pool, [1], qb, idx=idx, n_rows=[n])
    check(pool, [1], qv, lambda t, s: idx[0, 200:], got, lse)
    # one worker for all tiles: the same among many tokens
    T = 200
    many = np.tile(idx, (T, 1))
    q2 = np.tile(qb, (T, 1, 1))
    got, lse = run(pool, [T], q2, idx=many, n_rows=[n])
    for t in (0, 7, 77, T - 1):
        check_token(C.bf16_decode(got).astype(np.float64)[t], lse[t].astype(np.float64), pool.values(0, idx[0, 200:]), qv[0], SCALE)


@pytest.mark.parametrize("heads", [1, 4, 8, 16, 20, 21, 31, 32, 33])
@pytest.mark.parametrize("window", [0, 70, 400])
def test_few_heads_many_tokens(heads, window):
    """Several tokens share a pass over their sequence's rows: chunks, drafts and
    lone tokens side by side, causal, windowed, with empty and far-apart ranges."""
    rng = np.random.default_rng(72)
    rows, tokens = [900, 0, 333, 64, 1500, 10], [37, 3, 1, 8, 0, 5]
    pool = Pool(rows, 16, 73)
    n = sum(tokens)
    seq = np.repeat(np.arange(6), tokens)
    end = np.concatenate([np.maximum(0, r - (c - 1 - np.arange(c))) for r, c in zip(rows, tokens)]).astype(np.int64)
    begin = np.maximum(0, end - window) if window else np.zeros(n, dtype=np.int64)
    end[[2, 9]] = 0                       # a token that sees nothing among ones that do
    begin[5], end[5] = 870, 871           # neighbours whose ranges do not meet
    begin[6], end[6] = 0, 3
    q, qv = queries(n + 2, heads, 74)
    got, lse = run(pool, tokens, q, begin=np.append(begin, [0, 0]), end=np.append(end, [9, 9]), pad=8)
    check(pool, tokens, qv, lambda t, s: np.arange(begin[t], max(end[t], begin[t])), got, lse)


@pytest.mark.parametrize("heads", [1, 2, 3, 11, 13, 16, 24])
def test_units_of_few_columns(heads):
    """Two, one and two tokens: units whose columns end far below 32, or between 32
    and 48; every value of the output is the token's own."""
    rows, tokens = [11, 80, 76], [2, 1, 2]
    pool = Pool(rows, 128, 79, extra_entries=400)
    end = np.array([10, 11, 80, 75, 76])
    for seed in range(4):
        q, qv = queries(7, heads, 790 + seed)
        got, lse = run(pool, tokens, q, end=np.append(end, [3, 3]), pad=16)
        check(pool, tokens, qv, lambda t, s: np.arange(end[t]), got, lse)
    q, qv = queries(40, heads, 795)
    got, lse = run(pool, [0, 33, 5], q, end=np.append(np.arange(33) + 40, [70, 71, 72, 73, 74, 9, 9]))
    check(pool, [0, 33, 5], qv, lambda t, s: np.arange(t + 40 if s == 1 else 70 + t - 33), got, lse)


@pytest.mark.parametrize("heads", [8, 20, 64])
def test_rows_that_only_some_tokens_see(heads):
    """A drafted token's range that reaches into rows never written (NaN where their
    values would be) leaves its neighbours' results alone; pages between the tokens'
    ranges that no token sees may be anywhere."""
    R, seen = 16, 1000
    pool = Pool([seen + 40, 4000], R, 77)
    codes, tails = R * 224, R * 128
    for j in range(seen, seen + 40):  # plausible scales, NaN and infinities for values
        page = pool.pages[pool.table[0, j // R]]
        page[codes + 128 * (j % R):codes + 128 * (j % R) + 128] = [0x00, 0x7E, 0x00, 0x7C, 0x00, 0xFC, 0x01, 0xFE] * 16
        page[codes + tails + 16 * (j % R):][:16] = [200] * 15 + [0]
    end = np.array([seen - 2, seen - 1, seen + 7, seen + 40, seen, seen - 3])
    begin = np.array([0, 400, 0, 900, 0, -5])
    q, qv = queries(6, heads, 78)
    got, lse = run(pool, [6, 0], q, begin=begin, end=end)
    out = C.bf16_decode(got).astype(np.float64)
    for t in (0, 1, 4, 5):
        check_token(out[t], lse[t].astype(np.float64), pool.values(0, np.arange(max(0, begin[t]), end[t])), qv[t], SCALE)
    # rows 200 .. 599 placed nowhere, and no token's
    pool.table[0, 200 // R + 1:592 // R] = -3
    begin, end = np.array([0, 0, 600, 700, 3, 0]), np.array([200, 150, 1000, 800, 3, 0])
    got, lse = run(pool, [6, 0], q, begin=begin, end=end)
    check(pool, [6, 0], qv, lambda t, s: np.arange(begin[t], max(begin[t], end[t])), got, lse)


@pytest.mark.parametrize("heads", [5, 16])
def test_few_heads_over_long_rows_and_many_units(heads):
    pool = Pool([6000, 200], 64, 75)
    tokens = [130, 70]
    n = sum(tokens)
    end = np.concatenate([6000 - 129 + np.arange(130), 200 - 69 + np.arange(70)])
    q, qv = queries(n, heads, 76)
    got, lse = run(pool, tokens, q, end=end)
    check(pool, tokens, qv, lambda t, s: np.arange(end[t]), got, lse)
    again, lse2 = run(pool, tokens, q, end=end)
    assert np.array_equal(got, again) and np.array_equal(lse.view(np.uint32), lse2.view(np.uint32))


@pytest.mark.parametrize("heads", [8, 64])
def test_a_head_does_not_touch_its_neighbours(heads):
    """Heads and tokens of very different size side by side; then NaN and infinity in
    some: the others' results stay bit for bit."""
    pool = Pool([500, 4000], 32, 80)  # (room enough that few heads' tokens share passes)
    rng = np.random.default_rng(81)
    size = rng.integers(-60, 5, (9, heads, 1))
    q, qv = bf16(rng.standard_normal((9, heads, 512)) * 2.0**size)
    end = 500 - 8 + np.arange(9)
    got, lse = run(pool, [9, 0], q, end=end)
    check(pool, [9, 0], qv, lambda t, s: np.arange(end[t]), got, lse)
    bad = q.copy()
    bad[2, 3, 17], bad[5, :, 100], bad[7, 0, 511], bad[7, 1, 0] = 0x7FC0, 0x7F80, 0xFF80, 0xFFC1
    hit = np.zeros((9, heads), dtype=bool)
    hit[2, 3] = hit[5] = hit[7, :2] = True
    got2, lse2 = run(pool, [9, 0], bad, end=end)
    assert np.array_equal(got2[~hit], got[~hit])
    assert np.array_equal(lse2[~hit].view(np.uint32), lse[~hit].view(np.uint32))
    # (an infinite query has no finite logit: its softmax is NaN as well)
    assert np.isnan(C.bf16_decode(got2[hit])).all() and np.isnan(lse2[hit]).all()
    # the same where a unit's parts are joined, by each of the joins
    idx = np.tile(np.arange(500, dtype=np.int32), (9, 1))
    for n in (1, 9, 40):
        i = np.resize(idx, (n, 500))
        out, l = run(pool, [n, 0], np.resize(bad, (n, heads, 512)), idx=i, n_rows=[500, 0])
        h = np.resize(hit, (n, heads))
        assert np.array_equal(np.isnan(C.bf16_decode(out)).all(axis=2), h) and np.array_equal(np.isnan(l), h)
        assert np.array_equal(np.isnan(C.bf16_decode(out)).any(axis=2), h)
    long = Pool([9000], 64, 84)
    out, l = run(long, [1], bad[2:3], end=[9000])
    assert np.array_equal(np.isnan(C.bf16_decode(out)).all(axis=2), hit[2:3]) and np.array_equal(np.isnan(l), hit[2:3])


@pytest.mark.parametrize("heads", [8, 64])
def test_a_token_that_sees_nothing_is_zeros_whatever_its_query(heads):
    pool = Pool([90, 0, 9000], 16, 82)
    q, qv = queries(4, heads, 83)
    q[1] = 0x7FC0
    q[3] = 0xFF80
    got, lse = run(pool, [3, 1, 0], q, end=[70, 0, 90, 0])
    check(pool, [3, 1, 0], qv, lambda t, s: np.arange([70, 0, 90, 0][t]), got, lse)
    idx = np.full((4, 80), -1, dtype=np.int32)
    idx[0, :70], idx[2, :70] = np.arange(70), np.arange(20, 90)
    got, lse = run(pool, [3, 1, 0], q, idx=idx, n_rows=[90, 0, 0])
    check(pool, [3, 1, 0], qv, lambda t, s: idx[t][idx[t] >= 0], got, lse)


@pytest.mark.parametrize("spread", [0, 6, 12, 20, 60])
def test_row_and_block_scale_spread(spread):
    """Each block and each row at its own power of two, the RoPE part too: rows
    of very different size side by side, blocks far below their row's largest."""
    rng = np.random.default_rng(39 + spread)
    n = 400
    f = 2.0 ** rng.integers(-spread, spread + 1, (n, 16))
    x = rng.standard_normal((n, 512)) * np.repeat(f, 32, axis=1) * 2.0 ** rng.integers(-spread // 2, spread // 2 + 1, (n, 1))
    x[7] = 0.0
    x[8, :448] = 0.0
    x[9, 448:] = 0.0
    pool = Pool([n], 16, 40, x=[x.astype(np.float32)])
    q, qv = queries(1, 64, 41)
    scale = SCALE * 2.0 ** -(1.5 * spread)
    got, lse = run(pool, [1], q, end=[n], scale=scale)
    check(pool, [1], qv, lambda t, s: np.arange(n), got, lse, scale=scale)


@pytest.mark.parametrize("size", [0.0, 2.0 ** -100, 2.0 ** -20, 300.0, 2.0 ** 90])
def test_query_sizes(size):
    """Queries far outside FP16's range, and heads of very different size."""
    pool = Pool([300], 32, 42)
    h = np.ones((1, 64, 1))
    h[0, ::3] = 2.0 ** -12
    q, qv = bf16(np.random.default_rng(43).standard_normal((1, 64, 512)) * size * h)
    scale = SCALE / max(size, 2.0 ** -100)
    got, lse = run(pool, [1], q, end=[300], scale=scale)
    check(pool, [1], qv, lambda t, s: np.arange(300), got, lse, scale=scale)


def test_tiny_and_zero_rows():
    """All rows zero; all rows at the least scale; both beside ordinary ones."""
    rng = np.random.default_rng(44)
    x = rng.standard_normal((4, 150, 512))
    x[0] = 0.0
    x[1] *= 2.0 ** -97
    x[2, ::2] *= 2.0 ** -97
    x[3] *= 2.0 ** 90
    pool = Pool([150] * 4, 32, 45, x=[a.astype(np.float32) for a in x])
    q, qv = queries(4, 64, 46)
    for s, scale in ((0, SCALE), (1, SCALE), (2, SCALE), (3, SCALE * 2.0 ** -90)):
        got, lse = run(pool, [0] * s + [1] + [0] * (3 - s), q[s:s + 1], end=[150], scale=scale)
        check_token(C.bf16_decode(got).astype(np.float64)[0], lse[0].astype(np.float64), pool.values(s, np.arange(150)), qv[s], scale)


def test_unplaced_rows_are_left_out_and_flagged():
    pool = Pool([200, 90], 16, 47)
    q, qv = queries(2, 64, 48)
    pool.table[0, 3], pool.table[0, 9], pool.table[1, 0] = -1, pool.n_pages, -(1 << 31)
    keep = [np.array([r for r in range(200) if r // 16 not in (3, 9)]), np.arange(16, 90)]
    got, lse = run(pool, [1, 1], q, end=[200, 90], status=-7)
    check(pool, [1, 1], qv, lambda t, s: keep[s], got, lse)
    # a range that runs past the table: what it places counts
    full = Pool([32], 16, 49, extra_entries=0)
    got, lse = run(full, [1], q[:1], end=[1 << 40], status=-7)
    check(full, [1], qv[:1], lambda t, s: np.arange(32), got, lse)


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 300, 512, 1100])
@pytest.mark.parametrize("heads", [64, 16, 100])
def test_sparse_lists(k, heads):
    rng = np.random.default_rng(50 + k)
    rows, tokens = [3000, 1, 700], [3, 1, 2]
    pool = Pool(rows, 64, 51)
    n = sum(tokens)
    seq = np.repeat(np.arange(3), tokens)
    idx = np.stack([rng.integers(0, rows[s], k) for s in seq]).astype(np.int32)  # rows may repeat: each counts
    idx[rng.random(idx.shape) < 0.2] = -1
    idx[1] = -1                      # a list without a row
    idx[2, :] = -1
    idx[2, k - 1] = 2999             # one row, at the list's end
    q, qv = queries(n + 2, heads, 52)
    got, lse = run(pool, tokens, q, idx=np.concatenate([idx, np.full((2, k), 1 << 30, np.int32)]), n_rows=rows, pad=8)
    check(pool, tokens, qv, lambda t, s: idx[t][idx[t] >= 0], got, lse)


def test_sparse_entries_outside_are_skipped_and_flagged():
    pool = Pool([100, 50], 32, 53)
    q, qv = queries(2, 64, 54)
    idx = np.tile(np.arange(80, dtype=np.int32), (2, 1))
    idx[0, 3], idx[0, 70], idx[1, 0] = -2, 100, -(1 << 31)
    idx[0, 5] = (1 << 31) - 1
    got, lse = run(pool, [1, 1], q, idx=idx, n_rows=[100, 50], status=-7)
    keep = [np.array([j for j in range(80) if j not in (3, 5, 70)]), np.arange(1, 50)]
    check(pool, [1, 1], qv, lambda t, s: keep[s], got, lse)


def test_sparse_over_every_row_is_the_dense_result():
    """The same rows in the same order: the same numbers."""
    pool = Pool([777], 64, 55)
    q, _ = queries(1, 64, 56)
    a, la = run(pool, [1], q, end=[777])
    b, lb = run(pool, [1], q, idx=np.arange(777, dtype=np.int32)[None], n_rows=[777])
    assert np.array_equal(a, b) and np.array_equal(la, lb)


def test_many_tokens_of_a_list_each():
    """A prompt's chunk: tokens by the hundred over the same sequence."""
    rng = np.random.default_rng(57)
    pool = Pool([4000], 64, 58)
    T, k = 700, 130
    idx = np.stack([rng.choice(4000, k, replace=False) for _ in range(T)]).astype(np.int32)
    q, qv = queries(T, 64, 59)
    got, lse = run(pool, [T], q, idx=idx, n_rows=[4000])
    out = C.bf16_decode(got).astype(np.float64)
    for t in list(range(0, T, 23)) + [T - 1]:
        check_token(out[t], lse[t].astype(np.float64), pool.values(0, idx[t]), qv[t], SCALE)


def test_rows_beyond_32_bit_offsets():
    """A pool of more than 4 GiB, the sequence's pages at both of its ends."""
    B = require_gpu()
    R = 64
    pool = Pool([200], R, 60, extra_pages=0)
    n_pages = (5 << 30) // (R * 368)
    pool.dev = torch.zeros((n_pages, R * 368), dtype=torch.uint8, device="cuda")
    small = dev(pool.pages)
    new = np.array([0, n_pages - 1, 1, n_pages - 2])[:pool.n_pages]
    for p in range(pool.n_pages):
        pool.dev[int(new[p])] = small[p]
    q, qv = queries(1, 64, 61)
    old = pool.table.copy()
    pool.table = np.where(old >= 0, new[np.maximum(old, 0)], -1).astype(np.int32)
    got, lse = run(pool, [1], q, end=[200])
    pool.table = old
    check(pool, [1], qv, lambda t, s: np.arange(200), got, lse)
    del pool.dev
    torch.cuda.empty_cache()
    assert B is not None


def test_captured_call_follows_its_inputs_on_another_stream():
    """One graph of two attention calls on one workspace, replayed with other
    lengths (other splits, empty ones among them) and values."""
    B = require_gpu()
    pool = Pool([5000, 300], 64, 62)
    pages, table = dev(pool.pages), dev(pool.table)
    ws = new_ws(B.ds4x_paged_attn_workspace())
    cu = dev(np.array([0, 1, 2], dtype=np.int32))
    end = torch.tensor([100, 300], device="cuda")
    idx = torch.full((2, 96), -1, dtype=torch.int32, device="cuda")
    n_rows = torch.tensor([5000, 300], device="cuda")
    qd = torch.zeros((2, 64, 512), dtype=torch.bfloat16, device="cuda")
    outs = [torch.zeros_like(qd) for _ in range(2)]
    lses = [torch.zeros((2, 64), device="cuda") for _ in range(2)]

    def calls():
        B.ds4x_paged_attn(pages, 64, table, cu, end, qd, SCALE, outs[0], lses[0], ws)
        B.ds4x_paged_sparse_attn(pages, 64, table, cu, n_rows, idx, qd, SCALE, outs[1], lses[1], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    rng = np.random.default_rng(63)
    for ends in ([5000, 0], [1, 300], [0, 0], [4999, 299]):
        q, qv = queries(2, 64, 64 + ends[0])
        ix = np.where(rng.random((2, 96)) < 0.5, rng.integers(0, 300, (2, 96)), -1).astype(np.int32)
        qd.copy_(bf16_dev(q))
        end.copy_(torch.tensor(ends))
        idx.copy_(dev(ix))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            g.replay()
        torch.cuda.synchronize()
        check(pool, [1, 1], qv, lambda t, s: np.arange(ends[s]), bf16_host_bits(outs[0]), lses[0].cpu().numpy())
        check(pool, [1, 1], qv, lambda t, s: ix[t][ix[t] >= 0], bf16_host_bits(outs[1]), lses[1].cpu().numpy())
    assert B.ds4x_workspace_status(ws) == 0


@pytest.mark.parametrize("heads", [12, 64])
def test_captured_ragged_tokens(heads):
    """One graph, replayed with the tokens dealt otherwise over the sequences (few
    heads: other plans) and other lengths; tokens behind the last sequence stay."""
    B = require_gpu()
    rows, n = [700, 3000, 40], 40
    pool = Pool(rows, 64, 90)
    pages, table = dev(pool.pages), dev(pool.table)
    ws = new_ws(B.ds4x_paged_attn_workspace())
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    end = torch.zeros(n, dtype=torch.int64, device="cuda")
    q, qv = queries(n, heads, 91)
    qd = bf16_dev(q)
    out, lse = torch.zeros_like(qd), torch.zeros((n, heads), device="cuda")
    B.ds4x_paged_attn(pages, 64, table, cu, end, qd, SCALE, out, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.ds4x_paged_attn(pages, 64, table, cu, end, qd, SCALE, out, lse, ws)
    rng = np.random.default_rng(92)
    for tokens in ([40, 0, 0], [0, 0, 0], [1, 30, 4], [13, 13, 14], [0, 40, 0]):
        ends = np.array([rng.integers(0, rows[s] + 1) for s in np.repeat(np.arange(3), tokens)] + [5] * (n - sum(tokens)))
        cu.copy_(dev(np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)))
        end.copy_(dev(ends.astype(np.int64)))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check(pool, tokens, qv, lambda t, s: np.arange(ends[t]), bf16_host_bits(out), lse.cpu().numpy())
    assert B.ds4x_workspace_status(ws) == 0


def test_thousands_of_sequences():
    """More sequences than a plan holds at once; the last ones' tokens and rows."""
    S, heads = 4200, 16
    rng = np.random.default_rng(93)
    rows = rng.integers(0, 12, S)
    tokens = np.ones(S, dtype=int)
    tokens[[0, 9, 4095, 4096, S - 1]] = 5, 0, 4, 6, 7
    pool = Pool(list(rows), 16, 94)
    n = tokens.sum()
    seq = np.repeat(np.arange(S), tokens)
    end = np.array([rng.integers(0, rows[s] + 1) for s in seq])
    q, qv = queries(n, heads, 95)
    got, lse = run(pool, list(tokens), q, end=end)
    out = C.bf16_decode(got).astype(np.float64)
    for t in [*range(0, 12), *range(12, n, 401), *range(int(np.argmax(seq == 4094)), int(np.argmax(seq == 4098))), *range(n - 9, n)]:
        check_token(out[t], lse[t].astype(np.float64), pool.values(seq[t], np.arange(end[t])), qv[t], SCALE)


def test_two_calls_at_once():
    """Two streams, each with its workspace, its own cache and other shapes."""
    B = require_gpu()
    pools = [Pool([3000, 100], 64, 96), Pool([500, 2500], 16, 97)]
    shapes = [([1, 1], 64), ([30, 9], 10)]
    jobs = []
    for pool, (tokens, heads) in zip(pools, shapes):
        n = sum(tokens)
        end = np.repeat([pool.rows[0], pool.rows[1]], tokens) - np.arange(n) % 7
        q, qv = queries(n, heads, 98 + n)
        a = dict(pages=dev(pool.pages), table=dev(pool.table), cu=dev(np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)),
                 end=dev(end.astype(np.int64)), q=bf16_dev(q), ws=new_ws(B.ds4x_paged_attn_workspace()),
                 out=torch.zeros((n, heads, 512), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((n, heads), device="cuda"))
        jobs.append((pool, tokens, qv, end, a, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for pool, _, _, _, a, stream in jobs:
            with torch.cuda.stream(stream):
                B.ds4x_paged_attn(a["pages"], pool.R, a["table"], a["cu"], a["end"], a["q"], SCALE, a["out"], a["lse"], a["ws"])
    torch.cuda.synchronize()
    for pool, tokens, qv, end, a, _ in jobs:
        assert B.ds4x_workspace_status(a["ws"]) == 0
        check(pool, tokens, qv, lambda t, s: np.arange(end[t]), bf16_host_bits(a["out"]), a["lse"].cpu().numpy())


def test_append_select_attend_together():
    """A decode step as it is used: rows rotated and appended, the indexer's
    top-k over their 68-byte rows, attention over the selected rows and over
    every row; then one more row, and again."""
    B = require_gpu()
    rng = np.random.default_rng(65)
    n, R, k = 1500, 64, 256
    x = rng.standard_normal((n + 1, 512)).astype(np.float32)
    keys = rng.standard_normal((n + 1, 128)).astype(np.float32)
    freq = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    pos = dev(np.arange(n + 1, dtype=np.int64) * 4 + 3)
    pool = Pool([n + 1], R, 66)
    pages, table = dev(pool.pages), dev(pool.table)
    idx_rows, _ = pack(idx_in=keys)
    ws, ws_i = new_ws(B.ds4x_paged_attn_workspace()), new_ws(B.ds4x_index_score_topk_workspace(n + 1, k))
    qi = bf16_dev(bf16(rng.standard_normal((64, 128)))[0])
    w = dev((rng.random(64) / 8).astype(np.float32))
    q, qv = queries(1, 64, 67)
    qd = bf16_dev(q)
    one, xd = dev(np.array([0, 1], dtype=np.int32)), dev(x)
    for first, last in ((0, n), (n, n + 1)):
        cu = dev(np.array([0, last - first], dtype=np.int32))
        B.ds4x_paged_append(pages, R, table, cu, dev(np.array([first], dtype=np.int64)), xd[first:last], ws, pos=pos[first:last], inv_freq=freq)
        sel = torch.empty(k, dtype=torch.int32, device="cuda")
        B.ds4x_index_score_topk(idx_rows, last, qi, w, k, sel, None, ws_i)
        out, lse = torch.empty((2, 1, 64, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 1, 64), device="cuda")
        rows = dev(np.array([last], dtype=np.int64))
        B.ds4x_paged_sparse_attn(pages, R, table, one, rows, sel[None], qd, SCALE, out[0], lse[0], ws)
        B.ds4x_paged_attn(pages, R, table, one, rows, qd, SCALE, out[1], lse[1], ws)
        torch.cuda.synchronize()
        assert B.ds4x_workspace_status(ws) == 0
        pool.pages = pages.cpu().numpy()
        v = pool.values(0, np.arange(last))
        # what was appended: the rotated rows to the format's accuracy (E2M1: a quarter of the block's largest at most)
        turned = O.rotate(x[:last], np.arange(last) * 4 + 3, freq.cpu().numpy(), False)
        assert np.abs(v - turned).max() <= np.abs(turned).max() / 4
        picked = sel.cpu().numpy()
        assert len(set(picked.tolist())) == k and picked.min() >= 0
        for i, r in enumerate((v[picked], v)):
            check_token(C.bf16_decode(bf16_host_bits(out[i, 0])).astype(np.float64), lse[i, 0].cpu().numpy().astype(np.float64), r, qv[0], SCALE)
