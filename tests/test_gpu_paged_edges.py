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


def test_odd_queries_of_neighbouring_units():
    """Eight units a worker, one tile each; NaN and infinite queries in some heads of
    some tokens.  Each marks its own outputs and no others, time and again."""
    B = require_gpu()
    T, n = 8 * torch.cuda.get_device_properties(0).multi_processor_count, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    pages, table = appended(torch.randn((1, n, 512), generator=g, device="cuda"), 64)
    q = torch.randn((T, 64, 512), generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    end = torch.full((T,), n, dtype=torch.int64, device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    out, lse = attend(pages, 64, table, cu, end, q, ws)
    hit = torch.rand((T, 64), generator=g, device="cuda") < 0.4
    hit[::2] = False
    hit[1::4] = True
    bad = q.clone()
    at = torch.randint(512, (T, 64, 1), generator=g, device="cuda")
    odd = torch.where(torch.rand((T, 64, 1), generator=g, device="cuda") < 0.5, float("nan"), float("inf")).bfloat16()
    bad.scatter_(2, at, torch.where(hit[..., None], odd, q.gather(2, at)))
    for _ in range(20):
        o, l = attend(pages, 64, table, cu, end, bad, ws)
        assert same_bits(o[~hit], out[~hit]) and same_bits(l[~hit], lse[~hit])
        assert torch.isnan(o[hit]).all() and torch.isnan(l[hit]).all()


def sized(shape, seed, low, high):
    """Rows each at its own power of two, from 2^low to 2^high."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    return x * torch.exp2(torch.randint(low, high + 1, (*shape[:-1], 1), generator=g, device="cuda").float())


@pytest.mark.parametrize("heads", [8, 64])
def test_rows_of_different_size_give_the_same_bits_each_time(heads):
    B = require_gpu()
    S, n = 40, 5000
    x = sized((S, n, 512), 2, -2, 2)
    x[:, 700::900] = sized(x[:, 700::900].shape, 3, -40, -25)
    x[:, 1500::1300] = sized(x[:, 1500::1300].shape, 4, 21, 24)
    pages, table = appended(x, 64)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    T = 3
    q = (torch.randn((S * T, heads, 512), generator=g, device="cuda") * 2.0**-20).bfloat16()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * T
    end = n - torch.arange(S * T, device="cuda") % T
    ws = new_ws(B.ds4x_paged_attn_workspace())
    out, lse = attend(pages, 64, table, cu, end, q, ws)
    for _ in range(40):
        o, l = attend(pages, 64, table, cu, end, q, ws)
        assert same_bits(o, out) and same_bits(l, lse)
    pool = Pool([n], 64, 6, x=[np.zeros((n, 512), np.float32)])
    pool.pages, pool.table = pages.cpu().numpy(), table.cpu().numpy()
    for t in (0, S * T - 1):
        v = pool.values(t // T, np.arange(int(end[t])))
        check_token(out[t].double().cpu().numpy(), lse[t].double().cpu().numpy(), v, q[t].double().cpu().numpy(), SCALE)


def test_a_session_of_large_rows_does_not_touch_its_neighbours():
    """Short sessions side by side, several a worker: every other one's rows at sizes
    far apart, or not, leave the rest bit for bit."""
    B = require_gpu()
    S, n = 700, 128
    x = sized((S, n, 512), 7, -1, 1)
    y = x.clone()
    y[1::2] = sized(y[1::2].shape, 8, -40, 40)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    q = torch.randn((S, 64, 512), generator=g, device="cuda").bfloat16()
    cu, end = torch.arange(S + 1, dtype=torch.int32, device="cuda"), torch.full((S,), n, dtype=torch.int64, device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    got = []
    for z in (x, y):
        pages, table = appended(z, 32)
        got.append(attend(pages, 32, table, cu, end, q, ws))
    assert same_bits(got[0][0][::2], got[1][0][::2]) and same_bits(got[0][1][::2], got[1][1][::2])
    assert not same_bits(got[0][1][1::2], got[1][1][1::2])


@pytest.mark.parametrize("heads", [5, 8, 20])
def test_a_row_that_one_token_sees_leaves_the_others_bits(heads):
    """Tokens that share a pass: the rows that only later ones see are ordinary, far
    larger, far smaller, or bytes never written; the earlier ones' bits stay."""
    B = require_gpu()
    S, n, T, R = 150, 200, 8, 16
    x = sized((S, n, 512), 10, -1, 1)
    end = (n - T + 1 + torch.arange(S * T, device="cuda") % T)
    begin = torch.arange(S * T, device="cuda") % 2 * 60  # and rows at the front that every other token sees
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    q = torch.randn((S * T, heads, 512), generator=g, device="cuda").bfloat16()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * T
    ws = new_ws(B.ds4x_paged_attn_workspace())

    def bits(y, garbage=None):
        pages, table = appended(y, R)
        if garbage is not None:
            for r in range(garbage, n):  # plausible scales, NaN for values
                page = pages[table[:, r // R].long()]
                page[:, R * 224 + 128 * (r % R):][:, :128] = 0xFF
                page[:, R * 352 + 16 * (r % R):][:, :16] = 240 + r % 16
                pages[table[:, r // R].long()] = page
        o, l = attend(pages, R, table, cu, end, q, ws, begin=begin)
        return o.view(S, T, heads, 512), l.view(S, T, heads)

    out, lse = bits(x)
    for t in (0, 3, 6):  # tokens up to t keep their rows
        keep = n - T + 1 + t
        for size in (30, -60, None):
            y = x.clone()
            if size is not None:
                y[:, keep:] = sized(y[:, keep:].shape, 12, size - 1, size + 1)
            o, l = bits(y, keep if size is None else None)
            assert same_bits(o[:, :t + 1], out[:, :t + 1]) and same_bits(l[:, :t + 1], lse[:, :t + 1]), (t, size)
    y = x.clone()
    y[:, 5:60] = sized(y[:, 5:60].shape, 13, 25, 45)
    o, l = bits(y)
    assert same_bits(o[:, 1::2], out[:, 1::2]) and same_bits(l[:, 1::2], lse[:, 1::2])


@pytest.mark.parametrize("heads", [64, 16])
@pytest.mark.parametrize("n", [1 << 15, 1 << 20])
def test_a_row_above_many_small_ones(n, heads):
    """One row far above flat ones, each token's rows all one worker's: the many small
    weights together are a part of the output that must not be lost.

    Bound, beside paged_path's: a small weight enters the second product in fp16
    whose largest weight is at least 2^7: it is off by 2^-11 of itself where fp16 is
    normal; below that half a step is 2^-25, so 2^-25 / 2^7 = 2^-32 of the largest (or
    all of itself, where that is less: it becomes zero).  The products' fp32 sum goes
    over a run of 2^15 rows, 16 at a time, each of the 17 terms of a step cut off at
    2^-24 of the largest: 2^11 * 17 * 2^-24 < 2^-8 of the sum of sizes."""
    B = require_gpu()
    R, T = 64, torch.cuda.get_device_properties(0).multi_processor_count * (64 // heads)
    rng = np.random.default_rng(14)
    x = rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, -0.5], (16 * R, 512)).astype(np.float32)
    x[:, :32] = 0
    x[:, 448] = 5.0                # every row's largest exponent: 0
    x[0] = 0
    x[0, 0], x[0, 448], x[0, 100], x[0, 480] = 6.0, 5.0, 2.0, 1.0
    pages, _ = appended(torch.from_numpy(x).cuda()[None], R)
    table = (torch.arange(n // R, dtype=torch.int32, device="cuda") % 15 + 1)[None].contiguous()
    table[0, 0] = 0
    # logits: c for the one row, 0 for the others, in nats
    qv = np.zeros((heads, 512))
    qv[:, 0] = np.linspace(16.0, 18.5, heads) / (6 * SCALE)
    bits, qv = bf16(qv)
    q = bf16_dev(np.tile(bits, (T, 1, 1)))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    end = torch.full((T,), n, dtype=torch.int64, device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    out, lse = attend(pages, R, table, cu, end, q, ws)
    # the rows that there are, each as often as it stands
    tb = table[0].cpu().numpy()
    count = np.zeros(16 * R)
    for p in range(16):
        count[p * R:(p + 1) * R] = (tb == p).sum()
    v, count = x[count > 0].astype(np.float64), count[count > 0]
    w = np.exp(qv @ v.T * SCALE - (qv @ v[0] * SCALE)[:, None]) * count  # the one row's: 1
    z = w.sum(axis=1)
    p = w / z[:, None]
    ref, ref_lse = p @ v, (qv @ v[0]) * SCALE + np.log(z)
    size = p @ np.abs(v)
    few = (np.minimum(2.0 ** -32 * count / z[:, None], p) + 2.0 ** -11 * p) @ np.abs(v)
    dl = 32 * 2.0 ** -23 * np.abs(qv[:, :1]) * 6 * SCALE + 2.0 ** -21 * 20
    tol = 2.0 ** -8 * np.abs(ref) + few + (2.0 ** -8 + 2 * dl) * size
    for t in (0, T // 2, T - 1):
        o, l = out[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
        err = np.abs(o - ref)
        assert np.all(err <= tol), (t, (err / np.maximum(size, 1e-30)).max(), (tol / np.maximum(size, 1e-30)).min())
        assert np.all(np.abs(l - ref_lse) <= dl[:, 0] + 2.0 ** -18 * 20)


@pytest.mark.parametrize("heads, per", [(64, 1), (100, 1), (16, 3), (5, 8)])
@pytest.mark.parametrize("uneven", [False, True])
def test_units_of_several_runs(heads, per, uneven):
    """Units longer than one sum goes over (512 tiles of 64 rows): ends at, before and
    behind a run's, shares of one, two and three runs, whole and cut units, several
    tokens a unit, empty tokens among them; the same bits again.

    Bound: paged_path's, with the products' sum of a run (2^-8, above)."""
    B = require_gpu()
    R, run_rows = 64, 512 * 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator(device="cuda")
    g.manual_seed(30)
    pages, _ = appended(torch.randn((1, 16 * R, 512), generator=g, device="cuda") + 0.25, R)
    S = 12 if uneven else sms * 2
    room = 1 << (20 if uneven else 17)
    table = (torch.arange(room // R, dtype=torch.int32, device="cuda") * 7 % 16).expand(S, -1).contiguous()
    rng = np.random.default_rng(31)
    some = np.array([run_rows - 1, run_rows, run_rows + 1, 2 * run_rows, 2 * run_rows + 64, 3 * run_rows + 17, 0, 5, room])
    end = np.sort(rng.choice(some[some <= room], (S, per)), axis=1) if not uneven else room - np.sort(rng.integers(0, 200000, (S, per)))[:, ::-1]
    begin = np.where(rng.random((S, per)) < 0.3, rng.integers(0, 3000, (S, per)), 0)
    end, begin = end.reshape(-1), begin.reshape(-1)
    bits, qv = queries(S * per, heads, 32, 2.0)
    q = bf16_dev(bits)
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda") * per
    ws = new_ws(B.ds4x_paged_attn_workspace())
    de, db = dev(end.astype(np.int64)), dev(begin.astype(np.int64))
    out, lse = attend(pages, R, table, cu, de, q, ws, begin=db)
    o2, l2 = attend(pages, R, table, cu, de, q, ws, begin=db)
    assert same_bits(out, o2) and same_bits(lse, l2)
    pool = Pool([16 * R], R, 33, x=[np.zeros((16 * R, 512), np.float32)])
    pool.pages, pool.table = pages.cpu().numpy(), np.arange(16)[None]
    v = pool.values(0, np.arange(16 * R))
    page = table[0].cpu().numpy()
    for t in sorted({0, 1, S * per - 1, *rng.choice(S * per, 20).tolist()}):
        rows = np.arange(begin[t], max(begin[t], end[t]))
        count = np.bincount(page[rows // R] * R + rows % R, minlength=16 * R)
        o, l = out[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
        if len(rows) == 0:
            assert np.all(o == 0) and np.all(np.isneginf(l))
            continue
        logit = np.where(count > 0, qv[t] @ v.T * SCALE, -np.inf)
        top = logit.max(axis=1, keepdims=True)
        w = np.exp(logit - top) * count
        z = w.sum(axis=1, keepdims=True)
        p, ref_lse = w / z, (top + np.log(z))[:, 0]
        size = p @ np.abs(v)
        dl = (32 * 2.0 ** -23 * SCALE * (np.abs(qv[t]) @ np.abs(v).T)).max(axis=1) + 2.0 ** -21 * np.maximum(1, np.abs(top[:, 0]))
        tol = 2.0 ** -8 * np.abs(p @ v) + (2.0 ** -11 + 2.0 ** -8 + 2 * dl[:, None]) * size + 2.0 ** -20
        assert np.all(np.abs(o - p @ v) <= tol), (t, begin[t], end[t], np.abs(o - p @ v).max())
        assert np.all(np.abs(l - ref_lse) <= dl + 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse))


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


@pytest.mark.parametrize("heads", [64, 8])
def test_an_empty_range_past_the_table_is_no_fault(heads):
    """A token that sees nothing is zeros and flags nothing, wherever its range lies."""
    pool = Pool([3000, 100], 16, 18)
    tokens = [5, 3]
    end = np.array([3000, 1 << 40, 1 << 62, 5, 1 << 33, 100, 1 << 40, 99])
    begin = np.array([0, 1 << 40, (1 << 63) - 1, 7, 1 << 34, 0, 1 << 41, 3])
    q, qv = queries(8, heads, 19)
    got, lse = run(pool, tokens, q, begin=begin, end=end)
    check(pool, tokens, qv, lambda t, s: np.arange(begin[t], max(end[t], begin[t])) if end[t] <= 3000 else np.arange(0), got, lse)
    # one row past it is one
    end[1], begin[1] = pool.table.shape[1] * 16 + 1, pool.table.shape[1] * 16
    run(pool, tokens, q, begin=begin, end=end, status=-7)


@pytest.mark.parametrize("rows", [-1, -(1 << 31), -(1 << 32) + 90, -(1 << 63) + 90, -(1 << 63)])
def test_a_sequence_of_fewer_than_no_rows_has_none(rows):
    pool = Pool([100, 50], 32, 20)
    q, qv = queries(2, 64, 21)
    idx = np.tile(np.arange(50, dtype=np.int32), (2, 1))
    got, lse = run(pool, [1, 1], q, idx=idx, n_rows=[rows, 50], status=-7)
    check(pool, [1, 1], qv, lambda t, s: np.arange(50) if s else np.arange(0), got, lse)


@pytest.mark.parametrize("heads", [64, 12])
def test_outputs_between_queries(heads):
    """Queries and outputs of one buffer, token by token in turn: what the call gives apart."""
    B = require_gpu()
    pool = Pool([900, 300], 32, 22)
    tokens = [9, 4]
    q, qv = queries(13, heads, 23)
    end = np.concatenate([np.arange(892, 901), np.arange(297, 301)])
    want, want_lse = run(pool, tokens, q, end=end)
    both = torch.full((13, 2, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    both[:, 0] = bf16_dev(q)
    lse = torch.zeros((13, heads), device="cuda")
    cu, ws = dev(np.array([0, 9, 13], dtype=np.int32)), new_ws(B.ds4x_paged_attn_workspace())
    B.ds4x_paged_attn(dev(pool.pages), 32, dev(pool.table), cu, dev(end.astype(np.int64)), both[:, 0], SCALE, both[:, 1], lse, ws)
    assert np.array_equal(bf16_host_bits(both[:, 1].contiguous()), want) and np.array_equal(lse.cpu().numpy(), want_lse)
    assert np.array_equal(bf16_host_bits(both[:, 0].contiguous()), q)


@pytest.mark.parametrize("heads", [5, 64])
def test_runs_without_a_row(heads):
    """A long unit whose first, middle or last runs' pages are nowhere (and flagged), one
    without any row at all, NaN queries among them."""
    B = require_gpu()
    R, run = 64, 512
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    S = 4 * sms
    g = torch.Generator(device="cuda")
    g.manual_seed(34)
    pages, _ = appended(torch.randn((1, 4 * R, 512), generator=g, device="cuda"), R)
    table = (torch.arange(3 * run, dtype=torch.int32, device="cuda") % 4).expand(S, -1).contiguous()
    table[0::4, :run], table[1::4, run:2 * run], table[2::4, 2 * run:], table[3::4] = -1, -1, -1, -1
    q = torch.randn((S, heads, 512), generator=g, device="cuda").bfloat16()
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    end = torch.full((S,), 3 * run * R, dtype=torch.int64, device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    out, lse = attend(pages, R, table, cu, end, q, ws, status=-7)
    assert torch.all(out[3::4] == 0) and torch.all(lse[3::4] == -float("inf"))
    # 4 pages, each 256 times
    v = Pool([4 * R], R, 35, x=[np.zeros((4 * R, 512), np.float32)])
    v.pages, v.table = pages.cpu().numpy(), np.arange(4)[None]
    rows = v.values(0, np.arange(4 * R))
    for t in (0, 1, 2, S - 4, S - 3, S - 2):
        check_token(out[t].double().cpu().numpy(), lse[t].double().cpu().numpy() - np.log(256), rows, q[t].double().cpu().numpy(), SCALE)
    bad = q.clone()
    bad[:, 1, 77] = float("nan")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    o, l = attend(pages, R, table, cu, end, bad, ws, status=-7)
    keep = [h for h in range(heads) if h != 1]
    seen = torch.arange(S, device="cuda") % 4 != 3
    assert same_bits(o[:, keep], out[:, keep]) and same_bits(l[:, keep], lse[:, keep])
    assert torch.isnan(o[seen, 1]).all() and torch.isnan(l[seen, 1]).all()
    assert torch.all(o[~seen] == 0) and torch.all(l[~seen] == -float("inf"))


@pytest.mark.parametrize("heads, lists", [(3, False), (65, False), (65, True)])
def test_as_many_tokens_as_a_call_takes(heads, lists):
    """65,535 tokens; with 65 heads the queries go past 2^31 elements."""
    B = require_gpu()
    T, S, n, R = 65535, 300, 70, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(36)
    pages, table = appended(torch.randn((S, n, 512), generator=g, device="cuda"), R)
    cuts = torch.sort(torch.randint(T + 1, (S - 1,), generator=g, device="cuda"))[0].int()
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cuts, torch.full((1,), T, dtype=torch.int32, device="cuda")])
    q = torch.randn((T, heads, 512), generator=g, device="cuda", dtype=torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((T, heads), device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    end = torch.randint(n + 1, (T,), generator=g, device="cuda")
    idx = torch.randint(-1, n, (T, 40), generator=g, device="cuda", dtype=torch.int32)
    if lists:
        B.ds4x_paged_sparse_attn(pages, R, table, cu, torch.full((S,), n, dtype=torch.int64, device="cuda"), idx, q, SCALE, out, lse, ws)
    else:
        B.ds4x_paged_attn(pages, R, table, cu, end, q, SCALE, out, lse, ws)
    assert B.ds4x_workspace_status(ws) == 0
    pool = Pool([n] * S, R, 37, x=[np.zeros((n, 512), np.float32)] * S)
    pool.pages, pool.table = pages.cpu().numpy(), table.cpu().numpy()
    seq = torch.searchsorted(cu[1:], torch.arange(T, device="cuda", dtype=torch.int32), right=True).cpu().numpy()
    for t in [0, 1, 2, 8191, 32767, 32768, *range(40000, 65535, 1771), T - 2, T - 1]:
        rows = idx[t].cpu().numpy() if lists else np.arange(int(end[t]))
        check_token(out[t].double().cpu().numpy(), lse[t].double().cpu().numpy(), pool.values(seq[t], rows[rows >= 0]), q[t].double().cpu().numpy(), SCALE)
    del q, out
    torch.cuda.empty_cache()
