"""Trees whose nodes share units (few heads, tables wide enough or drafts long
enough that the call has several tiles a worker): what one node does not see has
no part in its results, whatever it holds and whatever its neighbours are."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, bf16_host_bits, dev, new_ws, require_gpu
from oracle import codecs as C
from oracle import drafts as D
from paged_path import Pool, check_token
from test_gpu_drafts_together import Steps
from test_gpu_tree_attn import SCALE, check, queries, run

pytestmark = pytest.mark.gpu


def assert_shared(table, R, n_seqs, n, heads):
    """The condition under which neighbouring nodes share a unit."""
    require_gpu()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = n * -(-table.shape[1] * R // 64)
    assert heads <= 32 and n > n_seqs and most > 2 * min(sms, 160)


def hostile(pool, s, rows, rng):
    """Bytes that are widened but are no row: the record's last byte 0, scales of
    every kind, RoPE values NaN, infinite and large, any codes."""
    R = pool.R
    for r in rows:
        page, at = pool.table[s, r // R], r % R
        pool.pages[page, at * 224:at * 224 + 224] = rng.integers(0, 256, 224)
        tail = rng.choice(np.array([0x7E00, 0xFE00, 0x7C00, 0xFC00, 0x7BFF, 0x0001, 0x3C00], dtype=np.uint16), 64)
        pool.pages[page, R * 224 + at * 128:R * 224 + at * 128 + 128] = tail.view(np.uint8)
        scales = rng.choice(np.array([0, 1, 100, 127, 150, 254, 255], dtype=np.uint8), 16)
        scales[15] = 0
        pool.pages[page, R * 352 + at * 16:R * 352 + at * 16 + 16] = scales


def same(a, b):
    return np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.uint32), b[1].view(np.uint32))


# few units and many, of one worker and split over several
SIZES = [(11, 150, 400), (40, 150, 400), (40, 3000, 0), (14, 5000, 100), (130, 700, 0)]


@pytest.mark.parametrize("heads", [1, 3, 8, 12, 16, 20, 32])
@pytest.mark.parametrize("n, row0, extra", SIZES)
def test_rows_that_a_node_does_not_see_leave_its_bits(n, row0, extra, heads):
    rng = np.random.default_rng(150 + n)
    parent = D.tree(rng, n, "random")
    q, qv = queries(n, heads, 151)
    begin = np.full(n, 30)
    clean = Pool([row0 + n], 32, 152, extra_entries=extra + 1)
    assert_shared(clean.table, 32, 1, n, heads)
    got, lse = run(clean, [parent], [row0], q, begin=begin)
    check(clean, [parent], [row0], qv, got, lse, begin)
    for node in (0, n // 3, n - 1):
        other = Pool([row0 + n], 32, 152, extra_entries=extra + 1)
        hostile(other, 0, sorted(set(range(row0 + n)) - set(D.sees(parent, node, row0, 30))), rng)
        got2, lse2 = run(other, [parent], [row0], q, begin=begin)
        assert same((got[node], lse[node]), (got2[node], lse2[node]))


@pytest.mark.parametrize("heads", [1, 16, 20])
@pytest.mark.parametrize("n, row0, extra", SIZES)
def test_windows_that_leave_rows_to_some_nodes(n, row0, extra, heads):
    """Every second node's window begins late: the rows before it are hostile for
    the others only where no one of them is compared."""
    rng = np.random.default_rng(160 + n)
    parent = D.tree(rng, n, "level")
    q, _ = queries(n, heads, 161)
    begin = np.where(np.arange(n) % 2 == 0, row0 - 40, row0 - 7)
    got, lse = run(Pool([row0 + n], 32, 162, extra_entries=extra + 1), [parent], [row0], q, begin=begin)
    other = Pool([row0 + n], 32, 162, extra_entries=extra + 1)
    assert_shared(other.table, 32, 1, n, heads)
    hostile(other, 0, range(row0 - 7), rng)
    got2, lse2 = run(other, [parent], [row0], q, begin=begin)
    late = np.arange(n) % 2 == 1
    assert same((got[late], lse[late]), (got2[late], lse2[late]))


@pytest.mark.parametrize("heads", [2, 16, 20])
@pytest.mark.parametrize("n, row0, extra", SIZES)
def test_queries_that_are_not_finite_stay_in_their_node(n, row0, extra, heads):
    rng = np.random.default_rng(170 + n)
    parent = D.tree(rng, n, "level")
    pool = Pool([row0 + n], 32, 171, extra_entries=extra + 1)
    assert_shared(pool.table, 32, 1, n, heads)
    q, _ = queries(n, heads, 172)
    got, lse = run(pool, [parent], [row0], q)
    odd = q.copy()
    odd[3, 0, 5] = 0x7FC0
    odd[6, heads - 1, 0] = 0x7F80
    odd[n - 1, heads // 2, 511] = 0xFF80
    hit = np.zeros((n, heads), dtype=bool)
    hit[3, 0] = hit[6, heads - 1] = hit[n - 1, heads // 2] = True
    got2, lse2 = run(pool, [parent], [row0], odd)
    assert same((got[~hit], lse[~hit]), (got2[~hit], lse2[~hit]))
    assert np.all(np.isnan(lse2[hit])) and np.all(np.isnan(C.bf16_decode(got2[hit])))


@pytest.mark.parametrize("heads", [64, 100])
def test_queries_that_are_not_finite_through_the_joins_of_many_units(heads):
    """Nodes by themselves, their histories split over workers."""
    n, row0 = 40, 3000
    parent = D.tree(np.random.default_rng(173), n, "level")
    pool = Pool([row0 + n], 64, 174)
    q, _ = queries(n, heads, 175)
    got, lse = run(pool, [parent], [row0], q)
    odd = q.copy()
    hit = np.zeros((n, heads), dtype=bool)
    for node, h, d, bits in ((0, 0, 0, 0x7FC0), (17, heads - 1, 300, 0x7F80), (39, 33, 511, 0xFFFF)):
        odd[node, h, d] = bits
        hit[node, h] = True
    got2, lse2 = run(pool, [parent], [row0], odd)
    assert same((got[~hit], lse[~hit]), (got2[~hit], lse2[~hit]))
    assert np.all(np.isnan(lse2[hit])) and np.all(np.isnan(C.bf16_decode(got2[hit])))


@pytest.mark.parametrize("heads", [1, 12, 16, 20])
def test_parents_that_are_none_count_as_roots_and_are_flagged(heads):
    parent = [-1, 0, 2, 5, 1, -2, 3, 1 << 30, -(1 << 31), 4] + [9] * 30
    clean = [-1, 0, -1, -1, 1, -1, 3, -1, -1, 4] + [9] * 30
    pool = Pool([90 + 40], 16, 176, extra_entries=300)
    assert_shared(pool.table, 16, 1, 40, heads)
    q, qv = queries(40, heads, 177)
    got, lse = run(pool, [parent], [90], q, status=-7)
    check(pool, [clean], [90], qv, got, lse)


@pytest.mark.parametrize("heads", [3, 16, 20])
def test_rows_past_the_table_are_left_out_and_flagged(heads):
    """Drafts that run off a table's end and that begin beyond it, and a page that
    is none, in units of several nodes."""
    rng = np.random.default_rng(178)
    parent = D.tree(rng, 12, "chain")
    room = 4096
    pool = Pool([room] * 3, 64, 179, extra_entries=0)
    pool.table[2, 2] = pool.n_pages + 5
    assert_shared(pool.table, 64, 3, 36, heads)
    q, qv = queries(36, heads, 180)
    row0 = [room - 6, 1 << 40, 300]
    begin = np.full(36, room - 100)
    begin[24:] = 0
    got, lse = run(pool, [parent] * 3, row0, q, begin=begin, status=-7)
    out = C.bf16_decode(got).astype(np.float64)
    for t in range(36):
        s, j = divmod(t, 12)
        rows = [r for r in (D.sees(parent, j, row0[s], begin[t]) if s != 1 else range(room - 100, room)) if r < room]
        rows = [r for r in rows if not (s == 2 and 128 <= r < 192)]
        check_token(out[t], lse[t].astype(np.float64), pool.values(s, rows), qv[t], SCALE)


@pytest.mark.parametrize("heads", [1, 5, 16, 20])
def test_rows_of_very_different_size(heads):
    """Scales that lie far apart, on some nodes' lines only: a node whose rows are
    tame keeps its bits beside one whose are not."""
    rng = np.random.default_rng(181)
    n, row0 = 30, 80
    parent = D.tree(rng, n, "random")
    x = rng.standard_normal((row0 + n, 512)).astype(np.float32)
    tame = Pool([row0 + n], 32, 182, x=[x.copy()], extra_entries=300)
    q, qv = queries(n, heads, 183)
    assert_shared(tame.table, 32, 1, n, heads)
    got, lse = run(tame, [parent], [row0], q, scale=1e-3)
    x[row0 + 5] *= 2.0 ** 40
    x[row0 + 9] *= 2.0 ** -60
    x[row0 + 17] *= 2.0 ** -45
    far = Pool([row0 + n], 32, 182, x=[x], extra_entries=300)
    got2, lse2 = run(far, [parent], [row0], q, scale=1e-3)
    check(far, [parent], [row0], qv, got2, lse2, scale=1e-3)
    apart = np.array([not {5, 9, 17} & set(D.line(parent, j)) for j in range(n)])
    assert 5 < apart.sum() < n
    assert same((got[apart], lse[apart]), (got2[apart], lse2[apart]))


@pytest.mark.parametrize("heads", [2, 20])
def test_captured_call_follows_its_inputs(heads):
    B = require_gpu()
    rng = np.random.default_rng(184)
    n = 40
    pool = Pool([2040, 2040], 16, 185)
    assert_shared(pool.table, 16, 2, n, heads)
    pages, table = dev(pool.pages), dev(pool.table)
    cu, parent = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    row0 = torch.zeros(2, dtype=torch.int64, device="cuda")
    q = torch.zeros((n, heads, 512), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((n, heads), device="cuda")
    ws = new_ws(B.ds4x_paged_attn_workspace())
    call = lambda st=None: B.ds4x_paged_tree_attn(pages, 16, table, cu, row0, parent, q, SCALE, out, lse, ws, stream=st)  # noqa: E731
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k, (before, nodes) in enumerate([([30, 2000], [7, 33]), ([1990, 0], [20, 20]), ([10, 11], [40, 0]), ([0, 1500], [1, 39])]):
        trees = [D.tree(rng, m, "random") if m else [] for m in nodes]
        bits, qv = queries(n, heads, 186 + k)
        cu.copy_(torch.tensor([0, nodes[0], sum(nodes)], dtype=torch.int32))
        parent.copy_(torch.tensor([p for t in trees for p in t], dtype=torch.int32))
        row0.copy_(torch.tensor(before))
        q.copy_(bf16_dev(bits))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        check(pool, trees, before, qv, bf16_host_bits(out), lse.cpu().numpy())
    assert B.ds4x_workspace_status(ws) == 0


@pytest.mark.parametrize("captured", [False, True])
def test_steps_follow_one_another(captured):
    """A server's steps with a table made for long contexts."""
    steps = Steps(63)
    steps.d["table"] = dev(np.pad(steps.table, ((0, 0), (0, 500)), constant_values=-7))
    assert_shared(steps.d["table"], 16, 3, 24, 20)
    graph = None
    for k, shape in enumerate(["chain", "level", "random", "star", "level", "chain"]):
        steps.inputs(shape)
        steps.read_drafted()
        if captured and graph is None:
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                steps.calls()     # (moves rows: appended again by the replay)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                steps.calls()
        if captured:
            graph.replay()
        else:
            steps.calls()
        torch.cuda.synchronize()
        steps.check()
    assert steps.B.ds4x_workspace_status(steps.ws) == 0
