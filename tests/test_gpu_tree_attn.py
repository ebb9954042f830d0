"""ds4x_paged_tree_attn against the float64 oracle, within the bounds that
paged_path derives for the attention (the products and the softmax are the
same; a node only sees other rows)."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, bf16_host_bits, dev, new_ws, require_gpu
from oracle import codecs as C
from oracle import drafts as D
from paged_path import Pool, bf16, check_token

pytestmark = pytest.mark.gpu
SCALE = 512.0 ** -0.5


def run(pool, trees, row0, q, begin=None, status=0, lse=True, pad=0, scale=SCALE):
    """trees: each sequence's parents; q [n, heads, 512] bf16 bits, with more
    tokens than the trees have as padding: (out bits, lse)."""
    B = require_gpu()
    n, H = q.shape[:2]
    cu = dev(np.concatenate([[0], np.cumsum([len(t) for t in trees])]).astype(np.int32))
    parent = np.full(n, 9, dtype=np.int32)
    flat = [p for t in trees for p in t]
    parent[:len(flat)] = flat
    wq = torch.zeros((n, H * 512 + pad), dtype=torch.bfloat16, device="cuda")
    wq[:, :H * 512] = bf16_dev(q).view(n, -1)
    wo = torch.full((n, H * 512 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    qd, od = wq[:, :H * 512].unflatten(1, (H, 512)), wo[:, :H * 512].unflatten(1, (H, 512))
    ls = torch.full((n, H), 7.0, device="cuda") if lse else None
    ws = new_ws(B.ds4x_paged_attn_workspace())
    i64 = lambda a: None if a is None else dev(np.asarray(a, dtype=np.int64))  # noqa: E731
    B.ds4x_paged_tree_attn(dev(pool.pages), pool.R, dev(pool.table), cu, i64(row0), dev(parent), qd, scale, od, ls, ws,
                           row_begin=i64(begin))
    torch.cuda.synchronize()
    assert B.ds4x_workspace_status(ws) == status
    assert torch.all(wo[:, H * 512:] == 7.0)
    return bf16_host_bits(od.contiguous()), ls.cpu().numpy() if lse else None


def check(pool, trees, row0, qv, got, lse, begin=None, scale=SCALE):
    out = C.bf16_decode(got).astype(np.float64)
    t = 0
    for s, parent in enumerate(trees):
        for j in range(len(parent)):
            rows = D.sees(parent, j, row0[s], 0 if begin is None else begin[t])
            check_token(out[t], None if lse is None else lse[t].astype(np.float64), pool.values(s, rows), qv[t], scale)
            t += 1
    assert np.all(out[t:] == 7.0) and (lse is None or np.all(lse[t:] == 7.0))


def queries(n, heads, seed):
    return bf16(np.random.default_rng(seed).standard_normal((n, heads, 512)))


@pytest.mark.parametrize("row0", [0, 1, 40, 63, 64, 65, 300, 1999])
@pytest.mark.parametrize("heads, page_rows, n, shape", [(64, 64, 1, "chain"), (64, 16, 9, "level"), (20, 32, 13, "random"),
                                                        (1, 128, 70, "level"), (33, 256, 6, "star"), (100, 16, 7, "level"),
                                                        (128, 64, 5, "forest"), (16, 64, 130, "random")])
def test_one_sequence(row0, heads, page_rows, n, shape):
    rng = np.random.default_rng(row0 + n)
    parent = D.tree(rng, n, shape)
    pool = Pool([row0 + n], page_rows, 200 + row0)
    q, qv = queries(n, heads, row0)
    got, lse = run(pool, [parent], [row0], q)
    check(pool, [parent], [row0], qv, got, lse)


@pytest.mark.parametrize("heads", [64, 20, 7, 72])
def test_ragged_drafts_windows_and_padding(heads):
    """Sequences without a token, with one and many nodes, empty and longer
    histories; each node a first position of its own: none, inside the history,
    inside its own line, beyond its own position; padding behind."""
    rng = np.random.default_rng(40)
    row0, nodes = [0, 700, 5, 1300, 64, 257, 128], [5, 0, 3, 21, 1, 12, 66]
    shapes = ["level", "chain", "star", "random", "chain", "forest", "random"]
    trees = [D.tree(rng, n, s) for n, s in zip(nodes, shapes)]
    pool = Pool([r + n for r, n in zip(row0, nodes)], 32, 41)
    n = sum(nodes)
    begin = np.empty(n, dtype=np.int64)
    t = 0
    for s, parent in enumerate(trees):
        for j in range(nodes[s]):
            place = row0[s] + len(D.line(parent, j)) - 1
            begin[t] = rng.choice([-7, 0, rng.integers(0, row0[s] + 1), max(0, row0[s] - 3), row0[s] + 1, place, place + 1,
                                   place + 100, 1 << 62])
            t += 1
    q, qv = queries(n + 3, heads, 42)
    got, lse = run(pool, trees, row0, q, begin=np.append(begin, [5, -9, 1 << 50]), pad=24)
    check(pool, trees, row0, qv, got, lse, begin)
    got2, none = run(pool, trees, row0, q, begin=np.append(begin, [5, -9, 1 << 50]), lse=False)
    assert none is None and np.array_equal(got, got2)


@pytest.mark.parametrize("heads", [64, 8])
def test_long_histories(heads):
    """Histories that are split over many workers, the draft behind the last
    part; a second call gives the same bits."""
    rng = np.random.default_rng(43)
    row0, nodes = [9000, 130, 20010, 77], [6, 9, 3, 70]
    trees = [D.tree(rng, n, "level") for n in nodes]
    pool = Pool([r + n for r, n in zip(row0, nodes)], 128, 44)
    q, qv = queries(sum(nodes), heads, 45)
    got, lse = run(pool, trees, row0, q)
    check(pool, trees, row0, qv, got, lse)
    again, lse2 = run(pool, trees, row0, q)
    assert np.array_equal(got, again) and np.array_equal(lse.view(np.uint32), lse2.view(np.uint32))


@pytest.mark.parametrize("n, heads, shape", [(1024, 2, "random"), (1024, 16, "chain"), (1000, 1, "level"), (255, 64, "level")])
def test_large_drafts(n, heads, shape):
    """As many nodes as a draft has; lines over many words and tiles."""
    rng = np.random.default_rng(46)
    parent = D.tree(rng, n, shape)
    pool = Pool([100 + n], 64, 47)
    q, qv = queries(n, heads, 48)
    begin = np.array([0 if rng.integers(2) else 100 + max(0, len(D.line(parent, j)) - 40) for j in range(n)])
    got, lse = run(pool, [parent], [100], q, begin=begin)
    check(pool, [parent], [100], qv, got, lse, begin)


@pytest.mark.parametrize("heads", [64, 12, 1])
def test_rows_that_a_node_does_not_see_leave_its_bits(heads):
    """Other nodes' rows and the rows before a window: whatever bytes."""
    rng = np.random.default_rng(49)
    n, row0 = 11, 150
    parent = D.tree(rng, n, "random")
    q, _ = queries(n, heads, 50)
    begin = np.full(n, 30)
    pool = Pool([row0 + n], 16, 51)
    got, lse = run(pool, [parent], [row0], q, begin=begin)
    for node in (0, 4, 9, 10):
        other = Pool([row0 + n], 16, 51)
        seen = D.sees(parent, node, row0, 30)
        for r in sorted(set(range(row0 + n)) - set(seen)):
            page, at = other.table[0, r // 16], r % 16
            for first, size in ((at * 224, 224), (16 * 224 + at * 128, 128), (16 * 352 + at * 16, 16)):
                other.pages[page, first:first + size] = 0xFF
        got2, lse2 = run(other, [parent], [row0], q, begin=begin)
        assert np.array_equal(got[node], got2[node])
        assert np.array_equal(lse[node].view(np.uint32), lse2[node].view(np.uint32))


@pytest.mark.parametrize("heads", [64, 16])
def test_queries_that_are_not_finite_stay_in_their_node(heads):
    rng = np.random.default_rng(52)
    parent, row0, n = D.tree(rng, 9, "level"), 200, 9
    pool = Pool([row0 + n], 32, 53)
    q, _ = queries(n, heads, 54)
    got, lse = run(pool, [parent], [row0], q)
    odd = q.copy()
    odd[3, 0, 5] = 0x7FC0
    odd[6, heads - 1, 0] = 0x7F80
    got2, lse2 = run(pool, [parent], [row0], odd)
    hit = np.zeros((n, heads), dtype=bool)
    hit[3, 0] = hit[6, heads - 1] = True
    assert np.array_equal(got[~hit], got2[~hit]) and np.array_equal(lse[~hit].view(np.uint32), lse2[~hit].view(np.uint32))
    assert np.all(np.isnan(lse2[hit])) and np.all(np.isnan(C.bf16_decode(got2[hit])))


@pytest.mark.parametrize("heads", [64, 16, 128])
def test_parents_that_are_none_count_as_roots_and_are_flagged(heads):
    parent = [-1, 0, 2, 5, 1, -2, 3, 1 << 30, -(1 << 31), 4]
    clean = [-1, 0, -1, -1, 1, -1, 3, -1, -1, 4]
    pool = Pool([90 + 10], 16, 55)
    q, qv = queries(10, heads, 56)
    got, lse = run(pool, [parent], [90], q, status=-7)
    check(pool, [clean], [90], qv, got, lse)


@pytest.mark.parametrize("heads", [64, 16])
def test_nodes_without_a_place_are_zeros_and_flagged(heads):
    """A sequence that begins below row 0; nodes past the largest draft; their
    neighbours are as ever."""
    rng = np.random.default_rng(57)
    small, big = D.tree(rng, 7, "level"), D.tree(rng, 1030, "random")
    pool = Pool([50 + 7, 7, 20 + 1030], 64, 58)
    trees, row0 = [small, small, big], [50, -1, 20]
    q, qv = queries(7 + 7 + 1030, heads, 59)
    got, lse = run(pool, trees, row0, q, status=-7)
    out = C.bf16_decode(got).astype(np.float64)
    gone = np.zeros(len(out), dtype=bool)
    gone[7:14] = gone[-6:] = True
    assert np.all(out[gone] == 0) and np.all(np.isneginf(lse[gone]))
    for t in list(range(7)) + list(range(14, 14 + 1024, 31)):
        s, j = (0, t) if t < 7 else (2, t - 14)
        check_token(out[t], lse[t].astype(np.float64), pool.values(s, D.sees(trees[s], j, row0[s])), qv[t], SCALE)


@pytest.mark.parametrize("heads", [64, 16])
def test_rows_past_the_table_are_left_out_and_flagged(heads):
    """A draft that runs off its table's end, one that begins beyond it, and a
    page that is none; the lines' other rows count."""
    rng = np.random.default_rng(60)
    parent = D.tree(rng, 12, "chain")
    pool = Pool([128, 128, 128], 16, 61, extra_entries=0)
    q, qv = queries(36, heads, 62)
    row0 = [122, 1 << 40, 100]
    pool.table[2, 2] = pool.n_pages + 5
    got, lse = run(pool, [parent] * 3, row0, q, status=-7)
    out = C.bf16_decode(got).astype(np.float64)
    for t in range(36):
        s, j = divmod(t, 12)
        rows = [r for r in (D.sees(parent, j, min(row0[s], 128)) if s != 1 else range(128)) if r < 128]
        rows = [r for r in rows if not (s == 2 and 32 <= r < 48)]
        check_token(out[t], lse[t].astype(np.float64), pool.values(s, rows), qv[t], SCALE)


def test_rows_of_very_different_size():
    """Rows whose scales lie far apart on some lines only."""
    rng = np.random.default_rng(63)
    n, row0 = 14, 80
    parent = D.tree(rng, n, "random")
    x = rng.standard_normal((row0 + n, 512)).astype(np.float32)
    x[row0 + 5] *= 2.0 ** 40
    x[row0 + 9] *= 2.0 ** -60
    x[33] *= 2.0 ** -45
    for heads in (64, 16):
        pool = Pool([row0 + n], 32, 64, x=[x])
        q, qv = queries(n, heads, 65)
        got, lse = run(pool, [parent], [row0], q, scale=1e-3)
        check(pool, [parent], [row0], qv, got, lse, scale=1e-3)


def test_a_chain_is_the_causal_attention():
    """parent[j] = j - 1: what ds4x_paged_attn gives for rising row_end."""
    B = require_gpu()
    n, row0, heads = 9, 777, 64
    pool = Pool([row0 + n], 64, 66)
    q, qv = queries(n, heads, 67)
    got, lse = run(pool, [D.tree(None, n, "chain")], [row0], q)
    out = torch.empty((n, heads, 512), dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty((n, heads), device="cuda")
    B.ds4x_paged_attn(dev(pool.pages), 64, dev(pool.table), dev(np.array([0, n], np.int32)),
                      dev(np.arange(row0 + 1, row0 + n + 1)), bf16_dev(q), SCALE, out, l2, new_ws(B.ds4x_paged_attn_workspace()))
    for o, l in ((got, lse), (bf16_host_bits(out), l2.cpu().numpy())):
        check(pool, [D.tree(None, n, "chain")], [row0], qv, o, l)


@pytest.mark.parametrize("heads", [64, 16])
def test_captured_call_follows_its_inputs_on_another_stream(heads):
    B = require_gpu()
    rng = np.random.default_rng(68)
    shapes = [([30, 200], [7, 5]), ([90, 0], [2, 10]), ([10, 211], [12, 0])]
    n = 12
    pool = Pool([240, 240], 16, 69)
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
    for k, (before, nodes) in enumerate(shapes):
        trees = [D.tree(rng, m, "random") if m else [] for m in nodes]
        bits, qv = queries(n, heads, 70 + k)
        cu.copy_(torch.tensor([0, nodes[0], sum(nodes)], dtype=torch.int32))
        parent.copy_(torch.tensor([p for t in trees for p in t], dtype=torch.int32))
        row0.copy_(torch.tensor(before))
        q.copy_(bf16_dev(bits))
        graph.replay()
        torch.cuda.synchronize()
        check(pool, trees, before, qv, bf16_host_bits(out), lse.cpu().numpy())
    assert B.ds4x_workspace_status(ws) == 0


def test_many_sequences():
    """More sequences than the plan holds at once, of one to three nodes."""
    rng = np.random.default_rng(71)
    S = 5000
    nodes = rng.integers(0, 4, S)
    trees = [D.tree(rng, int(m), "random") if m else [] for m in nodes]
    row0 = rng.integers(0, 20, S)
    pool = Pool([int(r + m) for r, m in zip(row0, nodes)], 16, 72)
    q, qv = queries(int(nodes.sum()), 4, 73)
    got, lse = run(pool, trees, row0, q)
    check(pool, trees, row0, qv, got, lse)


@pytest.mark.parametrize("heads", [1, 40])
def test_as_many_tokens_as_a_call_takes(heads):
    """65,535 nodes of 70 sequences, more units than the plan holds in shared
    memory; some checked."""
    rng = np.random.default_rng(74)
    nodes = [936] * 69 + [65535 - 69 * 936]
    trees = [D.tree(rng, n, "level") for n in nodes]
    row0 = rng.integers(0, 90, 70)
    pool = Pool([int(r + n) for r, n in zip(row0, nodes)], 64, 75)
    q, qv = queries(65535, heads, 76)
    got, lse = run(pool, trees, row0, q)
    out = C.bf16_decode(got[::311]).astype(np.float64)
    for k, t in enumerate(range(0, 65535, 311)):
        s, j = divmod(t, 936)
        check_token(out[k], lse[t].astype(np.float64), pool.values(s, D.sees(trees[s], j, int(row0[s]))), qv[t], SCALE)


@pytest.mark.parametrize("heads", [20, 64])
def test_wide_tables(heads):
    """A table wider than the rows need changes how work is split only where
    the call has few tiles; the values are within the bounds all the same."""
    rng = np.random.default_rng(77)
    nodes, row0 = [9, 4, 30], [500, 3, 1200]
    trees = [D.tree(rng, n, "random") for n in nodes]
    rows = [r + n for r, n in zip(row0, nodes)]
    q, qv = queries(sum(nodes), heads, 78)
    for extra in (0, 400):
        pool = Pool(rows, 32, 79, extra_entries=extra)
        got, lse = run(pool, trees, row0, q)
        check(pool, trees, row0, qv, got, lse)


@pytest.mark.parametrize("heads", [1, 2, 3, 5])
@pytest.mark.parametrize("rows", [150, 9000])
def test_few_heads_and_many_nodes_a_unit(heads, rows):
    """Up to 32 nodes share a unit where heads are few: over few and many tiles,
    with windows that differ by node and rows that some nodes do not see."""
    rng = np.random.default_rng(80 + heads)
    nodes = [70, 33, 0, 90, 31]
    row0 = [rows, rows // 3, 5, rows - 40, 1]
    trees = [D.tree(rng, n, s) if n else [] for n, s in zip(nodes, ["random", "level", "chain", "level", "forest"])]
    pool = Pool([r + n for r, n in zip(row0, nodes)], 16, 81)
    n = sum(nodes)
    begin = np.empty(n, dtype=np.int64)
    t = 0
    for s, parent in enumerate(trees):
        for j in range(len(parent)):
            place = row0[s] + len(D.line(parent, j)) - 1
            begin[t] = rng.choice([0, max(0, row0[s] - 70), row0[s] + 2, place, place + 1])
            t += 1
    q, qv = queries(n, heads, 82)
    got, lse = run(pool, trees, row0, q, begin=begin)
    check(pool, trees, row0, qv, got, lse, begin)
    got, lse = run(pool, trees, row0, q)
    check(pool, trees, row0, qv, got, lse)
