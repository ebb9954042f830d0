"""ds4x_paged_keep: bytes of the whole pool against the same moves on numpy."""

import numpy as np
import pytest
import torch

from gpu_path import dev, new_ws, require_gpu
from oracle import drafts as D
from paged_path import Pool

pytestmark = pytest.mark.gpu


def bytes_of(pool, s, r):
    R, page, at = pool.R, pool.table[s, r // pool.R], r % pool.R
    return [(page, slice(at * 224, at * 224 + 224)), (page, slice(R * 224 + at * 128, R * 224 + at * 128 + 128)),
            (page, slice(R * 352 + at * 16, R * 352 + at * 16 + 16))]


def moved(pool, row0, paths):
    """The pool's bytes after every sequence's moves."""
    pages = pool.pages.copy()
    for s, path in enumerate(paths):
        for i, j in enumerate(path):
            for a, b in zip(bytes_of(pool, s, row0[s] + i), bytes_of(pool, s, row0[s] + j)):
                pages[a] = pool.pages[b]
    return pages


def run(pool, nodes, row0, paths, n_path=None, status=0, extra=0, stream=None):
    B = require_gpu()
    n = sum(nodes)
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    path = np.full(n + extra, -1, dtype=np.int32)
    for s, p in enumerate(paths):
        path[cu[s]:cu[s] + len(p)] = p
    pages, ws = dev(pool.pages), new_ws(256)
    torch.cuda.synchronize()
    B.ds4x_paged_keep(pages, pool.R, dev(pool.table), dev(cu), dev(np.asarray(row0, dtype=np.int64)), dev(path),
                      dev(np.asarray([len(p) for p in paths] if n_path is None else n_path, dtype=np.int32)), ws, stream=stream)
    torch.cuda.synchronize()
    assert B.ds4x_workspace_status(ws) == status
    return pages.cpu().numpy()


def random_path(rng, n, k):
    return [0] + sorted(rng.choice(np.arange(1, n), size=k - 1, replace=False).tolist()) if n else []


@pytest.mark.parametrize("page_rows", [16, 32, 64, 128, 256])
def test_lines_of_ragged_drafts(page_rows):
    rng = np.random.default_rng(90 + page_rows)
    nodes, row0 = [6, 1, 0, 40, 130, 17, 256], [0, 15, 33, 250, 7, 16, 1000]
    paths = [random_path(rng, n, int(rng.integers(1, n + 1)) if n else 0) for n in nodes]
    pool = Pool([r + n for r, n in zip(row0, nodes)], page_rows, 91)
    assert np.array_equal(run(pool, nodes, row0, paths, extra=3), moved(pool, row0, paths))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 65, 500, 999, 1000])
def test_long_lines_over_themselves(k):
    """Moves whose places are other moves' sources, over many rounds."""
    rng = np.random.default_rng(k)
    for path in (random_path(rng, 1000, k), [0] + list(range(1001 - k, 1000)), list(range(k))):
        pool = Pool([13 + 1000], 64, 92)
        assert np.array_equal(run(pool, [1000], [13], [path]), moved(pool, [13], [path]))


def test_drafts_longer_than_the_other_calls_take():
    rng = np.random.default_rng(93)
    path = random_path(rng, 5000, 3000)
    pool = Pool([5000], 128, 94)
    assert np.array_equal(run(pool, [5000], [0], [path]), moved(pool, [0], [path]))


def test_entries_outside_are_left_out_and_flagged():
    pool = Pool([50, 50], 16, 95)
    paths, row0 = [[0, 3, 1, 5, 30, -1, 7], [0, 2]], [20, 20]
    got = run(pool, [12, 12], row0, paths, status=-7)
    assert np.array_equal(got, moved(pool, row0, [[0, 3, 2, 5, 4, 5, 7], [0, 2]]))


def test_counts_outside_are_clipped():
    pool = Pool([50, 50, 50], 16, 96)
    row0 = [20, 20, 20]
    got = run(pool, [3, 3, 3], row0, [[0, 2, 2], [0, 2, 2], [0, 2, 2]], n_path=[9, -4, 0], status=-7)
    assert np.array_equal(got, moved(pool, row0, [[0, 2, 2], [], []]))


def test_rows_without_a_place_stay_and_are_flagged():
    pool = Pool([64, 64, 64], 16, 97, extra_entries=0)
    keep_table = pool.table.copy()
    pool.table[1, 2] = -1
    row0, paths = [58, 30, -2], [[0, 2, 4, 7], [0, 1, 5, 9], [0, 1, 4]]
    got = run(pool, [10, 20, 6], row0, paths, status=-7)
    # past the table: 58 + 7; in the page that is none: rows 32..47; below row 0: place -2, -1
    pool.table = keep_table
    assert np.array_equal(got, expected_unplaced(pool, row0, paths))


def expected_unplaced(pool, row0, paths):
    placed = lambda s, r: 0 <= r < 64 and not (s == 1 and 32 <= r < 48)  # noqa: E731
    pages = pool.pages.copy()
    for s, path in enumerate(paths):
        for i, j in enumerate(path):
            if placed(s, row0[s] + i) and placed(s, row0[s] + j):
                for a, b in zip(bytes_of(pool, s, row0[s] + i), bytes_of(pool, s, row0[s] + j)):
                    pages[a] = pool.pages[b]
    return pages


def test_thousands_of_sequences_on_another_stream():
    rng = np.random.default_rng(98)
    nodes = rng.integers(0, 6, 3000).tolist()
    row0 = rng.integers(0, 20, 3000).tolist()
    paths = [random_path(rng, n, int(rng.integers(1, n + 1))) if n else [] for n in nodes]
    pool = Pool([r + n for r, n in zip(row0, nodes)], 16, 99)
    assert np.array_equal(run(pool, nodes, row0, paths, stream=torch.cuda.Stream()), moved(pool, row0, paths))


def test_the_oracle_moves_the_same_rows():
    pool = Pool([30], 16, 100)
    rows = [pool.values(0, [r]).tobytes() for r in range(30)]
    path = [0, 2, 5, 6, 9]
    pool.pages = run(pool, [10], [12], [path])
    assert [pool.values(0, [r]).tobytes() for r in range(30)] == D.keep(rows, 12, path)
