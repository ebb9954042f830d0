"""ds4x_paged_append at its edges: values that are not finite."""

import numpy as np
import pytest
import torch

from gpu_path import require_gpu
from paged_path import Pool, bf16
from test_gpu_paged_rows import expected, run_append

pytestmark = pytest.mark.gpu
BIG = np.finfo(np.float32).max


def finite(x):
    return np.where(np.isnan(x), 0.0, np.clip(x, -BIG, BIG)).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_finite_are_flagged_and_defined(dtype, bad):
    """NaN as zero, infinities as the largest floats, wherever they stand; the rows and
    blocks beside them as ever."""
    require_gpu()
    rng = np.random.default_rng(40)
    at = [0, 31, 32, 200, 255, 256, 440, 447, 448, 449, 480, 500, 511]
    n = 3 * len(at) + 4
    x = bf16(rng.standard_normal((n, 512)))[1].astype(np.float32)
    for i, c in enumerate(at):
        x[3 * i, c] = bad
    x[n - 3, :] = bad
    x[n - 2, 448:], x[n - 2, 10:500:7] = bad, -bad
    pool = Pool([n], 16, 41)
    pages, back, _ = run_append(pool, [n], [0], x, dtype=dtype, status=-7)
    want, vals = expected(pool, [n], [0], finite(x))
    assert np.array_equal(pages, want) and np.array_equal(back.astype(np.float64), vals) and np.isfinite(back).all()
    for t in (torch.float32, torch.bfloat16):  # none in the rows that are placed: no flag
        clean = np.concatenate([finite(x[1:2]), np.full((3, 512), bad, np.float32)])
        run_append(pool, [1], [5], clean, dtype=t)


@pytest.mark.parametrize("style", [0, 1])
def test_rotated_values_that_are_not_finite(style):
    """A pair with NaN is zeros; a pair that turns past the largest float saturates;
    the other pairs and rows are what they are without."""
    n = 6
    rng = np.random.default_rng(42)
    x = rng.standard_normal((n, 512)).astype(np.float32)
    i = np.arange(32)
    a, b = (448 + i, 480 + i) if style else (448 + 2 * i, 449 + 2 * i)
    clean = x.copy()
    x[1, a[3]], x[2, b[9]] = np.nan, np.inf
    x[3, a[7]] = x[3, b[7]] = 3.2e38  # at an eighth of a turn: 0 and 4.5e38
    freq = np.full(32, np.pi / 4, dtype=np.float32)
    pool = Pool([n], 64, 43)
    pos = np.ones(n, dtype=np.int64)
    _, good, _ = run_append(pool, [n], [0], clean, pos=pos, freq=freq, style=style)
    _, got, _ = run_append(pool, [n], [0], x, pos=pos, freq=freq, style=style, status=-7)
    assert np.isfinite(got).all()
    same = [0, 4, 5]
    assert np.array_equal(got[same], good[same]) and np.array_equal(got[:, :448], good[:, :448])
    assert got[1, a[3]] == 0 and got[1, b[3]] == 0
    rest = np.setdiff1d(np.arange(448, 512), [a[3], b[3]])
    assert np.array_equal(got[1, rest], good[1, rest])
    # (infinity times a cosine and a sine of one sign)
    top = 65504 * 2.0 ** 96
    assert got[2, a[9]] == -top and got[2, b[9]] == top
    assert got[3, b[7]] == top
