"""The paged cache's oracle against brute force and closed forms."""

import numpy as np
import pytest
import torch

from oracle import codecs as C
from oracle import paged as O
from oracle.attention import dense_attn_decode
from paged_path import Pool, bf16, check_token


def test_codes_and_scales_are_the_indexer_rows_rule():
    """Away from the exponent limits a 32-value block is packed as the
    indexer row's blocks are."""
    x = np.random.default_rng(1).standard_normal((50, 512)).astype(np.float32) * 3
    code, _, scales = O.quantise(x)
    rows = C.pack_idx_rows(np.ascontiguousarray(x[:, :128])).reshape(50, 68)
    assert np.array_equal(code[:, 0:128:2] | (code[:, 1:128:2] << 4), rows[:, :64])
    assert np.array_equal(scales[:, :4], rows[:, 64:])


@pytest.mark.parametrize("mag", [0.0, 2.0 ** -120, 6 * 2.0 ** -96, 1.0, 6.0, 6.0000005, 2.0 ** 90, 6 * 2.0 ** 96, 2.0 ** 110])
def test_scale_limits(mag):
    x = np.zeros((1, 512), dtype=np.float32)
    x[0, 5] = -mag
    code, tail, scales = O.quantise(x)
    e = int(scales[0, 0]) - 127
    assert -96 <= e <= 96 and scales[0, 14] == scales[0, :14].max()
    if e > -96:
        assert mag > 6 * 2.0 ** (e - 1)
    if e < 96:
        assert mag <= 6 * 2.0 ** e
    assert np.all(scales[0, 1:14] == 31) and scales[0, 15] == 0
    v = O.values(code, tail, scales)
    assert abs(v[0, 5] + min(mag, 6 * 2.0 ** 96)) <= 2.0 ** e


def test_rotation_is_torch_complex_product():
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((9, 512)), rng.integers(-5000, 1 << 20, 9)
    f = 10000.0 ** (-np.arange(32) / 32)
    z = torch.polar(torch.ones(9, 32, dtype=torch.float64), torch.tensor(pos[:, None] * f))
    for halves in (False, True):
        t = torch.tensor(x[:, 448:])
        t = torch.complex(t[:, :32], t[:, 32:]) if halves else torch.complex(t[:, 0::2], t[:, 1::2])
        t = torch.view_as_real(t * z)
        want = torch.cat([t[..., 0], t[..., 1]], 1) if halves else t.flatten(1)
        got = O.rotate(x, pos, f, halves)
        assert np.allclose(got[:, 448:], want.numpy(), atol=1e-9) and np.array_equal(got[:, :448], x[:, :448])


def test_write_and_read_are_inverse_and_place_by_the_table():
    pool = Pool([37, 0, 16], 16, 3)
    for s, r in enumerate(pool.rows):
        assert np.array_equal(pool.values(s, np.arange(r)), O.values(*O.quantise(pool.x[s])) if r else np.zeros((0, 512)))
    # planes at fixed places
    p, row = pool.pages[pool.table[0, 1]], O.quantise(pool.x[0][16 + 3:16 + 4])
    assert p[3 * 224] == row[0][0, 0] | row[0][0, 1] << 4
    assert np.array_equal(p[16 * 224 + 3 * 128:16 * 224 + 4 * 128].view("<f2"), row[1][0])
    assert np.array_equal(p[16 * 352 + 3 * 16:16 * 352 + 4 * 16], row[2][0])


def test_attention_is_the_dense_attention_of_the_framework():
    """Rows that both formats hold exactly: the two oracles agree."""
    rng = np.random.default_rng(4)
    x = (rng.choice(O.GRID, (40, 512)) * rng.choice([-1.0, 1.0], (40, 512))).astype(np.float32)
    x[:, 0:448:32] = 6.0  # the same scale in every block
    bits, q = bf16(rng.standard_normal((64, 512)))
    v = O.values(*O.quantise(x))
    assert np.array_equal(v, x)
    out, lse, _, _ = O.attention(v, q, 0.05)
    _, exact, ref_lse = dense_attn_decode(C.pack_kv_rows(x), 40, bits, 0.05)
    assert np.allclose(out, exact, atol=1e-12) and np.allclose(lse, ref_lse, atol=1e-12)
    check_token(bf16(out)[1], lse, v, q, 0.05)
    check_token(np.zeros((3, 512)), np.full(3, -np.inf), v[:0], q[:3], 0.05)
    with pytest.raises(AssertionError):
        check_token(bf16(out * 1.02)[1], lse, v, q, 0.05)
