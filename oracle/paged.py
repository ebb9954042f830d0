"""The paged 4-bit cache in plain float64: a row's quantiser, its packing into
pages, the position rotation and attention over rows.

A row is 448 E2M1 values with a power-of-two scale per 32 and 64 FP16 values
with one scale, the row's largest; pages are three planes (codes, RoPE values,
scales) as include/ds4x.h lays them out.  Written from that description; the
library has no code in common with it.
"""

import numpy as np

DIM, NOPE, TAIL, GROUP, ROW_BYTES = 512, 448, 64, 32, 368
E_MIN, E_MAX = -96, 96
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exponent(amax, top):
    """The least e in [E_MIN, E_MAX] with amax <= top 2^e, by trying them all."""
    e = np.full(np.shape(amax), E_MAX)
    for k in range(E_MAX - 1, E_MIN - 1, -1):
        e = np.where(amax <= top * 2.0 ** k, k, e)
    return e


def rotate(x, pos, inv_freq, halves):
    """The RoPE part of rows x [n, 512] turned at positions pos [n]."""
    x = np.array(x, dtype=np.float64)
    # whole turns dropped in extended precision before cos and sin
    two_pi = np.longdouble(2) * np.arctan2(np.longdouble(0), np.longdouble(-1))
    turn = np.asarray(pos, dtype=np.longdouble)[:, None] * np.asarray(inv_freq, dtype=np.longdouble)[None, :]
    ang = np.asarray(np.fmod(turn, two_pi), dtype=np.float64)
    i = np.arange(TAIL // 2)
    a, b = (NOPE + i, NOPE + 32 + i) if halves else (NOPE + 2 * i, NOPE + 2 * i + 1)
    u, v = x[:, a].copy(), x[:, b].copy()
    x[:, a], x[:, b] = u * np.cos(ang) - v * np.sin(ang), u * np.sin(ang) + v * np.cos(ang)
    return x


def quantise(x):
    """x [n, 512] -> (codes u8 [n, 448], tail f16 [n, 64], scale bytes u8 [n, 16])."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[0]
    blocks = x[:, :NOPE].reshape(n, NOPE // GROUP, GROUP)
    e = exponent(np.abs(blocks).max(axis=2), 6.0)
    y = np.minimum(np.abs(blocks) / 2.0 ** e[:, :, None], 6.0)
    d = np.abs(y[..., None] - GRID)
    # nearest, of two as near the even code
    rank = np.where(d == d.min(axis=3, keepdims=True), np.arange(8) + 16 * (np.arange(8) % 2), 99)
    code = (rank.min(axis=3) % 16 + 8 * np.signbit(blocks)).astype(np.uint8).reshape(n, NOPE)
    top = np.maximum(e.max(axis=1), exponent(np.abs(x[:, NOPE:]).max(axis=1), 8.0))
    tail = np.clip(x[:, NOPE:] / 2.0 ** top[:, None], -65504, 65504).astype(np.float16)
    scales = np.zeros((n, 16), dtype=np.uint8)
    scales[:, :14] = e + 127
    scales[:, 14] = top + 127
    return code, tail, scales


def values(code, tail, scales):
    """The float64 rows that quantised rows stand for."""
    s = 2.0 ** (scales[:, :15].astype(np.float64) - 127)
    mag = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    return np.concatenate([mag * np.repeat(s[:, :14], GROUP, axis=1), tail.astype(np.float64) * s[:, 14:]], axis=1)


def write(pages, page_rows, page, at, code, tail, scales):
    """Places rows at (page[i], at[i]) of pages u8 [n_pages, page_rows * 368]."""
    R = page_rows
    for i in range(len(page)):
        p = pages[page[i]]
        p[at[i] * 224:at[i] * 224 + 224] = code[i, 0::2] | (code[i, 1::2] << 4)
        o = R * 224 + at[i] * 128
        p[o:o + 128] = tail[i].astype("<f2").view(np.uint8)
        o = R * 352 + at[i] * 16
        p[o:o + 16] = scales[i]


def read(pages, page_rows, page, at):
    """The float64 rows at (page[i], at[i])."""
    R = page_rows
    page, at = np.asarray(page, dtype=np.int64), np.asarray(at, dtype=np.int64)
    n = len(page)
    byte = lambda first, m: pages[page[:, None], first[:, None] + np.arange(m)]  # noqa: E731
    c = byte(at * 224, 224)
    code = np.empty((n, NOPE), dtype=np.uint8)
    code[:, 0::2], code[:, 1::2] = c & 15, c >> 4
    tail = np.ascontiguousarray(byte(R * 224 + at * 128, 128)).view("<f2").reshape(n, TAIL)
    return values(code, tail, byte(R * 352 + at * 16, 16))


def attention(v, q, scale):
    """q [heads, 512] over rows v [n, 512]: (out, lse, p, logits); zeros and
    -inf for no rows."""
    H = q.shape[0]
    if len(v) == 0:
        return np.zeros((H, DIM)), np.full(H, -np.inf), np.zeros((H, 0)), np.zeros((H, 0))
    l = (q @ v.T) * scale
    m = l.max(axis=1, keepdims=True)
    p = np.exp(l - m)
    z = p.sum(axis=1, keepdims=True)
    p /= z
    return p @ v, (m + np.log(z))[:, 0], p, l
