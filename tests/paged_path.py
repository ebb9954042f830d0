"""Helpers of the paged cache's tests: a pool with ragged sequences on numpy
and on the GPU, and the bounds that the attention's outputs keep.

Bounds, per output element o = sum_j p_j v_j (row j's largest exponent E_j):
  - the bf16 output is off by half a step: 2^-8 |o|;
  - a softmax weight enters the second product as fp16 relative to the largest
    one: half a step, 2^-11, while it is above 2^-14 of it, else 2^-25 of it.
    The rows enter relative to 2^E_j, at most 8 in size, and the weight carries
    2^E_j, so the second kind is at most 8 * 2^-25 * max_j(p_j 2^E_j) a row;
  - a row's value whose scale lies 2^14 or more below its row's largest rounds
    at 2^-25 2^E_j (half of the least fp16 step);
  - a logit is a sum of 512 products of exact operands in fp32: 32 steps of 16
    products, each step off by at most 2^-23 of the sum of their sizes (a
    truncating adder), and its scaling and exponential by 2^-21 of
    max(1, |l|): dl; p is then off by 2 dl relative (numerator and sum);
  - the rest (fp32 sums over tiles and parts) by 2^-18 relative.
"""

import numpy as np

from oracle import paged as O


class Pool:
    """n_seqs sequences of rows[s] rows in a shuffled pool of pages filled with
    bytes that would show (NaN in the RoPE values, scale 255)."""

    def __init__(self, rows, page_rows, seed, x=None, extra_pages=2, extra_entries=1, fill=0xFF):
        self.rng = np.random.default_rng(seed)
        self.R, self.rows = page_rows, list(rows)
        need = [max(1, -(-r // page_rows)) for r in rows]
        self.n_pages = sum(need) + extra_pages
        order = self.rng.permutation(self.n_pages)
        self.table = np.full((len(rows), max(need) + extra_entries), -7, dtype=np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            at += k
        self.pages = np.full((self.n_pages, page_rows * O.ROW_BYTES), fill, dtype=np.uint8)
        if x is None:
            x = [self.rng.standard_normal((r, O.DIM)).astype(np.float32) for r in rows]
        self.x = x
        for s, r in enumerate(rows):
            if r:
                j = np.arange(r)
                O.write(self.pages, page_rows, self.table[s, j // page_rows], j % page_rows, *O.quantise(x[s]))

    def values(self, s, rows):
        rows = np.asarray(rows, dtype=np.int64)
        return O.read(self.pages, self.R, self.table[s, rows // self.R], rows % self.R)


def bf16(x):
    """float array -> (bf16 bits, the values they stand for)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    bits = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return bits, (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def check_token(out, lse, v, q, scale):
    """One token's out [heads, 512] and lse [heads] (float64) over rows v."""
    ref, ref_lse, p, l = O.attention(v, q, scale)
    if len(v) == 0:
        assert np.all(out == 0)
        assert lse is None or np.all(np.isneginf(lse))
        return
    big = np.exp2(np.ceil(np.log2(np.maximum(np.abs(v).max(axis=1), 2.0 ** -99))))  # >= 2^E_j / 8
    dl = (32 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(v).T)).max(axis=1) + 2.0 ** -21 * np.maximum(1, np.abs(l).max(axis=1))
    small = 8 * (8 * 2.0 ** -25 * len(v) * (p * big).max(axis=1) + 2.0 ** -25 * (p @ big))
    size = p @ np.abs(v)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * dl[:, None] + 2.0 ** -18) * size + small[:, None]
    bad = ~(np.abs(out - ref) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, worst {np.abs(out - ref).max()} at tolerance "
                           f"{tol.flat[np.abs(out - ref).argmax()]}")
    if lse is not None:
        assert np.all(np.abs(lse - ref_lse) <= dl + 2.0 ** -18 + 2.0 ** -22 * np.abs(ref_lse))
