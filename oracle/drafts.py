"""Checking drafted tokens in plain float64: what a draft's nodes see, the walk
that decides which of them stand, and the rows that are kept.

Written from the description in include/ds4x.h; the library has no code in
common with it.
"""

import numpy as np


def line(parent, node):
    """The nodes from a root to `node`."""
    out = [node]
    while parent[out[-1]] >= 0:
        out.append(parent[out[-1]])
    return out[::-1]


def sees(parent, node, row0, begin=0):
    """The rows that a node sees, ascending: those before the draft and its
    line's, from position `begin` on."""
    own = line(parent, node)
    return list(range(max(0, begin), row0)) + [row0 + a for d, a in enumerate(own) if row0 + d >= begin]


def verify(parent, tokens, target, draft, u):
    """One sequence's walk: (path, new tokens, how near a decision was to its
    border, relative to what it was compared with)."""
    clean = lambda p: np.where(p > 0, p, 0.0)  # noqa: E731  (negative and NaN are zero)
    target = clean(np.asarray(target, dtype=np.float64))
    draft = None if draft is None else clean(np.asarray(draft, dtype=np.float64))
    path, out, near = [0], [], np.inf
    vocab = target.shape[1]
    while True:
        cur = path[-1]
        p, mass = target[cur].copy(), 1.0
        took = None
        for j in range(cur + 1, len(parent)):
            if parent[j] != cur:
                continue
            x = tokens[j]
            inside = 0 <= x < vocab
            w = p[x] if inside else 0.0
            q = 1.0 if draft is None else draft[cur][x] if inside else 0.0
            bar = float(u[j]) * q * mass
            if inside and (bar > 0 or w > 0):  # (two zeros are exact)
                near = min(near, abs(bar - w) / max(bar, w, 1e-300))
            if bar < w:
                took = j
                break
            if draft is None:
                mass -= w
                if inside:
                    p[x] = 0.0
            else:
                # p / mass is the renormalised rest
                p = np.maximum(p - mass * draft[cur], 0.0)
                mass = p.sum()
        if took is None:
            c = np.cumsum(p)
            if not c[-1] > 0 and cur in parent[cur + 1:]:
                # rounded rows left nothing: the target's row as it is, if the draft's is one beside it
                whole, drawn = np.cumsum(target[cur]), 0.0 if draft is None else draft[cur].sum()
                if 2 * whole[-1] > drawn:
                    p, c = target[cur], whole
            if not c[-1] > 0:
                out.append(-1)
            else:
                want = float(u[0]) * c[-1]
                y = int(np.searchsorted(c, want, side="right"))
                while p[min(y, vocab - 1)] == 0 or y >= vocab:
                    y -= 1
                out.append(y)
                edge = np.abs(c[p > 0] - want).min() if want > 0 else np.inf
                near = min(near, edge / c[-1])
            return path, out, near
        path.append(took)
        out.append(int(tokens[took]))


def keep(rows, row0, path):
    """A sequence's rows (a list) after row row0 + path[i] moved to row0 + i."""
    new = list(rows)
    for i, j in enumerate(path):
        new[row0 + i] = rows[row0 + j]
    return new


# ---- drafts to test with ----------------------------------------------------------

def tree(rng, n, shape):
    """Parents of n nodes: "chain", "star" (all follow node 0), "level" (two to
    four children a node), "random", or "forest" (several roots)."""
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "star":
        return [-1] + [0] * (n - 1)
    if shape == "level":
        return [-1] + [int(rng.integers((j - 1) // 4, (j - 1) // 2 + 1)) for j in range(1, n)]
    low = -1 if shape == "forest" else 0
    return [-1] + [int(rng.integers(low, j)) for j in range(1, n)]
