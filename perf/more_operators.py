"""What is measured of the operators that check drafted tokens over the paged
4-bit cache, and their plain forms.

A step of a server that drafts: each sequence's call tokens are the nodes of a
tree.  Node 0 is the sequence's newest token, the others were drafted to follow
their parent; their rows have been appended to the sequence's pages, node j's
as row row0 + j.

  tree     attention of each node over the rows before the tree and over its
           own line of ancestors
  verify   which drafted tokens the target's probabilities accept, by given
           random numbers, and the token that follows them
  keep     the accepted line's rows moved up behind row0; the sequence's new
           rows are read back

The cache's rows are as perf/operators.py describes them: 512 values, 448 in
E2M1 with a power-of-two scale per 32, 64 in FP16 with a scale of their own, in
pages of three planes.  Nodes are ragged over the sequences: sequence s has the
tokens cu[s] .. cu[s + 1] - 1 of a call.
"""

import math
import random

import torch

own = False

DIM, NOPE, TAIL, GROUP = 512, 448, 64, 32
CODES, TAILS, SCALES = NOPE // 2, TAIL * 2, 16
ROW = CODES + TAILS + SCALES
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E_MIN, E_MAX = -96, 96
SCALE = 1.0 / math.sqrt(DIM)


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # a small draft over a short history, one session
        dict(name="tree_short", op="tree", seqs=1, nodes=6, shape="level", uneven=False, heads=64, rows=777, ragged=0, window=0, page_rows=32, salt=1),
        # a draft of 26 nodes over every compressed row of a million-token context at ratio 128
        dict(name="tree_8192", op="tree", seqs=1, nodes=26, shape="level", uneven=False, heads=64, rows=8192, ragged=0, window=0, page_rows=64, salt=2),
        # 24 sessions of few heads with small uneven drafts, ragged from an empty history, a sliding window
        dict(name="tree_window", op="tree", seqs=24, nodes=13, shape="line", uneven=True, heads=20, rows=9001, ragged=1, window=4999, page_rows=16, salt=3),
        # one session, a wide draft
        dict(name="tree_wide", op="tree", seqs=1, nodes=255, shape="level", uneven=False, heads=64, rows=32768, ragged=0, window=0, page_rows=128, salt=4),
        # 16 sessions of 8192 to 65536 rows, 32 nodes each
        dict(name="tree_sessions", op="tree", seqs=16, nodes=32, shape="line", uneven=False, heads=64, rows=65536, ragged=8192, window=0, page_rows=64, salt=5),
        # one session's chain of five sampled drafts
        dict(name="verify_one", op="verify", seqs=1, nodes=6, shape="chain", uneven=False, vocab=131072, dtype="f32", draft=True, cut=False, salt=6),
        # 61 sessions, several sampled children a node, an odd vocabulary, probabilities of a top-p sampler (most are zero)
        dict(name="verify_sampled", op="verify", seqs=61, nodes=9, shape="level", uneven=True, vocab=50257, dtype="f32", draft=True, cut=True, salt=7),
        # 16 sessions, trees of the draft's likeliest tokens, bf16
        dict(name="verify_tree", op="verify", seqs=16, nodes=32, shape="level", uneven=False, vocab=131072, dtype="bf16", draft=False, cut=False, salt=8),
        # 256 sessions' chains of seven sampled drafts
        dict(name="verify_chains", op="verify", seqs=256, nodes=8, shape="chain", uneven=False, vocab=131072, dtype="f32", draft=True, cut=False, salt=9),
        # one session's accepted line
        dict(name="keep_one", op="keep", seqs=1, nodes=26, shape="line", uneven=False, rows=8192, page_rows=64, salt=10),
        # 64 sessions' accepted lines
        dict(name="keep_batch", op="keep", seqs=64, nodes=32, shape="line", uneven=True, rows=4096, page_rows=16, salt=11),
        # long drafts, as text that repeats gives them
        dict(name="keep_long", op="keep", seqs=16, nodes=1000, shape="line", uneven=True, rows=4096, page_rows=64, salt=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "verify", "verify", "keep"))
    salt = rng.randrange(1 << 30)
    page_rows = rng.choice((16, 32, 64, 128, 256))
    if op == "tree":
        heads = rng.choice((64, 64, 64, 128, 1, 8, 16, 20, 33, 48, 100))
        nodes = _log(rng, 1, 256)
        seqs = _log(rng, 1, max(1, min(24, 1024 // nodes)))
        rows = _log(rng, 1, min(65536, 1048576 // seqs, 18000000 // (seqs * nodes * max(heads, 64) // 64)))
        return dict(op=op, seqs=seqs, nodes=nodes, shape=rng.choice(("level", "line", "chain")), uneven=rng.random() < 0.5, heads=heads, rows=rows,
                    ragged=rng.choice((0, 1, (rows + 1) // 2)), window=rng.choice((0, 0, 0, 2 + rows // 3, 3)), page_rows=page_rows, salt=salt)
    if op == "verify":
        nodes, vocab = _log(rng, 1, 64), _log(rng, 500, 200000)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(256, 1024 * 131072 // (nodes * vocab)))), nodes=nodes, shape=rng.choice(("level", "line", "chain")),
                    uneven=rng.random() < 0.5, vocab=vocab, dtype=rng.choice(("f32", "f32", "bf16")), draft=rng.random() < 0.6, cut=rng.random() < 0.4, salt=salt)
    nodes = _log(rng, 1, 1024)
    return dict(op=op, seqs=_log(rng, 1, min(64, 16384 // nodes)), nodes=nodes, shape="line", uneven=rng.random() < 0.5, rows=_log(rng, 1, 8192),
                page_rows=page_rows, salt=salt)


def _tree(rng, n, shape):
    """A draft's parents (-1 for node 0), each below its own number."""
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "level":  # level by level, the first levels wider
        return [-1] + [rng.randint((j - 1) // 4, (j - 1) // 2) for j in range(1, n)]
    # a line as deep as any, then others that leave it, none deeper
    depth = max(1, n // 3)
    parent = list(range(-1, min(n, depth + 1) - 1))
    while len(parent) < n:
        at = rng.randrange(depth)
        for k in range(rng.randint(1, depth - at)):
            if len(parent) < n:
                parent.append(at if k == 0 else len(parent) - 1)
    return parent


def _plan(case):
    """Each sequence's draft and its rows before it, from the case alone."""
    rng = random.Random(case["salt"])
    trees, rows = [], []
    for s in range(case["seqs"]):
        n = rng.randint((case["nodes"] + 1) // 2, case["nodes"]) if case["uneven"] else case["nodes"]
        trees.append(_tree(rng, n, case["shape"]))
        if case["op"] == "tree":
            # all of full length, or from `ragged` rows up, then from 1 the first of several without a row
            n = rng.randint(case["ragged"], case["rows"]) if case["ragged"] else case["rows"]
            rows.append(0 if case["ragged"] == 1 and s == 0 and case["seqs"] > 1 else n)
        elif case["op"] == "keep":
            rows.append(rng.randint(0, case["rows"]))
    return trees, rows


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _line(parent, leaf):
    """From node 0 to a node."""
    at = [leaf]
    while at[-1] > 0:
        at.append(parent[at[-1]])
    return at[::-1]


def _lines(case):
    """What each sequence keeps: the line to a node that leaves the first one (whose rows then all move)."""
    rng = random.Random(case["salt"] + 1)
    return [_line(p, rng.randrange(len(p) // 2, len(p))) for p in _plan(case)[0]]


def work(case):
    trees, rows = _plan(case)
    n = sum(map(len, trees))
    if case["op"] == "keep":
        moved = sum(j != i for line in _lines(case) for i, j in enumerate(line))
        return {"bytes": 2 * moved * (ROW - 1) + n * (ROW - 1 + DIM * 4) + n * 4, "flops": 0}
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": len(trees) * case["vocab"] * size * (2 if case["draft"] else 1) + n * (12 + size * (2 if case["draft"] else 1)) + n * 8,
                "flops": len(trees) * case["vocab"] * (3 if case["draft"] else 1)}
    heads, pairs, seen = case["heads"], 0, 0
    for p, r in zip(trees, rows):
        d = _depths(p)
        first = min(max(0, r + k - case["window"] + 1) for k in d) if case["window"] else 0
        seen += r - min(first, r) + len(p)
        pairs += sum(min(r + k + 1, case["window"]) if case["window"] else r + k + 1 for k in d)
    return {"bytes": seen * (ROW - 1) + n * heads * (DIM * 4 + 4) + n * 4, "flops": 4 * DIM * heads * pairs}


# ---- inputs -----------------------------------------------------------------------

def _pow2(e):
    """2^e as f32, exactly (int32 e in [-126, 127])."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax, top):
    """The least e in [E_MIN, E_MAX] with amax <= top 2^e, as int32 (exact: a power of two times `top` is a float)."""
    f, e = torch.frexp(amax / top)  # amax / top = f 2^e, f in [0.5, 1)
    e = torch.where(amax == 0, E_MIN, torch.where(f == 0.5, e - 1, e)).clamp(E_MIN, E_MAX).to(torch.int32)
    # the quotient may have rounded: put right by exact comparisons
    e = torch.where((amax > top * _pow2(e)) & (e < E_MAX), e + 1, e)
    return torch.where((amax <= top * _pow2(e - 1)) & (e > E_MIN), e - 1, e)


def _quantise(x):
    """x f32 [n, 512] -> codes u8 [n, 224], tails f16 [n, 64], scales u8 [n, 16]."""
    n = x.shape[0]
    nope, tail = x[:, :NOPE].reshape(n, NOPE // GROUP, GROUP), x[:, NOPE:]
    e = _exponent(nope.abs().amax(2), 6.0)
    y = nope * _pow2(-e)[:, :, None]
    a = y.abs()
    # to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code: the number of midpoints passed
    code = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).reshape(n, NOPE)
    top = torch.maximum(e.amax(1), _exponent(tail.abs().amax(1), 8.0))
    tails = (tail * _pow2(-top)[:, None]).clamp(-65504.0, 65504.0).to(torch.float16)
    scales = torch.zeros((n, SCALES), dtype=torch.uint8, device=x.device)
    scales[:, :NOPE // GROUP] = (e + 127).to(torch.uint8)
    scales[:, NOPE // GROUP] = (top + 127).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), tails, scales


def _planes(pages, R):
    """Views of the three planes: codes [P, R, 224], tails f16 [P, R, 64], scales [P, R, 16]."""
    P = pages.shape[0]
    c, t = R * CODES, R * (CODES + TAILS)
    return (pages[:, :c].unflatten(1, (R, CODES)), pages[:, c:t].view(torch.float16).unflatten(1, (R, TAIL)),
            pages[:, t:].unflatten(1, (R, SCALES)))


def _cache(g, R, need):
    """A pool of pages in a random order, as after many sequences came and went, with rows as an append would have left them."""
    P = sum(need) + 3
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    pages = torch.empty((P, R * ROW), dtype=torch.uint8, device="cuda")
    codes, tails, scales = _planes(pages, R)
    step = max(1, (1 << 18) // R)
    for p in range(0, P, step):
        m = min(step, P - p)
        c, t, s = _quantise(torch.randn((m * R, DIM), generator=g, device="cuda"))
        codes[p:p + m], tails[p:p + m], scales[p:p + m] = c.unflatten(0, (m, R)), t.unflatten(0, (m, R)), s.unflatten(0, (m, R))
    return pages, table


def _probabilities(case, g, n, parent, rank):
    """Target and draft probabilities after each of n nodes, and the tokens that were drafted: of a few likely tokens and a long
    tail, the draft's near the target's.  Sampled tokens are draws from the parent's draft, others its likeliest, in order."""
    V, dtype = case["vocab"], torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    wide = -(-V // 8) * 8
    target, draft = (torch.zeros((n, wide), dtype=dtype, device="cuda")[:, :V] for _ in range(2))
    tokens = torch.zeros(n, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // V)
    for f in range(0, n, step):
        m = min(step, n - f)
        logits = -1.3 * torch.log(torch.rand((m, V), generator=g, device="cuda").clamp_(min=1e-9))
        for to in (target, draft):
            p = torch.softmax(logits, 1)
            if case["cut"]:  # the least likely ones dropped, the rest renormalised
                p = torch.where(p < p.amax(1, keepdim=True) * 1e-3, 0.0, p)
                p = p / p.sum(1, keepdim=True)
            to[f:f + m] = p.to(dtype)
            logits += 0.7 * torch.randn((m, V), generator=g, device="cuda")
    if n > 1:
        for f in range(0, n, step):
            at = parent[f:f + step].clamp(min=0)
            q = draft[at].float()
            if case["draft"]:
                tokens[f:f + step] = (q / torch.empty_like(q).exponential_(generator=g)).argmax(1).to(torch.int32)
            else:
                best = torch.topk(q, min(V, 8), dim=1).indices
                tokens[f:f + step] = best.gather(1, rank[f:f + step, None].clamp(max=best.shape[1] - 1))[:, 0].to(torch.int32)
    return target, draft if case["draft"] else None, tokens


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    trees, rows = _plan(case)
    n, S = sum(map(len, trees)), len(trees)
    cu = [0]
    for p in trees:
        cu.append(cu[-1] + len(p))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    parent = [p for t in trees for p in t]
    st = dict(op=case["op"], most=max(map(len, trees)), cu=i32(cu), parent=i32(parent), ws=torch.zeros(48 << 20, dtype=torch.uint8, device="cuda"))
    if case["op"] == "verify":
        rank = []  # which of its parent's children a node is
        for t in trees:
            rank += [sum(q == p for q in t[:j]) for j, p in enumerate(t)]
        base = [c for c, t in zip(cu, trees) for _ in t]
        st["target"], st["draft"], st["tokens"] = _probabilities(case, g, n, torch.tensor([b + max(p, 0) for b, p in zip(base, parent)], device="cuda"),
                                                                 torch.tensor(rank, device="cuda"))
        st["u"] = torch.rand(n, generator=g, device="cuda")
        st["path"], st["out"] = torch.empty((2, n), dtype=torch.int32, device="cuda")
        st["count"] = torch.empty(S, dtype=torch.int32, device="cuda")
        return st
    R = st["R"] = case["page_rows"]
    st["pages"], st["table"] = _cache(g, R, [max(1, -(-(r + len(t)) // R)) for r, t in zip(rows, trees)])
    st["row0"] = torch.tensor(rows, dtype=torch.int64, device="cuda")
    if case["op"] == "keep":
        lines = _lines(case)
        st["path"] = i32([j for t, l in zip(trees, lines) for j in l + [-1] * (len(t) - len(l))])
        st["count"] = i32([len(l) for l in lines])
        st["back"] = torch.empty((n, DIM), dtype=torch.float32, device="cuda")
        return st
    st["q"] = torch.randn((n, case["heads"], DIM), generator=g, device="cuda").to(torch.bfloat16)
    st["out"] = torch.empty((n, case["heads"], DIM), dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device="cuda")
    # a window's first position for each node
    place = torch.tensor([r + d for t, r in zip(trees, rows) for d in _depths(t)], dtype=torch.int64, device="cuda")
    st["begin"] = (place - case["window"] + 1).clamp(min=0) if case["window"] else None
    st["max_rows"] = max(r + len(t) for t, r in zip(trees, rows))
    return st


# ---- one pass ---------------------------------------------------------------------

def _token_seq(st, n):
    """Each token's sequence and its number within it."""
    t = torch.arange(n, device=st["cu"].device)
    s = torch.searchsorted(st["cu"][1:], t.to(torch.int32), right=True)
    return s, t - st["cu"][s]


def _values(codes, tails, scales):
    """Rows' 512 values in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    nope = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    two = _pow2(scales[..., :15].int() - 127)
    nope = (nope.unflatten(-1, (NOPE // GROUP, GROUP)) * two[..., :14, None]).flatten(-2)
    return torch.cat((nope, tails.float() * two[..., 14:15]), -1)


def _rows(st, seq, row):
    """The values of the given rows of the given sequences (f32 [..., 512]; any row where the table names no page)."""
    R = st["R"]
    page = st["table"][seq, (row // R).clamp(0, st["table"].shape[1] - 1)].clamp(min=0).long()
    codes, tails, scales = _planes(st["pages"], R)
    at = (page, row % R)
    return _values(codes[at], tails[at], scales[at])


def _softmax_sum(logits, ok, v):
    """softmax over the last axis where ok, times v; zeros and -inf where nothing is left."""
    l = torch.where(ok, logits, float("-inf"))
    m = l.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(l - m0)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z == 0, 1.0, z)
    return out, (m0 + torch.log(z)).squeeze(-1)


def _plain_tree(st):
    q = st["q"].float()
    n, H = q.shape[:2]
    seq, j = _token_seq(st, n)
    S, T = st["table"].shape[0], st["most"]
    # lines[s, a, b]: b is a or one of its ancestors: powers of (1 + parent relation), squared until no line is longer
    lines = torch.eye(T, device=q.device).repeat(S, 1, 1)
    up = st["parent"].long()
    lines[seq, j, torch.where(up < 0, j, up)] = 1.0
    for _ in range(max(0, T - 1).bit_length()):
        lines = torch.matmul(lines, lines).clamp(max=1.0)
    lines = lines > 0
    place = st["row0"][:, None] + lines.sum(2) - 1  # a node's position
    row = torch.arange(st["max_rows"], device=q.device)
    v = _rows(st, torch.arange(S, device=q.device)[:, None], row.expand(S, -1))
    node = row - st["row0"][:, None]  # which node a row is
    at = node.clamp(0, T - 1)
    ok = torch.where((node < 0)[:, None, :], True, lines.gather(2, at[:, None, :].expand(-1, T, -1)) & (node < T)[:, None, :])
    if st["begin"] is not None:
        lo = torch.zeros((S, T), dtype=torch.int64, device=q.device)
        lo[seq, j] = st["begin"]
        pos = torch.where(node < 0, row, place.gather(1, at))
        ok = ok & (pos[:, None, :] >= lo[:, :, None])
    qp = torch.zeros((S, T, H, DIM), device=q.device)
    qp[seq, j] = q
    logits = torch.matmul(qp.flatten(1, 2), v.transpose(1, 2)) * SCALE
    out, lse = _softmax_sum(logits, ok.repeat_interleave(H, 1), v)
    return {"out": out.unflatten(1, (T, H))[seq, j].to(torch.bfloat16), "lse": lse.unflatten(1, (T, H))[seq, j]}


def _plain_verify(st):
    """All sequences' walks side by side, node by node: a node is tried when the walk stands at its parent.  In 64 bits: what is
    chosen turns on sums over the vocabulary."""
    cu, parent, u = st["cu"].long(), st["parent"], st["u"].double()
    S, V, n = cu.shape[0] - 1, st["target"].shape[1], parent.shape[0]
    first, end = cu[:-1], cu[1:]
    every = torch.arange(S, device=cu.device)
    cur, count = torch.zeros_like(first), torch.ones_like(first)
    w = st["target"][first].double()  # what is left of the target's probabilities, its mass, and how often the draft's have been taken off
    mass, t = torch.ones_like(first, dtype=torch.float64), torch.zeros_like(first, dtype=torch.float64)
    path = torch.full((S, st["most"]), -1, dtype=torch.int64, device=cu.device)
    path[:, 0] = 0
    out = torch.full_like(path, -1)
    for j in range(1, st["most"]):
        at = (first + j).clamp(max=n - 1)
        tried = (first + j < end) & (parent[at] == cur)
        x = st["tokens"][at].long()
        here = first + cur
        left = w[every, x]
        q = st["draft"][here, x].double() if st["draft"] is not None else 1.0
        took = tried & (u[at] * q * mass < left)
        lost = tried & ~took
        path[every, count] = torch.where(took, j, path[every, count])
        out[every, count - 1] = torch.where(took, x, out[every, count - 1])
        count = count + took
        cur = torch.where(took, j, cur)
        if st["draft"] is not None:
            t = torch.where(lost, t + mass, t)
            rest = (st["target"][here].double() - t[:, None] * st["draft"][here].double()).clamp(min=0.0)
            mass = torch.where(lost, rest.sum(1), mass)
        else:
            rest = w.index_put((every, x), torch.zeros((), dtype=torch.float64, device=cu.device))
            mass = torch.where(lost, mass - left, mass)
        w = torch.where(took[:, None], st["target"][at].double(), torch.where(lost[:, None], rest, w))
        mass, t = torch.where(took, 1.0, mass), torch.where(took, 0.0, t)
    c = torch.cumsum(w, 1)
    last = (c <= u[first][:, None] * c[:, -1:]).sum(1)
    out[every, count - 1] = torch.where(last < V, last, -1)
    seq, k = _token_seq(st, n)
    return {"path": path[seq, k].to(torch.int32), "out": out[seq, k].to(torch.int32), "count": count.to(torch.int32)}


def run(st):
    if own:
        from compressed_kv_sparse_csa_gb300 import binding as B

        if st["op"] == "tree":
            B.ds4x_paged_tree_attn(st["pages"], st["R"], st["table"], st["cu"], st["row0"], st["parent"], st["q"], SCALE, st["out"], st["lse"],
                                   st["ws"], row_begin=st["begin"])
            return {"out": st["out"], "lse": st["lse"]}
        if st["op"] == "verify":
            B.ds4x_verify_drafts(st["cu"], st["parent"], st["tokens"], st["target"], st["draft"], st["u"], st["path"], st["out"], st["count"], st["ws"])
            return {"path": st["path"], "out": st["out"], "count": st["count"]}
        B.ds4x_paged_keep(st["pages"], st["R"], st["table"], st["cu"], st["row0"], st["path"], st["count"], st["ws"])
        B.ds4x_paged_gather(st["pages"], st["R"], st["table"], st["cu"], st["row0"], st["back"], st["ws"])
        return {"rows": st["back"]}
    if st["op"] == "tree":
        return _plain_tree(st)
    if st["op"] == "verify":
        return _plain_verify(st)
    n = st["path"].shape[0]
    seq, j = _token_seq(st, n)
    row = st["row0"][seq] + j
    take = st["row0"][seq] + torch.where(j < st["count"][seq], st["path"].long(), j)
    planes = _planes(st["pages"], st["R"])
    page = lambda r: (st["table"][seq, r // st["R"]].long(), r % st["R"])  # noqa: E731
    moved = [p[page(take)] for p in planes]
    planes[0][page(row)], planes[1][page(row)], planes[2][page(row)] = moved
    return {"rows": _rows(st, seq, row)}


# ---- the definition in 64 bits ------------------------------------------------------

def _exact_row_values(st, page, at):
    """Rows (page, at) in 64 bits, byte by byte from the page layout."""
    R, flat = st["R"], st["pages"].view(-1)
    base = page.long() * (R * ROW)
    byte = lambda first, m: flat[(first[:, None] + torch.arange(m, device=flat.device))]  # noqa: E731
    c = byte(base + at * CODES, CODES).long()
    t = byte(base + R * CODES + at * TAILS, TAILS).contiguous().view(torch.float16).double()
    s = byte(base + R * (CODES + TAILS) + at * SCALES, SCALES).double() - 127
    x = torch.empty((c.shape[0], DIM), dtype=torch.float64, device=flat.device)
    for half, nib in ((0, c & 15), (1, c >> 4)):
        ex, man = (nib >> 1) & 3, nib & 1
        mag = torch.where(ex == 0, man * 0.5, (1 + man * 0.5) * torch.exp2(ex.double() - 1))
        x[:, half:NOPE:2] = torch.where(nib >= 8, -mag, mag)
    x[:, :NOPE] *= torch.exp2(s[:, :14]).repeat_interleave(GROUP, 1)
    x[:, NOPE:] = t * torch.exp2(s[:, 14:15])
    return x


def _exact_verify(case, st, trees):
    """The walk as it is written down, one sequence and one node at a time: a child x of the node is taken with probability
    p(x) / q(x); if it is not, p becomes max(p - q, 0), renormalised (without a draft's probabilities: p without x)."""
    path, out, count, first = [], [], [], 0
    u, tok = st["u"].double().tolist(), st["tokens"].tolist()
    for tree in trees:
        cur, line, said = 0, [0], []
        while True:
            p = st["target"][first + cur].double()
            q = st["draft"][first + cur].double() if st["draft"] is not None else None
            took = None
            for j in (j for j, up in enumerate(tree) if up == cur and j > cur):
                x = tok[first + j]
                if u[first + j] * (float(q[x]) if q is not None else 1.0) < float(p[x]):
                    took = j
                    break
                if q is None:
                    left = 1.0 - float(p[x])
                    p[x] = 0.0
                    p = p / left
                else:
                    p = torch.clamp(p - q, min=0.0)
                    p = p / p.sum()
            if took is None:
                c = torch.cumsum(p, 0)
                y = int(torch.searchsorted(c, u[first] * c[-1], right=True))
                said.append(y if y < case["vocab"] else -1)
                break
            line.append(took)
            said.append(tok[first + took])
            cur = took
        fill = [-1] * (len(tree) - len(line))
        path, out, count, first = path + line + fill, out + said + fill, count + [len(line)], first + len(tree)
    return {"path": torch.tensor(path, dtype=torch.int32), "out": torch.tensor(out, dtype=torch.int32), "count": torch.tensor(count, dtype=torch.int32)}


def exact(case, seed):
    st = prepare(case, seed)
    trees, rows = _plan(case)
    if case["op"] == "verify":
        return _exact_verify(case, st, trees)
    R, out, lse, first = st["R"], [], [], 0
    for s, (tree, before) in enumerate(zip(trees, rows)):
        n = len(tree)
        if case["op"] == "keep":
            line = _lines(case)[s]
            src = torch.tensor([before + (line[i] if i < len(line) else i) for i in range(n)], device="cuda")
            out.append(_exact_row_values(st, st["table"][s][src // R], src % R))
            continue
        at = torch.arange(before + n, device="cuda")
        v = _exact_row_values(st, st["table"][s][at // R], at % R)
        depth = _depths(tree)
        for f in range(0, n, 32):
            m = min(f + 32, n)
            sees = torch.zeros((m - f, before + n), dtype=torch.bool, device="cuda")
            for i in range(f, m):
                low = max(0, before + depth[i] - case["window"] + 1) if case["window"] else 0
                sees[i - f, min(low, before):before] = True
                for a in _line(tree, i):
                    if before + depth[a] >= low:
                        sees[i - f, before + a] = True
            l = torch.einsum("thd,rd->thr", st["q"][first + f:first + m].double(), v) * SCALE
            l.masked_fill_(~sees[:, None, :], float("-inf"))
            z = torch.logsumexp(l, 2)
            lse.append(z)
            out.append(torch.einsum("thr,rd->thd", torch.exp(l - z[:, :, None]), v))
        first += n
    if case["op"] == "keep":
        return {"rows": torch.cat(out)}
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
