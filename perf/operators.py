"""What is measured of the paged 4-bit cache's operators, and their plain forms.

The cache holds one 512-value vector a row, shared by all heads as key and
value: 448 values in E2M1 with one power-of-two scale per 32 values, and a
tail of 64 values in FP16 with a scale of its own.  Rows live in pages of
`page_rows` rows; a table names each sequence's pages.  A page of R rows is
three planes: codes u8 [R][224] (two a byte, the even value in the low
nibble), tails f16 [R][64], scales u8 [R][16] (14 block scales, the tail's
scale, a zero byte; byte b stands for 2^(b - 127)).  The tail's exponent is at
least every block's.

  append   rotate a new row's tail at its position, quantise, write it into
           its sequence's pages; the rows are read back from the pages
  attn     attention of each query token over a range of its sequence's rows
  sparse   attention of each query token over its own list of rows

Tokens are ragged over the sequences: sequence s has the tokens
cu[s] .. cu[s + 1] - 1.
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
        # one session's new row, far into a million-row history: a decode step's append
        dict(name="append_one", op="append", seqs=1, tokens=1, rows=1048576, page_rows=64, dtype="bf16", style=0, salt=1),
        # 61 sessions decoding together, one new fp32 row each
        dict(name="append_batch", op="append", seqs=61, tokens=61, rows=65536, page_rows=128, dtype="f32", style=1, salt=2),
        # a chunk of prompts of different lengths
        dict(name="append_prompts", op="append", seqs=7, tokens=16384, rows=4096, page_rows=32, dtype="bf16", style=0, salt=3),
        # a short history, one token
        dict(name="decode_short", op="attn", seqs=1, tokens=1, heads=64, rows=777, ragged=0, window=0, page_rows=32, salt=4),
        # every compressed row of a million-token context at ratio 128
        dict(name="decode_8192", op="attn", seqs=1, tokens=1, heads=64, rows=8192, ragged=0, window=0, page_rows=64, salt=5),
        # one session over a million rows
        dict(name="decode_1m", op="attn", seqs=1, tokens=1, heads=64, rows=1048576, ragged=0, window=0, page_rows=128, salt=6),
        # 16 sessions of 8192 to 65536 rows
        dict(name="decode_sessions", op="attn", seqs=16, tokens=1, heads=64, rows=65536, ragged=8192, window=0, page_rows=64, salt=7),
        # few heads, five tokens a session (a draft being checked), ragged from an empty history, a sliding window
        dict(name="draft_window", op="attn", seqs=24, tokens=5, heads=20, rows=9001, ragged=1, empty=True, window=4999, page_rows=16, salt=8),
        # a prompt's chunk over what is there before it
        dict(name="prefill_chunk", op="attn", seqs=1, tokens=2048, heads=64, rows=8192, ragged=0, window=0, page_rows=256, salt=9),
        # a decode step's 512 selected rows of a million
        dict(name="sparse_one", op="sparse", seqs=1, tokens=1, heads=64, rows=1048576, ragged=0, k=512, page_rows=64, salt=10),
        # 16 sessions, 512 rows each
        dict(name="sparse_sessions", op="sparse", seqs=16, tokens=1, heads=64, rows=65536, ragged=8192, k=512, page_rows=64, salt=11),
        # a prompt's chunk, 512 rows a token
        dict(name="sparse_prefill", op="sparse", seqs=1, tokens=2048, heads=64, rows=65536, ragged=0, k=512, page_rows=64, salt=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attn", "attn", "sparse"))
    page_rows, salt = rng.choice((16, 32, 64, 128, 256)), rng.randrange(1 << 30)
    if op == "append":
        tokens = _log(rng, 1, 16384)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 64)), tokens=tokens, rows=_log(rng, 1, 65536), page_rows=page_rows,
                    dtype=rng.choice(("bf16", "f32")), style=rng.choice((0, 1)), salt=salt)
    heads = rng.choice((64, 64, 64, 128, 1, 8, 16, 20, 33, 48, 100))
    if op == "attn":
        if rng.random() < 0.25:  # a prompt's chunk
            rows = _log(rng, 64, 8192)
            return dict(op=op, seqs=rng.choice((1, 1, 2, 3)), tokens=min(rows, _log(rng, 16, 512)), heads=min(heads, 64), rows=rows,
                        ragged=0, window=rng.choice((0, 0, 1 + rows // 2)), page_rows=page_rows, salt=salt)
        seqs, tokens = _log(rng, 1, 32), rng.choice((1, 1, 1, 2, 3, 7))
        rows = _log(rng, 1, min(1048576, 1048576 // seqs // (tokens * max(heads, 64) // 64)))
        return dict(op=op, seqs=seqs, tokens=tokens, heads=heads, rows=rows, ragged=rng.choice((0, 1, (rows + 1) // 2)), empty=seqs > 1 and rng.random() < 0.2,
                    window=rng.choice((0, 0, 0, 1 + rows // 3)), page_rows=page_rows, salt=salt)
    if rng.random() < 0.4:
        seqs, tokens = 1, _log(rng, 8, 1024)
    else:
        seqs, tokens = _log(rng, 1, 24), rng.choice((1, 1, 2, 4))
    rows = _log(rng, 50, min(1048576, 2097152 // seqs, (1 << 27) // (seqs * tokens)))
    return dict(op=op, seqs=seqs, tokens=tokens, heads=heads, rows=rows, ragged=rng.choice((0, (rows + 1) // 2)),
                k=_log(rng, 1, 512), page_rows=page_rows, salt=salt)


def _plan(case):
    """The case's sequences: tokens per sequence, rows per sequence (after the append), from the case alone."""
    rng, S = random.Random(case["salt"]), case["seqs"]
    if case["op"] == "append":  # ragged prompts: a random split of the tokens, at least one each
        n = case["tokens"]
        cuts = sorted(rng.sample(range(1, n), S - 1)) if S > 1 else []
        tok = [b - a for a, b in zip([0] + cuts, cuts + [n])]
        before = [case["rows"] if S == 1 else rng.randrange(case["rows"] + 1) for _ in range(S)]
        return tok, [a + b for a, b in zip(before, tok)]
    tok = [case["tokens"]] * S
    # all of full length, or from `ragged` rows up; the first sequence without a row where the case says so
    rows = [rng.randint(case["ragged"], case["rows"]) if case["ragged"] else case["rows"] for _ in range(S)]
    if case.get("empty"):
        rows[0] = 0
    return tok, rows


def _ranges(case):
    """Each token's visible rows [begin, end): its sequence's rows up to its own, the last token seeing all."""
    begin, end = [], []
    for t, n in zip(*_plan(case)):
        for j in range(t):
            e = max(0, n - (t - 1 - j))
            end.append(e)
            begin.append(max(0, e - case["window"]) if case.get("window") else 0)
    return begin, end


def work(case):
    tok, rows = _plan(case)
    row = NOPE // 2 + 2 * TAIL + NOPE // GROUP + 1
    if case["op"] == "append":
        n, size = case["tokens"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (DIM * size + row) + n * (row + DIM * 2), "flops": n * 6 * TAIL}
    begin, end = _ranges(case)
    heads, n = case["heads"], len(end)
    io = n * heads * (DIM * 4 + 4)
    if case["op"] == "attn":
        seen, at = 0, 0
        for t, r in zip(tok, rows):  # each sequence's rows once, those that some token sees
            seen += max(0, max(end[at:at + t]) - min(begin[at:at + t]))
            at += t
        pairs = sum(max(0, e - b) for b, e in zip(begin, end))
        return {"bytes": seen * row + io, "flops": 4 * DIM * heads * pairs}
    pairs = sum(min(case["k"], e) for e in end)
    # a row that several tokens list is read once
    seen = sum(min(sum(min(case["k"], e) for e in end[i * case["tokens"]:(i + 1) * case["tokens"]]), rows[i]) for i in range(case["seqs"]))
    return {"bytes": seen * row + n * case["k"] * 4 + io, "flops": 4 * DIM * heads * pairs}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, R = "cuda", case["page_rows"]
    tok, rows = _plan(case)
    S, n = len(tok), sum(tok)
    need = [max(1, -(-r // R)) for r in rows]
    P = sum(need) + 3
    # the pool's pages in a random order, as after many sequences came and went; unused table entries are -1
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.full((S, max(need) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = perm[at:at + k]
        at += k
    cu = torch.tensor([sum(tok[:s]) for s in range(S + 1)], dtype=torch.int32, device=dev)
    st = dict(op=case["op"], R=R, table=table, cu=cu, ws=torch.zeros(48 << 20, dtype=torch.uint8, device=dev))
    if case["op"] == "append":
        st["pages"] = torch.zeros((P, R * ROW), dtype=torch.uint8, device=dev)
        x = torch.randn((n, DIM), generator=g, device=dev)
        st["x"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        st["row0"] = torch.tensor([r - t for r, t in zip(rows, tok)], dtype=torch.int64, device=dev)
        st["pos"] = torch.cat([torch.arange(r - t, r, device=dev) for r, t in zip(rows, tok)]) * 4 + 3  # a row of four tokens, its last one's place
        st["freq"] = (10000.0 ** (-torch.arange(TAIL // 2, device=dev, dtype=torch.float64) / (TAIL // 2))).to(torch.float32)
        st["style"] = case["style"]
        st["back"] = torch.empty((n, DIM), dtype=torch.bfloat16, device=dev)
        return st
    pages = torch.empty((P, R * ROW), dtype=torch.uint8, device=dev)
    codes, tails, scales = _planes(pages, R)
    step = max(1, (1 << 18) // R)
    for p in range(0, P, step):  # rows as an append would have left them
        m = min(step, P - p)
        c, t, s = _quantise(torch.randn((m * R, DIM), generator=g, device=dev))
        codes[p:p + m], tails[p:p + m], scales[p:p + m] = c.unflatten(0, (m, R)), t.unflatten(0, (m, R)), s.unflatten(0, (m, R))
    begin, end = _ranges(case)
    st["pages"] = pages
    st["q"] = torch.randn((n, case["heads"], DIM), generator=g, device=dev).to(torch.bfloat16)
    st["out"] = torch.empty((n, case["heads"], DIM), dtype=torch.bfloat16, device=dev)
    st["lse"] = torch.empty((n, case["heads"]), dtype=torch.float32, device=dev)
    st["end"] = torch.tensor(end, dtype=torch.int64, device=dev)
    if case["op"] == "attn":
        st["begin"] = torch.tensor(begin, dtype=torch.int64, device=dev) if case["window"] else None
        # tokens and rows as padded lists per sequence
        st["max_rows"], st["max_tok"] = max(1, max(rows)), max(tok)
    else:
        st["rows"] = torch.tensor(rows, dtype=torch.int64, device=dev)
        # k distinct rows of those that the token sees, in no order; -1 where it sees fewer
        key = torch.rand((n, max(case["k"], max(rows))), generator=g, device=dev)
        key.masked_fill_(torch.arange(key.shape[1], device=dev) >= st["end"][:, None], -1.0)
        val, idx = torch.topk(key, case["k"], dim=1)
        st["idx"] = torch.where(val >= 0, idx, -1).to(torch.int32)
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


def _rotate(st, x):
    ang = st["pos"].double()[:, None] * st["freq"].double()
    c, s = torch.cos(ang).float(), torch.sin(ang).float()
    tail = x[:, NOPE:]
    a, b = (tail[:, 0::2], tail[:, 1::2]) if st["style"] == 0 else (tail[:, :TAIL // 2], tail[:, TAIL // 2:])
    a, b = a * c - b * s, a * s + b * c
    tail = torch.stack((a, b), 2).flatten(1) if st["style"] == 0 else torch.cat((a, b), 1)
    return torch.cat((x[:, :NOPE], tail), 1)


def _softmax_sum(logits, ok, v):
    """softmax over the last axis where ok, times v; zeros and -inf where nothing is left."""
    l = torch.where(ok, logits, float("-inf"))
    m = l.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(l - m0)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z == 0, 1.0, z)
    return out, (m0 + torch.log(z)).squeeze(-1)


def run(st):
    if own:
        from compressed_kv_sparse_csa_gb300 import binding as B

        if st["op"] == "append":
            B.ds4x_paged_append(st["pages"], st["R"], st["table"], st["cu"], st["row0"], st["x"], st["ws"], pos=st["pos"],
                                inv_freq=st["freq"], rope_style=st["style"])
            B.ds4x_paged_gather(st["pages"], st["R"], st["table"], st["cu"], st["row0"], st["back"], st["ws"])
            return {"rows": st["back"]}
        if st["op"] == "attn":
            B.ds4x_paged_attn(st["pages"], st["R"], st["table"], st["cu"], st["end"], st["q"], SCALE, st["out"], st["lse"], st["ws"],
                              row_begin=st["begin"])
        else:
            B.ds4x_paged_sparse_attn(st["pages"], st["R"], st["table"], st["cu"], st["rows"], st["idx"], st["q"], SCALE, st["out"],
                                     st["lse"], st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    if st["op"] == "append":
        seq, j = _token_seq(st, st["x"].shape[0])
        row = st["row0"][seq] + j
        page, at = st["table"][seq, row // st["R"]].long(), row % st["R"]
        codes, tails, scales = _planes(st["pages"], st["R"])
        codes[page, at], tails[page, at], scales[page, at] = _quantise(_rotate(st, st["x"].float()))
        return {"rows": _rows(st, seq, row).to(torch.bfloat16)}
    q = st["q"].float()
    n, H = q.shape[:2]
    seq, j = _token_seq(st, n)
    if st["op"] == "sparse":
        idx = st["idx"].long()
        v = _rows(st, seq[:, None], idx.clamp(min=0))
        out, lse = _softmax_sum(torch.matmul(q, v.transpose(1, 2)) * SCALE, (idx >= 0)[:, None, :], v)
        return {"out": out.to(torch.bfloat16), "lse": lse}
    S, T = st["table"].shape[0], st["max_tok"]
    row = torch.arange(st["max_rows"], device=q.device)
    v = _rows(st, torch.arange(S, device=q.device)[:, None], row.expand(S, -1))
    qp = torch.zeros((S, T, H, DIM), device=q.device)
    qp[seq, j] = q
    lo, hi = torch.zeros((2, S, T), dtype=torch.int64, device=q.device)
    hi[seq, j] = st["end"]
    if st["begin"] is not None:
        lo[seq, j] = st["begin"]
    ok = (row >= lo[..., None]) & (row < hi[..., None])
    logits = torch.matmul(qp.flatten(1, 2), v.transpose(1, 2)) * SCALE
    out, lse = _softmax_sum(logits, ok.repeat_interleave(H, 1), v)
    return {"out": out.unflatten(1, (T, H))[seq, j].to(torch.bfloat16), "lse": lse.unflatten(1, (T, H))[seq, j]}


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


def exact(case, seed):
    st = prepare(case, seed)
    tok, rows = _plan(case)
    begin, end = _ranges(case) if case["op"] != "append" else (None, None)
    if case["op"] == "append":
        x = st["x"].double()
        turn = st["pos"].double()[:, None] * st["freq"].double()[None, :]
        i = torch.arange(TAIL // 2, device=x.device)
        ia, ib = (NOPE + 2 * i, NOPE + 2 * i + 1) if case["style"] == 0 else (NOPE + i, NOPE + TAIL // 2 + i)
        a, b = x[:, ia].clone(), x[:, ib].clone()
        x[:, ia], x[:, ib] = a * turn.cos() - b * turn.sin(), b * turn.cos() + a * turn.sin()
        grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        tops = []
        for blk in range(NOPE // GROUP):
            part = x[:, blk * GROUP:(blk + 1) * GROUP]
            amax = part.abs().amax(1)
            e = torch.full_like(amax, E_MIN)
            for k in range(E_MIN, E_MAX):
                e = torch.where(amax > 6.0 * 2.0 ** k, float(k + 1), e)
            y = part / torch.exp2(e)[:, None]
            d = (y.abs()[:, :, None] - grid).abs()
            near = d == d.amin(2, keepdim=True)
            # of two as near, the even code
            code = torch.where(near, (torch.arange(8, device=x.device) % 2) * 16 + torch.arange(8, device=x.device), 99).amin(2) % 16
            x[:, blk * GROUP:(blk + 1) * GROUP] = torch.copysign(grid[code], y) * torch.exp2(e)[:, None]
            tops.append(e)
        tail = x[:, NOPE:]
        amax = tail.abs().amax(1)
        e = torch.full_like(amax, E_MIN)
        for k in range(E_MIN, E_MAX):
            e = torch.where(amax > 8.0 * 2.0 ** k, float(k + 1), e)
        e = torch.stack(tops + [e]).amax(0)[:, None]
        x[:, NOPE:] = (tail / torch.exp2(e)).to(torch.float16).double() * torch.exp2(e)
        return {"rows": x}
    heads = case["heads"]
    out = torch.zeros((sum(tok), heads, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(tok), heads), float("-inf"), dtype=torch.float64, device="cuda")

    def attend(t, v, first, last):
        """Tokens first..last-1 over rows v, where token i sees t[i]."""
        l = torch.einsum("thd,rd->thr", st["q"][first:last].double(), v) * SCALE
        l.masked_fill_(~t[:, None, :], float("-inf"))
        lse[first:last] = torch.logsumexp(l, 2)
        p = torch.exp(l - lse[first:last, :, None]).nan_to_num_(0.0)
        out[first:last] = torch.einsum("thr,rd->thd", p, v)

    at = 0
    for s in range(case["seqs"]):
        n, r = tok[s], rows[s]
        if case["op"] == "attn" and r:
            j = torch.arange(r, device="cuda")
            v = _exact_row_values(st, st["table"][s][j // st["R"]], j % st["R"])
            for f in range(at, at + n, 64):
                m = min(f + 64, at + n)
                lo, hi = (torch.tensor(z[f:m], device="cuda")[:, None] for z in (begin, end))
                attend((j >= lo) & (j < hi), v, f, m)
        elif case["op"] == "sparse":
            for f in range(at, at + n):
                j = st["idx"][f].long()
                j = j[j >= 0]
                if len(j):
                    v = _exact_row_values(st, st["table"][s][j // st["R"]], j % st["R"])
                    attend(torch.ones((1, len(j)), dtype=torch.bool, device="cuda"), v, f, f + 1)
        at += n
    return {"out": out, "lse": lse}
