"""A step of a server that drafts, call after call as it runs them: append the
drafts' rows at their depths' positions, attend over the trees, decide, keep the
accepted rows, and go on from there: the next step's attention sees them."""

import numpy as np
import pytest
import torch

from gpu_path import bf16_dev, bf16_host_bits, dev, new_ws, require_gpu
from oracle import codecs as C
from oracle import drafts as D
from oracle import paged as O
from paged_path import bf16, check_token
from test_gpu_verify import probabilities

pytestmark = pytest.mark.gpu
SCALE = 512.0 ** -0.5
R, S, N, H, V = 16, 3, 8, 20, 997


class Steps:
    """The device buffers of a server's step, and the rows on the host beside."""

    def __init__(self, seed):
        B = self.B = require_gpu()
        self.rng = np.random.default_rng(seed)
        self.rows = [0, 33, 14]          # committed rows per sequence
        pages = 12
        self.table = np.arange(S * pages, dtype=np.int32).reshape(S, pages)[:, ::-1].copy()
        self.host = [np.zeros((pages * R, 512)) for _ in range(S)]
        self.freq = (10000.0 ** -(np.arange(32) / 32.0)).astype(np.float32)
        n = S * N
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.d = dict(pages=torch.zeros((S * pages, R * 368), dtype=torch.uint8, device="cuda"), table=dev(self.table),
                      cu=i32(S + 1), parent=i32(n), tokens=i32(n), path=i32(n), out_tokens=i32(n), n_path=i32(S),
                      row0=torch.zeros(S, dtype=torch.int64, device="cuda"), pos=torch.zeros(n, dtype=torch.int64, device="cuda"),
                      x=torch.zeros((n, 512), dtype=torch.bfloat16, device="cuda"), freq=dev(self.freq),
                      q=torch.zeros((n, H, 512), dtype=torch.bfloat16, device="cuda"),
                      out=torch.zeros((n, H, 512), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((n, H), device="cuda"),
                      target=torch.zeros((n, 1000), device="cuda")[:, :V], draft=torch.zeros((n, 1000), device="cuda")[:, :V],
                      u=torch.zeros(n, device="cuda"), back=torch.zeros((n, 512), device="cuda"))
        self.ws = new_ws(B.ds4x_paged_attn_workspace())
        first = [self.rng.standard_normal((r, 512)).astype(np.float32) for r in self.rows]
        cu = np.concatenate([[0], np.cumsum(self.rows)]).astype(np.int32)
        B.ds4x_paged_append(self.d["pages"], R, self.d["table"], dev(cu), torch.zeros(S, dtype=torch.int64, device="cuda"),
                            dev(np.concatenate(first)), self.ws, inv_freq=self.d["freq"])
        for s, x in enumerate(first):
            if len(x):
                self.host[s][:len(x)] = O.values(*O.quantise(O.rotate(x, np.arange(len(x)), self.freq, False).astype(np.float32)))

    def calls(self):
        """One step, as a captured graph or eagerly."""
        B, d, ws = self.B, self.d, self.ws
        B.ds4x_paged_append(d["pages"], R, d["table"], d["cu"], d["row0"], d["x"], ws, pos=d["pos"], inv_freq=d["freq"])
        B.ds4x_paged_tree_attn(d["pages"], R, d["table"], d["cu"], d["row0"], d["parent"], d["q"], SCALE, d["out"], d["lse"], ws)
        B.ds4x_verify_drafts(d["cu"], d["parent"], d["tokens"], d["target"], d["draft"], d["u"], d["path"], d["out_tokens"],
                             d["n_path"], ws)
        B.ds4x_paged_keep(d["pages"], R, d["table"], d["cu"], d["row0"], d["path"], d["n_path"], ws)
        B.ds4x_paged_gather(d["pages"], R, d["table"], d["cu"], d["row0"], d["back"], ws)

    def inputs(self, shape):
        rng, d = self.rng, self.d
        nodes = [int(rng.integers(1, N + 1)) for _ in range(S)]
        self.trees = [D.tree(rng, m, shape) for m in nodes]
        self.n, self.at = sum(nodes), np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        depth = [len(D.line(t, j)) - 1 for t in self.trees for j in range(len(t))]
        self.pos = np.array([r + e for r, e in zip(np.repeat(self.rows, nodes), depth)], dtype=np.int64)
        xb, self.x = bf16(rng.standard_normal((self.n, 512)))
        qb, self.q = bf16(rng.standard_normal((self.n, H, 512)))
        self.target, self.draft = probabilities(rng, self.n, V), probabilities(rng, self.n, V)
        both = 0.7 * self.target + 0.3 * self.draft
        self.draft = (both / both.sum(axis=1, keepdims=True)).astype(np.float32)
        self.tokens = np.array([rng.choice(V, p=self.draft[self.at[s] + max(p, 0)].astype(np.float64) /
                                           self.draft[self.at[s] + max(p, 0)].astype(np.float64).sum())
                                for s, t in enumerate(self.trees) for p in t], dtype=np.int32)
        self.u = rng.random(self.n).astype(np.float32)
        put = lambda k, v: d[k][:len(v)].copy_(v if isinstance(v, torch.Tensor) else torch.tensor(np.asarray(v)))  # noqa: E731
        put("cu", self.at)
        put("parent", np.array([p for t in self.trees for p in t], dtype=np.int32))
        put("pos", self.pos)
        put("row0", np.array(self.rows, dtype=np.int64))
        put("x", bf16_dev(xb))
        put("q", bf16_dev(qb))
        put("target", self.target)
        put("draft", self.draft)
        put("tokens", self.tokens)
        put("u", self.u)

    def check(self):
        d = self.d
        out, lse = C.bf16_decode(bf16_host_bits(d["out"])).astype(np.float64), d["lse"].cpu().numpy().astype(np.float64)
        path, new, count = (d[k].tolist() for k in ("path", "out_tokens", "n_path"))
        back = d["back"].cpu().numpy().astype(np.float64)
        for s, tree in enumerate(self.trees):
            a, m, row0 = int(self.at[s]), len(tree), self.rows[s]
            # the drafts' rows, as the cache holds them: read back they are the host's within what the float
            # rotation may round differently, so the attention is checked over what the cache says it holds
            rows = self.host[s]
            rows[row0:row0 + m] = self.drafted[a:a + m]
            want = O.values(*O.quantise(O.rotate(self.x[a:a + m], self.pos[a:a + m], self.freq, False).astype(np.float32)))
            big = np.abs(want).max(axis=1, keepdims=True)
            assert np.all(np.abs(rows[row0:row0 + m] - want) <= 2.0 ** -9 * big)
            for j in range(m):
                check_token(out[a + j], lse[a + j], rows[D.sees(tree, j, row0)], self.q[a + j], SCALE)
            p, o, near = D.verify(tree, self.tokens[a:a + m], self.target[a:a + m], self.draft[a:a + m], self.u[a:a + m])
            assert near > 2.0 ** -36
            assert path[a:a + m] == p + [-1] * (m - len(p)) and new[a:a + m] == o + [-1] * (m - len(o)) and count[s] == len(p)
            rows[:row0 + m] = np.stack(D.keep(list(rows[:row0 + m]), row0, p))
            assert np.array_equal(back[a:a + m], rows[row0:row0 + m])
            self.rows[s] += len(p)

    def read_drafted(self):
        """What the appended rows are, before any is moved."""
        d = self.d
        back = torch.empty((S * N, 512), device="cuda")
        self.B.ds4x_paged_append(d["pages"], R, d["table"], d["cu"], d["row0"], d["x"], self.ws, pos=d["pos"], inv_freq=d["freq"])
        self.B.ds4x_paged_gather(d["pages"], R, d["table"], d["cu"], d["row0"], back, self.ws)
        self.drafted = back.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("captured", [False, True])
def test_steps_follow_one_another(captured):
    steps = Steps(60)
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
    assert sum(steps.rows) > 47 + 18  # a token at least a sequence and step


def test_two_steps_at_once():
    """Two servers' steps on two streams, each with its own workspace: the same
    results as one after the other."""
    a, b = Steps(61), Steps(62)
    for s in (a, b):
        s.inputs("level")
        s.read_drafted()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, s in zip(streams, (a, b)):
        with torch.cuda.stream(st):
            for _ in range(3):
                s.calls()
    torch.cuda.synchronize()
    for s in (a, b):
        s.check()
        assert s.B.ds4x_workspace_status(s.ws) == 0
