"""The decode step's calls run together, as a serving loop uses them: prompts into pages, steps of one token across page
boundaries, requests that end and others that take their pages, a pool that runs out; eagerly and captured. And drafted rows
under a filter verified against filtered target rows."""
import numpy as np
import pytest
import torch

import oracle
from tree_speculative_verification_gb300 import api
from tree_speculative_verification_gb300.step import DecodeStep

from _decode import PK, attention64, check_sample, cu

pytestmark = pytest.mark.gpu


class Loop:
    """DecodeStep beside plain lists of every request's rows."""

    def __init__(self, B, Hq, Hk, d, V, num_pages, max_pages, seed=0, **sampling):
        self.B, self.Hq, self.Hk, self.d, self.V = B, Hq, Hk, d, V
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.sampling = {"temperature": [1.0] * B, "top_k": [0] * B, "top_p": [1.0] * B, "min_p": [0.0] * B, **sampling}
        t = lambda n: cu(self.sampling[n], np.int32 if n == "top_k" else np.float32)
        self.step = DecodeStep(B, Hq, Hk, d, num_pages, max_pages, **{n: t(n) for n in self.sampling})
        self.rows = [[] for _ in range(B)]       # (k, v) rows of each request
        r = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
        self.qkv, self.logits, self.u = r(B, Hq + 2 * Hk, d), r(B, V, t=torch.float32), r(B, t=torch.float32)
        self.probs = r(B, V, t=torch.float32)

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def begin(self, lengths):
        x = self.rand(int(sum(lengths)), 2 * self.Hk, self.d)
        self.step.begin(cu(lengths), x[:, :self.Hk], x[:, self.Hk:])
        at = 0
        for b, n in enumerate(lengths):
            self.rows[b] += [(x[i, :self.Hk], x[i, self.Hk:]) for i in range(at, at + n)]
            at += n

    def inputs(self):
        self.qkv.copy_(self.rand(*self.qkv.shape))
        self.logits.copy_(3 * torch.randn(self.B, self.V, generator=self.g, device="cuda"))
        self.u.copy_(cu(self.rng.random(self.B), np.float32))

    def parts(self):
        x, a, b = self.qkv, self.Hq, self.Hq + self.Hk
        return x[:, :a], x[:, a:b], x[:, b:]

    def run(self):
        self.step.run(*self.parts(), self.logits, self.u, self.probs)

    def check(self, stuck=()):
        q, k, v = self.parts()
        for b in range(self.B):
            if self.rows[b] and b not in stuck:
                self.rows[b].append((k[b].clone(), v[b].clone()))
        assert self.step.len.tolist() == [len(r) for r in self.rows]
        for b, rows in enumerate(self.rows):
            got = self.step.out[b].double()
            if not rows:
                assert not got.any()
                continue
            K, V = (torch.stack([r[i] for r in rows], 1) for i in range(2))
            ref, tol = attention64(q[b], K, V, self.d ** -0.5)
            assert ((got - ref).abs() <= tol).all(), f"request {b}"
        s = self.sampling
        check_sample(self.logits.cpu().numpy(), self.u.cpu().numpy(), np.array(s["temperature"], np.float32),
                     np.array(s["top_k"]), np.array(s["top_p"], np.float32), np.array(s["min_p"], np.float32),
                     self.step.token.cpu().numpy(), self.probs.cpu().numpy())


MIXED = {"temperature": [1.0, 0.0, 0.7, 1.0, 1.2], "top_k": [0, 0, 20, 50, 0], "top_p": [0.9, 1.0, 1.0, 0.8, 1.0],
         "min_p": [0.0, 0.0, 0.0, 0.02, 0.05]}


@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(captured):
    """Requests grow across pages, one ends, another takes its place."""
    x = Loop(5, 8, 2, 128, 3001, 12, 8, **MIXED)
    x.begin([62, 1, 130, 0, 64])
    graph = None
    for i in range(9):
        x.inputs()
        if captured and i == 2:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
                x.run()
        graph.replay() if graph else x.run()
        x.check()
        if i == 4:
            x.step.end(cu([False, False, True, False, True], bool))
            x.rows[2], x.rows[4] = [], []
            x.begin([0, 0, 0, 200, 3])
    assert x.step.status.item() == 0
    assert int(x.step.pool.state[1]) == 12 - sum(-(-len(r) // PK) for r in x.rows)


def test_pool_that_runs_out():
    """A request without a page stays as long as it is, until another ends; no page is lost or held twice."""
    x = Loop(3, 2, 1, 64, 500, 3, 4, seed=5)
    x.begin([64, 63, 60])
    x.inputs()
    x.run()                                                    # request 0 needs a second page: there is none
    x.check(stuck=[0])
    assert x.step.status.item() == api.STATUS_NO_PAGES
    x.step.status.zero_()
    x.step.end(cu([False, True, False], bool))
    x.rows[1] = []
    for _ in range(3):
        x.inputs()
        x.run()
        x.check()
    assert x.step.status.item() == 0
    held = [int(p) for b in range(3) for p in x.step.pool.block_table[b, :int(x.step.pool.held[b])]]
    assert sorted(held) == [0, 1, 2]


@pytest.mark.parametrize("top_p,top_k", [(0.9, 0), (1.0, 40), (0.7, 100)])
def test_filtered_rows_verified(top_p, top_k):
    """A drafter's filtered rows and tokens, and target rows under the same filter, through verify_mss: the oracle's tokens for
    the same rows, and none that the filter dropped."""
    B, n, V, T = 12, 4, 2000, 0.8
    rng = np.random.default_rng(int(100 * top_p) + top_k)
    g = torch.Generator("cuda").manual_seed(1)
    target = 3 * torch.randn(B, n, V, generator=g, device="cuda")
    draft = target + torch.randn(B, n, V, generator=g, device="cuda")
    full = lambda v, t=np.float32: cu(np.full(B * n, v), t)
    f = dict(temperature=full(T), top_k=full(top_k, np.int32), top_p=full(top_p))
    ssm, token = torch.zeros_like(draft), torch.zeros(B * n, dtype=torch.int32, device="cuda")
    api.sample_tokens(token, draft.view(-1, V), cu(rng.random(B * n), np.float32), **f, probs=ssm.view(-1, V))
    kept = torch.zeros_like(target)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sample_tokens(None, target.view(-1, V), **f, kept=kept.view(-1, V), status=status)
    # a chain: node v's token is drawn from the drafter's row at node v - 1
    tokens = np.zeros((B, n), np.int32)
    tokens[:, 1:] = token.view(B, n).cpu().numpy()[:, :-1]
    parent = np.tile(np.arange(-1, n - 1, dtype=np.int32), (B, 1))
    q_row = np.tile(np.arange(-1, n - 1, dtype=np.int32), (B, 1))
    nodes = np.full(B, n, np.int32)
    uni = rng.random((B, 2, n), dtype=np.float32)
    t = api.Tree(B, n)
    api.tree_build(t, cu(tokens), cu(parent), cu(nodes))
    out, path, count = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, n + 1), (B, n + 1), (B,)))
    api.verify_mss(out, path, count, kept, ssm, cu(q_row), cu(uni, np.float32), T, t, status=status)
    assert status.item() == 0
    ref = oracle.verify_mss(kept.cpu().numpy(), ssm.cpu().numpy(), q_row, uni, parent, tokens, nodes, T)
    rows = (kept != api.DROPPED_LOGIT).cpu().numpy()
    for b in range(B):
        c = min(int(ref["lm_pos"][b]), int(ref["count"][b]))
        assert out[b, :c].tolist() == ref["tokens"][b, :c].tolist()
        for i in range(int(count[b])):
            node = int(path[b, i])
            assert rows[b, node, int(out[b, i])], "a token that the target's filter dropped"
    assert int(count.sum()) > B


def test_refused_rows_are_refused_by_the_verifier():
    """A row that cannot be drawn from is NaN, and empties the request that is verified against it."""
    x = torch.zeros(2, 1, 64, device="cuda")
    x[1] = float("nan")
    kept, status = torch.zeros_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sample_tokens(None, x.view(-1, 64), kept=kept.view(-1, 64), status=status)
    assert status.item() == api.STATUS_NONFINITE
    t = api.Tree(2, 1)
    api.tree_build(t, cu([[0], [0]]), cu([[-1], [-1]]), cu([1, 1]))
    out, path, count = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 2), (2, 2), (2,)))
    api.verify_mss(out, path, count, kept, kept, cu([[-1], [-1]]), cu(np.full((2, 2, 1), 0.5), np.float32), 1.0, t)
    assert count.tolist() == [1, 0]
