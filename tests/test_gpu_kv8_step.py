"""The 8-bit cache's calls run together, as a decoding loop uses them: append with norm and rotation, attention, commit,
and reading the cache back, step after step; eagerly, in one captured graph, and in DeviceStep."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api
from tree_speculative_verification_gb300.step import DeviceStep

from _helpers import oracle_tree, workload
from _kv8 import Setup, attention64, check_attention, get, values

pytestmark = pytest.mark.gpu


class Loop:
    """Decoding steps of GQA requests over a growing 8-bit cache. Every step's fused projection rows and tree are drawn
    beforehand; a step accepts the path root, child, child, ... of node 0's first children, up to `take` nodes."""

    def __init__(self, seed, paged, steps=4, Hq=8, Hk=2, d=128):
        rng = np.random.default_rng(seed)
        s = self.s = Setup([9, 1, 17], [61, 0, 130], n_max=17, seed=seed)
        self.Hq, self.Hk, self.d, self.steps = Hq, Hk, d, steps
        B, m = s.B, s.n_max
        self.kv = (api.KV8.paged(B * 4, Hk, d, torch.from_numpy(rng.permutation(B * 4).reshape(B, 4).astype(np.int32)).cuda())
                   if paged else api.KV8.dense(B, Hk, 256, d))
        self.kv.bt = None if not paged else self.kv.block_table.cpu().numpy()
        self.rope = api.QKRope(api.QKRope.frequencies(d, device="cuda"), 1 + 0.1 * s.randn(d, dtype=torch.float32),
                               1 + 0.1 * s.randn(d, dtype=torch.float32))
        self.proj = [s.randn(B, m, Hq + 2 * Hk, d) for _ in range(steps)]
        self.fill = [s.randn(B, m, Hq + 2 * Hk, d) for _ in range(2)]
        self.path, self.count, child = np.full((B, m + 1), -1, np.int32), np.zeros(B, np.int32), None
        for b in range(B):
            v, take = 0, 1 + b
            while v >= 0 and self.count[b] < take:
                self.path[b, self.count[b]] = v
                self.count[b] += 1
                child = np.flatnonzero(s.par[b, :s.n[b]] == v)
                v = int(child[0]) if len(child) else -1
        cu = lambda a: torch.from_numpy(a).cuda()
        self.path, self.count = cu(self.path), cu(self.count)
        self.par, self.nn, self.tokens = cu(s.par), cu(np.array(s.n, np.int32)), cu(np.zeros((B, m), np.int32))
        self.in_proj = torch.zeros_like(self.proj[0])
        self.q_rot = torch.zeros(B, m, Hq, d, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q_rot)
        self.ws = api.kv8_workspace(B, Hq, Hk, m, d, self.kv.L_max)
        self.prefix, self.next = s.prefix.clone(), torch.zeros_like(s.prefix)

    def parts(self):
        x = self.in_proj
        return x[:, :, :self.Hq], x[:, :, self.Hq:self.Hq + self.Hk], x[:, :, self.Hq + self.Hk:]

    def prompt(self):
        """The prefix rows, appended as chains of up to n_max nodes."""
        s, left = self.s, np.array(self.s.P)
        done = np.zeros_like(left)
        while (left > done).any():
            n = np.minimum(left - done, s.n_max).astype(np.int32)
            par = np.tile(np.arange(-1, s.n_max - 1, dtype=np.int32), (s.B, 1))
            at = torch.from_numpy(done.astype(np.int32)).cuda()
            # a finished request keeps one node, written to the row that the next append writes again
            api.tree_build(s.tree, self.tokens, torch.from_numpy(par).cuda(), torch.from_numpy(np.maximum(n, 1)).cuda(),
                           prefix_len=at)
            self.in_proj.copy_(self.fill[int(done.max()) % 2])
            q, k, v = self.parts()
            api.kv8_append(self.kv, k, v, at, s.tree, self.rope, status=s.status)
            done = done + n
        assert s.status.item() == 0

    def append_attend(self):
        s = self.s
        api.tree_build(s.tree, self.tokens, self.par, self.nn, prefix_len=self.prefix)
        q, k, v = self.parts()
        api.kv8_append(self.kv, k, v, self.prefix, s.tree, self.rope, q, self.q_rot, s.status)
        api.tree_attention_kv8(self.out, self.q_rot, self.kv, self.prefix, s.tree, ws=self.ws, status=s.status)

    def commit(self):
        api.kv8_commit(self.kv, self.prefix, self.next, self.path, self.count, self.s.tree, self.s.status)
        self.prefix.copy_(self.next)


@pytest.mark.parametrize("paged", [False, True])
def test_decoding_loop(paged):
    """Each step's attention against 64 bits over the cache as it stands, each commit against the rows before it, the
    cache read back at the end; then the same loop as one replayed graph, bit for bit."""
    a = Loop(21, paged)
    s = a.s
    a.prompt()
    a.prefix.copy_(s.prefix)
    before, outs = a.out.clone(), []
    for t in range(a.steps):
        a.in_proj.copy_(a.proj[t])
        s.P = a.prefix.tolist()
        a.append_attend()
        check_attention(s, a.q_rot, a.kv, a.out, before)
        outs.append(a.out.clone())
        rows = [get(a.kv, b, s.P[b] + s.n[b]) for b in range(s.B)]
        a.commit()
        assert a.prefix.tolist() == [p + int(c) for p, c in zip(s.P, a.count)]
        for b in range(s.B):
            at = list(range(s.P[b])) + [s.P[b] + int(s.dfs[b, v]) for v in a.path[b, :int(a.count[b])].tolist()]
            for x, y in zip(get(a.kv, b, len(at)), rows[b]):
                assert torch.equal(x, y[:, at])
    assert s.status.item() == 0
    end = a.prefix.tolist()
    k, v = (torch.full((s.B, a.Hk, max(end), a.d), 7.0, device="cuda") for _ in "kv")
    api.kv8_read(k, v, a.kv, a.prefix, status=s.status)
    assert s.status.item() == 0
    for b in range(s.B):
        kc, vc, ks, vs = get(a.kv, b, end[b])
        assert torch.equal(k[b, :, :end[b]].double(), values(kc, ks).float().double())
        assert torch.equal(v[b, :, :end[b]].double(), values(vc, vs).float().double())
        assert (k[b, :, end[b]:] == 7.0).all() and (v[b, :, end[b]:] == 7.0).all()

    c = Loop(21, paged)
    c.prompt()
    c.prefix.copy_(s.prefix)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append_attend()
        c.commit()
    for t in range(c.steps):
        c.in_proj.copy_(c.proj[t])
        g.replay()
        assert torch.equal(c.out, outs[t]), f"step {t}"
    assert c.prefix.tolist() == end and c.s.status.item() == 0
    for b in range(s.B):
        assert all(torch.equal(x, y) for x, y in zip(get(a.kv, b, end[b]), get(c.kv, b, end[b])))


@pytest.mark.parametrize("paged,rope", [(False, False), (True, False), (True, True)])
def test_device_step(paged, rope):
    """The merge workload's step over an 8-bit cache: attention against 64 bits over the codes, verification as on the
    bf16 cache, the accepted rows in place."""
    w = workload("merge", 4)
    r = api.QKRope(api.QKRope.frequencies(w.d, device="cuda")) if rope else None
    plain, st = DeviceStep(w), DeviceStep(w, paged=paged, seed=3, kv8=True, rope=r)
    st.kv.bt = None if not paged else st.kv.block_table.cpu().numpy()
    plain.run()
    st.build()
    st.append()
    st.attend()
    par, _, n, _, _ = oracle_tree(w)
    s = SimpleNamespace(B=w.B, n=n.tolist(), P=w.prefix_len.tolist(), dfs=st.tree.dfs_of.cpu().numpy(), par=par)
    out = st.out.clone()
    for b in (0, w.B - 1):
        ref, tol = attention64(s, b, st.q_rot, st.kv, 1, w.d ** -0.5)
        assert ((out[b, :s.n[b]].double() - ref).abs() <= tol).all()
    if rope:
        q = torch.zeros_like(st.q)
        api.tree_qk_norm_rope(q, None, st.q, None, r, st.tree)
        assert torch.equal(q, st.q_rot)
    rows = [get(st.kv, b, s.P[b] + s.n[b]) for b in range(w.B)]
    st.run()
    assert st.status.item() == plain.status.item()
    assert torch.equal(st.out, out)
    assert torch.equal(st.mss_tokens, plain.mss_tokens) and torch.equal(st.new_prefix_len, plain.new_prefix_len)
    npl, path = st.new_prefix_len.tolist(), st.mss_path.cpu().numpy()
    for b in range(w.B):
        at = list(range(s.P[b])) + [s.P[b] + int(s.dfs[b, v]) for v in path[b, :npl[b] - s.P[b]]]
        for x, y in zip(get(st.kv, b, len(at)), rows[b]):
            assert torch.equal(x, y[:, at])


def test_more_requests_than_the_plan_holds():
    """150 requests of ragged lengths, one of them rejected: the units are taken without a plan."""
    rng = np.random.default_rng(5)
    n = rng.integers(1, 12, 150).tolist()
    P = rng.integers(0, 300, 150).tolist()
    P[7], n[9] = 2000, 0
    s = Setup(n, P, seed=5)
    kv = s.cache(2, 128, paged=True)
    q = s.randn(s.B, s.n_max, 4, 128)
    out = torch.full_like(q, 7.0)
    before = out.clone()
    api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, ws=api.kv8_workspace(s.B, 4, 2, s.n_max, 128, kv.L_max),
                           status=s.status)
    torch.cuda.synchronize()
    assert s.status.item() == 0
    check_attention(s, q, kv, out, before)


def test_ragged_lengths_with_joined_parts():
    """One long request among short ones: its axis is cut, its parts joined, whichever block finishes last."""
    s = Setup([33, 4, 1, 20], [9000, 3, 0, 500], seed=6)
    kv = s.cache(2, 64)
    q = s.randn(s.B, s.n_max, 6, 64)
    ws = api.kv8_workspace(s.B, 6, 2, s.n_max, 64, kv.L_max)
    outs = []
    for _ in range(5):
        outs.append(torch.full_like(q, 7.0))
        api.tree_attention_kv8(outs[-1], q, kv, s.prefix, s.tree, ws=ws, status=s.status)
    assert s.status.item() == 0
    assert all(torch.equal(outs[0], x) for x in outs[1:])
    check_attention(s, q, kv, outs[0], torch.full_like(q, 7.0))


def test_one_workspace_for_calls_of_several_sizes():
    """Cut items of few and of many slots, one after another on the workspace of the largest: nothing that one call
    leaves is taken for another's counters."""
    cases = [([1] * 8, [2048] * 8, 32, 8, 128), ([3], [700], 2, 1, 64), ([40, 9], [5000, 1200], 8, 2, 128),
             ([1] * 8, [2048] * 8, 32, 8, 128)]
    setups = []
    for i, (n, P, Hq, Hk, d) in enumerate(cases):
        s = Setup(n, P, seed=30 + i)
        kv = s.cache(Hk, d)
        setups.append((s, kv, s.randn(s.B, s.n_max, Hq, d), api.kv8_workspace(s.B, Hq, Hk, s.n_max, d, kv.L_max)))
    one = torch.zeros(max(w.numel() for *_, w in setups), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for s, kv, q, ws in setups:
            own, shared = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
            api.tree_attention_kv8(own, q, kv, s.prefix, s.tree, ws=ws, status=s.status)
            api.tree_attention_kv8(shared, q, kv, s.prefix, s.tree, ws=one, status=s.status)
            assert torch.equal(own, shared) and s.status.item() == 0
            check_attention(s, q, kv, shared, torch.full_like(q, 7.0))


def test_every_request_rejected():
    s = Setup([0, 0], [5, 9], n_max=4, seed=40)
    kv = api.KV8.dense(2, 2, 64, 128)
    q = s.randn(2, 4, 4, 128)
    out = torch.full_like(q, 7.0)
    ws = api.kv8_workspace(2, 4, 2, 4, 128, 64)
    for _ in range(2):
        api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, ws=ws, status=s.status)
        api.kv8_append(kv, q[:, :, :2].contiguous(), q[:, :, :2].contiguous(), s.prefix, s.tree, status=s.status)
    assert (out == 7.0).all() and (kv.k.view(torch.uint8) == 0).all() and s.status.item() == 0


def test_offsets_past_32_bits():
    """Two requests of four heads whose second codes lie past 2^32 bytes: append, attention, commit and read there are
    those of a small cache."""
    rows, H, d = (1 << 32) // (4 * 128) + 4096, 4, 128
    s = Setup([20, 20], [300, 300], seed=50)
    k, v = s.randn(2, 20, H, d), s.randn(2, 20, H, d)
    q = s.randn(2, 20, 8, d)
    path = torch.full((2, 21), -1, dtype=torch.int32, device="cuda")
    path[:, 0], count = 0, torch.ones(2, dtype=torch.int32, device="cuda")
    far = torch.tensor([rows - 20, rows - 20], dtype=torch.int32, device="cuda")
    small = s.cache(H, d)
    got = []
    for L in (small.L_max, rows):
        kv = api.KV8.dense(2, H, L, d)
        for x, y in ((kv.k, small.k), (kv.v, small.v)):
            x.view(torch.uint8)[:, :, :300] = y.view(torch.uint8)[:, :, :300]
        kv.k_scale[:, :, :300], kv.v_scale[:, :, :300] = small.k_scale[:, :, :300], small.v_scale[:, :, :300]
        out, new = torch.zeros_like(q), torch.zeros_like(s.prefix)
        api.kv8_append(kv, k, v, s.prefix, s.tree, status=s.status)
        ws = api.kv8_workspace(2, 8, H, 20, d, L)
        api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, ws=ws, status=s.status)
        api.kv8_commit(kv, s.prefix, new, path, count, s.tree, status=s.status)
        ko, vo = (torch.zeros(2, H, 320, d, device="cuda") for _ in "kv")
        api.kv8_read(ko, vo, kv, s.prefix + 20, status=s.status)
        got.append([out, new, ko, vo])
        if L == rows:   # the cache's last rows
            api.kv8_append(kv, k, v, far, s.tree, status=s.status)
            kf, vf = (torch.zeros(2, H, 20, d, device="cuda") for _ in "kv")
            api.kv8_read(kf, vf, kv, far + 20, far, status=s.status)
            assert torch.equal(kf, ko[:, :, 300:]) and torch.equal(vf, vo[:, :, 300:])
    assert s.status.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][2][:, :, :320] != 0).any(-1).all()


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, over one cache."""
    s = Setup([12, 30, 7], [900, 2500, 64], seed=60)
    kv = s.cache(2, 128)
    q = [s.randn(3, 30, 8, 128) for _ in range(2)]
    ws = [api.kv8_workspace(3, 8, 2, 30, 128, kv.L_max) for _ in range(2)]
    want, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        want.append(torch.full_like(q[i], 7.0))
        api.tree_attention_kv8(want[i], q[i], kv, s.prefix, s.tree, ws=ws[i], status=s.status)
    got = [[torch.full_like(q[i], 7.0) for _ in range(8)] for i in range(2)]
    torch.cuda.synchronize()
    for r in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                api.tree_attention_kv8(got[i][r], q[i], kv, s.prefix, s.tree, ws=ws[i], status=s.status)
    torch.cuda.synchronize()
    assert s.status.item() == 0
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unrotated_values_keep_to_themselves(dtype):
    """Without the norm, an infinity behind the rotated part stays in its place, and one inside reaches its pair only."""
    s = Setup([5], [3], seed=70)
    rope = api.QKRope(api.QKRope.frequencies(64, device="cuda"), norm=False)
    q = s.randn(1, 5, 3, 128, dtype=dtype)
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    api.tree_qk_norm_rope(want, None, q, None, rope, s.tree)
    q[0, 2, 1, 70], q[0, 3, 0, 7] = float("inf"), float("-inf")
    api.tree_qk_norm_rope(got, None, q, None, rope, s.tree)
    assert got[0, 2, 1, 70] == float("inf") and not torch.isfinite(got[0, 3, 0, 7]) and not torch.isfinite(got[0, 3, 0, 39])
    want[0, 2, 1, 70] = want[0, 3, 0, 7] = want[0, 3, 0, 39] = 0
    got[0, 2, 1, 70] = got[0, 3, 0, 7] = got[0, 3, 0, 39] = 0
    assert torch.equal(want, got)
