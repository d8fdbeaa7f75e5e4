"""Shared by the 8-bit cache's GPU tests: trees built by the library, caches of
random rows (dense or in shuffled pages, everything behind the last row
poisoned), and the definitions in 64 bits."""
import math

import numpy as np
import torch

from tree_speculative_verification_gb300 import api

PK = api.PAGE_KEYS
F8 = torch.float8_e4m3fn


def parents(rng, n, depth=12):
    """A random tree: node v's parent is an earlier node of depth below the limit."""
    par, dep = [-1], [0]
    for v in range(1, n):
        ok = [u for u in range(v) if dep[u] < depth]
        u = int(ok[int(rng.integers(0, len(ok)))])
        par.append(u)
        dep.append(dep[u] + 1)
    return np.array(par, np.int32)


class Setup:
    """Trees of the given node counts (0: a request the library rejects) over the given prefixes."""

    def __init__(self, n_nodes, prefix, n_max=None, seed=0):
        rng = self.rng = np.random.default_rng(seed)
        self.n, self.P, self.B = list(n_nodes), list(prefix), len(n_nodes)
        self.n_max = n_max or max(n_nodes)
        par = np.full((self.B, self.n_max), -1, np.int32)
        for b, n in enumerate(self.n):
            par[b, :n] = parents(rng, n) if n else []
        self.par = par
        cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.tree = api.Tree(self.B, self.n_max)
        self.prefix = cu(np.array(self.P, np.int32))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.tree_build(self.tree, cu(np.zeros((self.B, self.n_max), np.int32)), cu(par), cu(np.array(self.n, np.int32)),
                       prefix_len=self.prefix)
        self.dfs, self.depth = self.tree.dfs_of.cpu().numpy(), self.tree.depth.cpu().numpy()

    def randn(self, *shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.from_numpy(self.rng.standard_normal(shape, dtype=np.float32)) * scale).to(dtype).cuda()

    def cache(self, H, d, paged=False, extra=3, rows=None, scale=1.0):
        """A cache whose first P + n rows are random and whose other rows hold NaN codes and scales."""
        L = max(p + n for p, n in zip(self.P, self.n))
        if paged:
            need = [(p + n + PK - 1) // PK for p, n in zip(self.P, self.n)]
            ids = self.rng.permutation(sum(need) + 2)
            bt = np.full((self.B, max(max(need), (self.n_max + PK - 1) // PK)), -1, np.int32)
            at = 0
            for b, k in enumerate(need):
                bt[b, :k], at = ids[at:at + k], at + k
            shape, table = (len(ids), H, PK), torch.from_numpy(bt).cuda()
        else:
            shape, table, bt = (self.B, H, max(L, self.n_max) + extra), None, None
        codes = [torch.full((*shape, d), 0x7f, dtype=torch.uint8, device="cuda").view(F8) for _ in "kv"]
        scales = [torch.full(shape, math.nan, device="cuda") for _ in "kv"]
        kv = api.KV8(*codes, *scales, table)
        kv.bt = bt
        for b in range(self.B):
            m = self.P[b] + self.n[b] if rows is None else rows[b]
            for x, z in zip(codes, scales):
                y, w = quantised(self.randn(H, m, d, dtype=torch.float32, scale=scale)
                                 * torch.exp(0.5 * self.randn(H, m, 1, dtype=torch.float32)))
                put(kv, x, z, b, y, w)
        return kv


def quantised(x):
    """The definition of the codes and scales, in fp32 on the CPU."""
    dev, x = x.device, x.cpu()
    scale = torch.clamp_min(x.abs().amax(-1) / 448.0, 2.0 ** -100)
    y = torch.clamp(x * (1.0 / scale)[..., None], -448.0, 448.0)
    return y.to(F8).to(dev), scale.to(dev)


def put(kv, codes, scales, b, y, w):
    """Rows 0 .. of request b."""
    m = y.shape[1]
    if kv.block_table is None:
        codes.view(torch.uint8)[b, :, :m], scales[b, :, :m] = y.view(torch.uint8), w
        return
    for j in range((m + PK - 1) // PK):
        g, r = int(kv.bt[b, j]), slice(j * PK, min(m, (j + 1) * PK))
        codes.view(torch.uint8)[g, :, :r.stop - r.start] = y.view(torch.uint8)[:, r]
        scales[g, :, :r.stop - r.start] = w[:, r]


def get(kv, b, m):
    """(k codes, v codes, k scales, v scales) of rows 0 .. m - 1 of request b, codes as uint8."""
    out = []
    for x in (kv.k.view(torch.uint8), kv.v.view(torch.uint8), kv.k_scale, kv.v_scale):
        if kv.block_table is None:
            out.append(x[b, :, :m].clone())
        else:
            out.append(torch.cat([x[int(g)] for g in kv.bt[b, :max(1, (m + PK - 1) // PK)]], 1)[:, :m].clone())
    return out


def values(codes, scale):
    return codes.view(F8).double() * scale.double()[..., None]


def norm_rope64(x, weight, pos, rope, d):
    """One projection's heads x [n][H][d] of one request at positions pos [n], in fp64; and |a| + |b| of each output."""
    x = x.double()
    if rope["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + rope["eps"])
        if weight is not None:
            x = x * weight.double()
    mag = x.abs()
    r = rope["rot"]
    if r:
        a = torch.as_tensor(np.asarray(pos, np.float64), device=x.device)[:, None, None] * rope["inv"].double()
        lo, hi = (slice(0, r, 2), slice(1, r, 2)) if rope["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        p, q = x[..., lo].clone(), x[..., hi].clone()
        x, mag = x.clone(), mag.clone()
        x[..., lo], x[..., hi] = p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()
        mag[..., lo] = mag[..., hi] = p.abs() + q.abs()
    return x, mag


def attention64(s, b, q, kv, G, scale):
    """fp64 outputs [n][Hq][d] of request b in input order, and the tolerance of each.

    A stored output is half a step of bf16 off its value (2^-8 of it). The probabilities that meet V may be rounded to
    nine bits (2^-9 of each weight), and a score may be off by what splitting a query into two e4m3 numbers loses: at
    most 2^-17 of its row's largest value in each of the d products, and by fp32 sums (2^-20 of the score's terms).
    With A = sum_j p_j |v_j| a weight error of relative size e moves the normalised output by at most 2 e A."""
    n, P = s.n[b], s.P[b]
    kc, vc, ks, vs = get(kv, b, P + n)
    K, V = values(kc, ks), values(vc, vs)
    d, Hq = K.shape[-1], q.shape[2]
    see = torch.zeros(n, P + n, dtype=torch.bool)
    see[:, :P] = True
    for v in range(n):
        u = v
        while u >= 0:
            see[v, P + int(s.dfs[b, u])] = True
            u = int(s.par[b, u])
    see = see.to(q.device)
    out = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for h in range(Hq):
        x = q[b, :n, h].double()
        k, v = K[h // G], V[h // G]
        S = x @ k.T * scale
        p = torch.softmax(S.masked_fill(~see, -math.inf), -1)
        vz = torch.where(torch.isfinite(v), v, 0.0)
        hit = (see.double() @ (~torch.isfinite(v)).double()) > 0         # a poisoned row is seen
        bad = (see.double() @ (~torch.isfinite(k)).any(-1, keepdim=True).double()) > 0
        pz = torch.where(torch.isfinite(p), p, 0.0)
        out[:, h] = torch.where(hit | bad, math.nan, pz @ vz)
        kz = torch.where(torch.isfinite(k), k, 0.0).abs()
        off = scale * (2.0 ** -17 * x.abs().amax(-1, keepdim=True) * kz.sum(-1) + 2.0 ** -20 * (x.abs() @ kz.T))
        off = off.masked_fill(~see, 0.0).amax(-1, keepdim=True)
        tol[:, h] = 2.0 ** -8 * out[:, h].abs() + 2 * (2.0 ** -9 + off) * (pz @ vz.abs()) + 1e-30
    return out, tol


def check_attention(s, q, kv, out, before, scale=None):
    """Every node's output within its tolerance, every other row as it was."""
    Hq, d = q.shape[2], q.shape[3]
    G = Hq // kv.H
    scale = scale or 1.0 / math.sqrt(d)
    for b in range(s.B):
        n = s.n[b]
        assert torch.equal(out[b, n:], before[b, n:]), f"request {b}: rows behind the last node"
        if not n:
            continue
        ref, tol = attention64(s, b, q, kv, G, scale)
        got = out[b, :n].double()
        nan = torch.isnan(ref)
        assert torch.equal(nan, torch.isnan(got)), f"request {b}: where outputs are NaN"
        err = torch.where(nan, 0.0, (got - ref).abs())
        worst = float((err / torch.where(nan, 1.0, tol)).max())
        assert worst <= 1.0, f"request {b}: error {worst:.2f} of its tolerance"
