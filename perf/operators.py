"""What is timed and checked of the 8-bit KV cache and of the head norms with rotation.

Five operators of a tree-verification step over a cache that holds e4m3 codes
with one fp32 scale per (row, head):

  rope    tree_qk_norm_rope   RMS norm of every query and key head, and the
                              rotation to position prefix + depth
  append  kv8_append          the same on the way into the cache: keys normed,
                              rotated, quantised; values quantised
  read    kv8_read            cache rows back as bf16 or fp32
  attend  tree_attention_kv8  attention of every tree node to the prefix and to
                              its ancestors, grouped query heads
  commit  kv8_commit          keep the accepted path's rows

With `own` false, `run` computes them by elementary torch operations in fp32;
with `own` true it makes the library's calls. Node counts and prefix lengths
follow from the case alone (so the work does), everything else from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 64                       # rows of a cache page
FP8_MAX, SCALE_MIN = 448.0, 2.0 ** -100
EPS = 1e-6


def listed():
    base = {"B": 1, "n": 1, "ragged": False, "Hq": 32, "Hk": 32, "d": 128, "Pmin": 0, "P": 0, "dtype": "bf16",
            "paged": False, "interleaved": False, "norm": True, "rot": 128}
    c = lambda name, op, **kw: {**base, **kw, "name": name, "op": op}  # noqa: E731
    return [
        # one new token for each of eight requests far into their contexts, fp32, small interleaved heads: latency
        c("rope_tokens_f32", "rope", B=8, Hq=16, Hk=4, d=64, rot=64, Pmin=30000, P=131072, dtype="f32",
          interleaved=True),
        # the OPT-30B-shaped layer's trees: 64 requests of 47 nodes, 56 heads
        c("rope_opt30b", "rope", B=64, n=47, Hq=56, Hk=56, Pmin=1024, P=1024),
        # a few short trees into a paged cache, fp32 projections that are rotated already
        c("append_paged_f32", "append", B=5, n=11, ragged=True, Hq=8, Hk=8, Pmin=3, P=200, dtype="f32", paged=True,
          norm=False, rot=0),
        # the OPT-30B-shaped layer's append with norm and rotation in the same pass
        c("append_opt30b", "append", B=64, n=47, Hq=56, Hk=56, Pmin=100, P=160),
        # one request's pages back in fp32 (a cache moved to another layout)
        c("read_paged_f32", "read", B=1, Hq=8, Hk=8, d=64, Pmin=777, P=777, dtype="f32", paged=True),
        # the merge-based layer's caches back as bf16 (16 ragged requests, 32 heads)
        c("read_merge", "read", B=16, n=25, ragged=True, Pmin=512, P=4096),
        # single-token decoding with grouped heads, the LLaMA-7B-shaped prefix
        c("attend_token_gqa", "attend", B=8, Hq=32, Hk=8, Pmin=2048, P=2048),
        # the OPT-30B-shaped layer: 64 requests of 47 nodes over 1024 keys
        c("attend_opt30b", "attend", B=64, n=47, Hq=56, Hk=56, Pmin=1024, P=1024),
        # ragged trees and prefixes of the merge-based layer, grouped heads, a paged cache
        c("attend_merge_gqa", "attend", B=16, n=25, ragged=True, Hq=32, Hk=8, Pmin=512, P=4096, paged=True),
        # the long-context layer: 4 requests, 128-node trees over 16384 keys, 64 heads
        c("attend_long", "attend", B=4, n=128, Hq=64, Hk=64, Pmin=16384, P=16384),
        # the accepted paths of a few small trees, paged
        c("commit_paged", "commit", B=4, n=21, ragged=True, Hq=8, Hk=8, d=64, Pmin=5, P=120, paged=True),
        # the OPT-30B-shaped layer's commit
        c("commit_opt30b", "commit", B=64, n=47, Hq=56, Hk=56, Pmin=64, P=128),
    ]


def draw(rng):
    """Sizes between the listed ones, of one of the five operators."""
    logint = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["rope", "append", "read", "attend", "attend", "commit"])
    d = rng.choice([64, 128, 128])
    G = rng.choice([1, 1, 2, 4, 7, 8])
    Hk = logint(1, 32)
    n = 1 if rng.random() < 0.25 else logint(2, 128)
    P = logint(1, 131072 if op == "rope" else 16384 if op in ("attend", "read") else 300)
    c = {"op": op, "n": n, "ragged": rng.random() < 0.5, "Hq": Hk * G, "Hk": Hk, "d": d,
         "Pmin": max(0, P - logint(1, P + 1)), "P": P, "dtype": "bf16", "paged": op != "rope" and rng.random() < 0.4,
         "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.75, "rot": rng.choice([0, d // 2, d, d])}
    if op == "rope" and not c["norm"]:
        c["rot"] = c["rot"] or d
    if op in ("rope", "append", "read") and rng.random() < 0.4:
        c["dtype"] = "f32"
    rows = {"rope": n * (Hk + Hk * G), "append": n * (Hk * 2 + Hk * G), "commit": (n + P) * Hk,
            "read": (P + n) * Hk, "attend": max((P + n) * Hk, n * Hk * G)}[op]
    # requests: as many as keep the rows (and, for attention, the products) below the largest listed case
    cap = {"rope": 300_000, "append": 450_000, "commit": 300_000, "read": 700_000, "attend": 3_000_000}[op]
    most = max(1, min(64, cap // max(1, rows)))
    if op == "attend":
        most = max(1, min(most, int(5.0e8 // (n * Hk * G * (P + n)))))
    c["B"] = logint(1, most)
    return c


def _lengths(c):
    """Node counts and prefix lengths, from the case alone."""
    b = np.arange(c["B"])
    n = 1 + (c["n"] - 1 - (b * 5) % c["n"]) if c["ragged"] else np.full(c["B"], c["n"])
    P = c["P"] - (b * 977) % (c["P"] - c["Pmin"] + 1)
    return n.astype(np.int32), P.astype(np.int32)


def work(c):
    """Every input read once, every output written once; products and sums of the definition."""
    n, P = (x.astype(np.int64) for x in _lengths(c))
    N, es, d, Hq, Hk = int(n.sum()), 2 if c["dtype"] == "bf16" else 4, c["d"], c["Hq"], c["Hk"]
    rot = N * d * (8 if c["norm"] or c["rot"] else 0)
    if c["op"] == "rope":
        return {"bytes": N * (Hq + Hk) * d * es * 2, "flops": rot * (Hq + Hk)}
    if c["op"] == "append":
        q = Hq if c["norm"] or c["rot"] else 0
        return {"bytes": N * (2 * q * d * es + 2 * Hk * (d * es + d + 4)), "flops": rot * (q + Hk) + 3 * N * 2 * Hk * d}
    if c["op"] == "read":
        rows = int((n + P).sum()) * Hk * 2
        return {"bytes": rows * (d + 4 + d * es), "flops": rows * d}
    if c["op"] == "attend":
        seen = int((n * P + n * np.minimum(n, 7)).sum())
        return {"bytes": int((n + P).sum()) * Hk * 2 * (d + 4) + 2 * N * Hq * d * es, "flops": 4 * d * Hq * seen}
    kept = int(np.minimum(n, 6).sum())
    return {"bytes": kept * Hk * 2 * (d + 4) * 2, "flops": 0}


# ------------------------------------------------------------------ inputs ----
def _trees(c, rng):
    """Random token trees in depth-first order: node i's parent is the last node before it of one depth less. Input
    ids are a random numbering with the root first."""
    n, P = _lengths(c)
    B, m = c["B"], c["n"]
    W = (m + 31) // 32
    t = {k: np.full((B, m), -1, np.int32) for k in ("perm", "dfs_of", "parent", "token", "depth", "pos", "sub_end")}
    t["n_nodes"], t["prefix"], t["anc"] = n, P, np.zeros((B, m, W), np.uint32)
    path = np.full((B, m + 1), -1, np.int32)
    count = np.zeros(B, np.int32)
    for b in range(B):
        nb = int(n[b])
        depth, last = np.zeros(nb, np.int32), {0: 0}
        par, end, bits = np.full(nb, -1, np.int32), np.full(nb, nb, np.int32), np.zeros((nb, m), bool)
        bits[0, 0] = True
        step = rng.integers(0, 1 << 30, nb)
        for i in range(1, nb):
            depth[i] = 1 + step[i] % min(int(depth[i - 1]) + 1, 12)
            par[i] = last[int(depth[i]) - 1]
            last[int(depth[i])] = i
            bits[i] = bits[par[i]]
            bits[i, i] = True
        for i in range(nb):
            later = np.nonzero(depth[i + 1:] <= depth[i])[0]
            end[i] = i + 1 + int(later[0]) if len(later) else nb
        perm = np.concatenate([[0], 1 + rng.permutation(nb - 1)]).astype(np.int32)
        t["perm"][b, :nb], t["parent"][b, :nb], t["depth"][b, :nb] = perm, par, depth
        t["dfs_of"][b, perm] = np.arange(nb)
        t["sub_end"][b, :nb], t["pos"][b, :nb], t["token"][b, :nb] = end, P[b] + depth, rng.integers(0, 32000, nb)
        full = np.zeros((nb, W * 32), bool)
        full[:, :m] = bits
        t["anc"][b, :nb] = np.packbits(full, axis=1, bitorder="little").view(np.uint32).reshape(nb, W)
        node, up = int(rng.integers(0, nb)), []          # an accepted path: the root down to some node, six at most
        while node >= 0:
            up.append(node)
            node = int(par[node])
        up = up[::-1][:6]
        path[b, :len(up)], count[b] = perm[up], len(up)
    t["anc"] = t["anc"].view(np.int32)
    return {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in {**t, "path": path, "count": count}.items()}


def _block_table(c, rng):
    n, P = _lengths(c)
    need = (n.astype(int) + P + PAGE - 1) // PAGE
    ids, at = rng.permutation(int(need.sum()) + 3), 0
    bt = np.full((c["B"], int(need.max())), -1, np.int32)
    for b, k in enumerate(need):
        bt[b, :k], at = ids[at:at + k], at + k
    return torch.from_numpy(bt).to(DEV), len(ids)


def _quantised(x):
    """e4m3 codes and fp32 scales of fp32 rows."""
    scale = (x.abs().amax(-1) / FP8_MAX).clamp_min(SCALE_MIN)
    y = (x * (1.0 / scale).unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX)
    return y.to(torch.float8_e4m3fn), scale


def _rotary(case, g):
    d, rot = case["d"], case["rot"]
    theta = 10000.0 if case["P"] < 8192 else 500000.0
    inv = (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).to(torch.float32).to(DEV)
    weight = lambda: 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)  # noqa: E731
    return {"inv_freq": inv, "q_weight": weight(), "k_weight": weight()}


def prepare(case, seed):
    """A step's tensors as a serving program holds them: the linearised trees, the projection's output (one buffer
    whose q, k and v are slices), the cache, the output buffers, and with `own` the library's handles."""
    rng, g = np.random.default_rng(seed), torch.Generator(DEV).manual_seed(int(seed))
    c, s = case, {"case": case}
    B, m, Hq, Hk, d, op = c["B"], c["n"], c["Hq"], c["Hk"], c["d"], c["op"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s["tree"] = _trees(c, rng)
    L = c["P"] + m + 3
    if op in ("rope", "append"):
        # heads of differing size, as a projection gives them; attention keys with a few strong channels
        qkv = torch.randn(B, m, Hq + 2 * Hk, d, generator=g, device=DEV)
        qkv *= torch.exp(0.5 * torch.randn(Hq + 2 * Hk, 1, generator=g, device=DEV))
        qkv[..., 3] *= 6.0
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
        s["rope"] = _rotary(c, g)
        s["q_out"] = torch.zeros(B, m, Hq, d, dtype=dt, device=DEV)
        s["k_out"] = torch.zeros(B, m, Hk, d, dtype=dt, device=DEV)
    if op != "rope":
        s["bt"], pages = _block_table(c, rng) if c["paged"] else (None, 0)
        shape = (pages, Hk, PAGE, d) if c["paged"] else (B, Hk, L, d)
        for name in ("k", "v"):
            codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
            scale = torch.empty(shape[:3], device=DEV)
            for i in range(shape[0]):                    # a request or a page at a time: little memory at once
                x = torch.randn(shape[1:], generator=g, device=DEV)
                if name == "k":
                    x[..., 3] *= 6.0
                    x *= 0.8
                else:
                    x *= torch.exp(0.3 * torch.randn(shape[1:3], generator=g, device=DEV)).unsqueeze(-1)
                codes[i], scale[i] = _quantised(x)
            s[name + "c"], s[name + "s"] = codes, scale
    if op == "read":
        s["k_out"] = torch.zeros(B, Hk, L, d, dtype=dt, device=DEV)
        s["v_out"] = torch.zeros(B, Hk, L, d, dtype=dt, device=DEV)
        s["rows"] = s["tree"]["prefix"] + s["tree"]["n_nodes"]
    if op == "attend":
        q = torch.randn(B, m, Hq, d, generator=g, device=DEV)
        q[..., 3] *= 3.0
        s["q"], s["out"] = q.to(dt), torch.zeros(B, m, Hq, d, dtype=dt, device=DEV)
    if op == "commit":
        s["new_prefix"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        from tree_speculative_verification_gb300 import api
        s["api"], t = api, s["tree"]
        s["t"] = api.Tree(B, m, DEV)
        for name in ("n_nodes", "perm", "dfs_of", "parent", "token", "depth", "pos", "sub_end", "anc"):
            getattr(s["t"], name).copy_(t[name])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op in ("rope", "append"):
            r = s["rope"]
            s["r"] = api.QKRope(r["inv_freq"] if c["rot"] else None, r["q_weight"] if c["norm"] else None,
                                r["k_weight"] if c["norm"] else None, eps=EPS, norm=c["norm"],
                                interleaved=c["interleaved"])
        if op != "rope":
            s["kv"] = api.KV8(s["kc"], s["vc"], s["ks"], s["vs"], s["bt"])
        if op == "attend":
            s["ws"] = api.kv8_workspace(B, Hq, Hk, m, d, s["kv"].L_max, DEV)
    return s


# --------------------------------------------------------------- plain form ----
def _norm_rope(x, weight, s):
    """x [B][n][H][d] -> fp32, normed and rotated (angles in 64 bits: positions reach far)."""
    c, t = s["case"], s["tree"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    if c["rot"]:
        pos = t["pos"].gather(1, t["dfs_of"].clamp_min(0).long())        # by input node
        angle = pos.double().unsqueeze(-1) * s["rope"]["inv_freq"].double()
        cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
        r = c["rot"]
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        x = torch.cat((y, x[..., r:]), -1)
    return x


def _nodes(s):
    """[B][n] bool: input ids that are nodes."""
    t = s["tree"]
    return t["dfs_of"] >= 0


def _cache_index(s, b, row):
    """Where cache row `row` of request b is: (strip or page, row in it)."""
    if s["bt"] is None:
        return b, row
    return s["bt"][b, row // PAGE].long(), row % PAGE


def _rows(s, codes, scale):
    """The cache as fp32 [B][Hk][rows][d]."""
    if s["bt"] is not None:
        at = s["bt"].clamp_min(0).long()
        codes, scale = codes.view(torch.uint8)[at], scale[at]            # [B][pages][Hk][PAGE][d]
        codes = codes.transpose(1, 2).flatten(2, 3).view(torch.float8_e4m3fn)
        scale = scale.transpose(1, 2).flatten(2, 3)
    return codes.float() * scale.unsqueeze(-1)


def _plain_rope(s):
    keep = _nodes(s)[:, :, None, None]
    for x, w, out in (("q", "q_weight", "q_out"), ("k", "k_weight", "k_out")):
        y = _norm_rope(s[x], s["rope"][w], s)
        s[out].copy_(torch.where(keep, y.to(s[out].dtype), s[out]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    c, t = s["case"], s["tree"]
    b, v = _nodes(s).nonzero(as_tuple=True)
    page, row = _cache_index(s, b, t["prefix"][b].long() + t["dfs_of"][b, v].long())
    turned = c["norm"] or c["rot"]
    k = _norm_rope(s["k"], s["rope"]["k_weight"], s) if turned else s["k"].float()
    for x, codes, scale in ((k, "kc", "ks"), (s["v"].float(), "vc", "vs")):
        y, z = _quantised(x[b, v])
        s[codes].view(torch.uint8)[page, :, row] = y.view(torch.uint8)
        s[scale][page, :, row] = z
    out = {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if turned:
        q = _norm_rope(s["q"], s["rope"]["q_weight"], s).to(s["q_out"].dtype)
        s["q_out"][b, v] = q[b, v]
        out["q"] = s["q_out"]
    return out


def _plain_read(s):
    for codes, scale, out in (("kc", "ks", "k_out"), ("vc", "vs", "v_out")):
        x = _rows(s, s[codes], s[scale])
        w = min(x.shape[2], s[out].shape[2])
        keep = torch.arange(w, device=DEV)[None, None, :, None] < s["rows"][:, None, None, None]
        s[out][:, :, :w] = torch.where(keep, x[:, :, :w].to(s[out].dtype), s[out][:, :, :w])
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_attend(s):
    c, t = s["case"], s["tree"]
    B, m, Hq, Hk, d = c["B"], c["n"], c["Hq"], c["Hk"], c["d"]
    K, V = _rows(s, s["kc"], s["ks"]), _rows(s, s["vc"], s["vs"])
    L = K.shape[2]
    order = t["perm"].clamp_min(0).long()[:, :, None, None].expand(B, m, Hq, d)
    q = s["q"].gather(1, order).float()                                  # depth-first order
    q = q.view(B, m, Hk, Hq // Hk, d).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, d)
    x = torch.matmul(q, K.transpose(2, 3)).mul_(1.0 / math.sqrt(d))      # [B][Hk][m * G][L]
    del K
    # key j is seen by every node if j < P, else it is tree node j - P, seen by its subtree
    i, j = torch.arange(m, device=DEV), torch.arange(L, device=DEV)
    P, n = t["prefix"][:, None], t["n_nodes"][:, None]
    node = (j[None] - P).clamp(0, m - 1).long()
    end = t["sub_end"].gather(1, node)                                   # [B][L]
    tree = (i[None, :, None] >= node[:, None]) & (i[None, :, None] < end[:, None]) & ((j[None] >= P) & (j[None] < P + n))[:, None]
    see = (tree | (j[None] < P)[:, None]) & (i[None] < n)[:, :, None]    # [B][m][L]
    x = x.view(B, Hk, m, Hq // Hk, L).masked_fill_(~see[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top > -math.inf, top, 0.0)).exp_().view(B, Hk, -1, L)
    o = torch.matmul(p, V) / p.sum(-1, keepdim=True)
    o = o.view(B, Hk, m, Hq // Hk, d).permute(0, 2, 1, 3, 4).reshape(B, m, Hq, d).to(s["out"].dtype)
    b, at = (t["perm"] >= 0).nonzero(as_tuple=True)
    s["out"][b, t["perm"][b, at].long()] = o[b, at]
    return s["out"]


def _plain_commit(s):
    t = s["tree"]
    b, i = (torch.arange(s["case"]["n"] + 1, device=DEV)[None] < t["count"][:, None]).nonzero(as_tuple=True)
    src = t["prefix"][b].long() + t["dfs_of"][b, t["path"][b, i].long()].long()
    sp, sr = _cache_index(s, b, src)
    dp, dr = _cache_index(s, b, t["prefix"][b].long() + i)
    for name in ("kc", "vc"):
        x = s[name].view(torch.uint8)
        x[dp, :, dr] = x[sp, :, sr]
    for name in ("ks", "vs"):
        s[name][dp, :, dr] = s[name][sp, :, sr]
    s["new_prefix"].copy_(t["prefix"] + t["count"])
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"], "prefix": s["new_prefix"]}


# -------------------------------------------------------------- the library ----
def _own(s):
    api, c, t, op = s["api"], s["case"], s["t"], s["case"]["op"]
    if op == "rope":
        api.tree_qk_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["r"], t, s["status"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        if not (c["norm"] or c["rot"]):
            api.kv8_append(s["kv"], s["k"], s["v"], s["tree"]["prefix"], t, status=s["status"])
            return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
        api.kv8_append(s["kv"], s["k"], s["v"], s["tree"]["prefix"], t, s["r"], s["q"], s["q_out"], s["status"])
        return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"], "q": s["q_out"]}
    if op == "read":
        api.kv8_read(s["k_out"], s["v_out"], s["kv"], s["rows"], status=s["status"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        api.tree_attention_kv8(s["out"], s["q"], s["kv"], s["tree"]["prefix"], t, ws=s["ws"], status=s["status"])
        return s["out"]
    api.kv8_commit(s["kv"], s["tree"]["prefix"], s["new_prefix"], s["tree"]["path"], s["tree"]["count"], t, s["status"])
    return {"k": s["kc"], "v": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"], "prefix": s["new_prefix"]}


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "attend": _plain_attend,
            "commit": _plain_commit}[state["case"]["op"]](state)


# ------------------------------------------------- the definition in 64 bits ----
def _exact_head(x, weight, pos, inv, case):
    """One token's heads [H][d] in fp64 by complex rotation."""
    x = x.double()
    if case["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS) * weight.double()
    r = case["rot"]
    if r:
        turn = torch.polar(torch.ones_like(inv, dtype=torch.float64), float(pos) * inv.double())
        head = x[:, :r]
        z = torch.complex(head[:, 0::2], head[:, 1::2]) if case["interleaved"] else torch.complex(head[:, :r // 2], head[:, r // 2:])
        z = z * turn
        y = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat((z.real, z.imag), -1)
        x = torch.cat((y, x[:, r:]), -1)
    return x


def _exact_row(s, name, b, rows):
    """Cache rows 0 .. rows - 1 of request b, fp64 [Hk][rows][d]."""
    codes, scale = s[name + "c"], s[name + "s"]
    if s["bt"] is None:
        return codes[b, :, :rows].double() * scale[b, :, :rows, None].double()
    x = [codes[int(p)].double() * scale[int(p)][..., None].double() for p in s["bt"][b, :-(-rows // PAGE)]]
    return torch.cat(x, 1)[:, :rows]


def exact(case, seed):
    s = prepare(case, seed)
    t, op = s["tree"], case["op"]
    n, P = (x.tolist() for x in _lengths(case))
    if op in ("rope", "append"):
        if case["B"] * case["n"] > 4000:
            return None
        r, pos, dfs = s["rope"], t["pos"].cpu(), t["dfs_of"].cpu()
        turned = case["norm"] or case["rot"]
        q, k = s["q_out"].double(), s["k_out"].double()
        for b in range(case["B"]):
            for v in range(n[b]):
                at = int(pos[b, dfs[b, v]])
                if op == "rope" or turned:
                    q[b, v] = _exact_head(s["q"][b, v], r["q_weight"], at, r["inv_freq"], case)
                k[b, v] = _exact_head(s["k"][b, v], r["k_weight"], at, r["inv_freq"], case) if op == "rope" or turned else s["k"][b, v].double()
        if op == "rope":
            return {"q": q, "k": k}
        # a scale is a number of the definition; a code is whichever neighbour the scaled value rounds to
        ks, vs = s["ks"].double(), s["vs"].double()
        for b in range(case["B"]):
            for v in range(n[b]):
                row = P[b] + int(dfs[b, v])
                page, row = (b, row) if s["bt"] is None else (int(s["bt"][b, row // PAGE]), row % PAGE)
                ks[page, :, row] = (k[b, v].abs().amax(-1) / FP8_MAX).clamp_min(SCALE_MIN)
                vs[page, :, row] = (s["v"][b, v].double().abs().amax(-1) / FP8_MAX).clamp_min(SCALE_MIN)
        out = {"k": None, "v": None, "k_scale": ks, "v_scale": vs}
        return {**out, "q": q} if turned else out
    if op == "read":
        k, v = s["k_out"].double(), s["v_out"].double()
        for b in range(case["B"]):
            k[b, :, :n[b] + P[b]] = _exact_row(s, "k", b, n[b] + P[b])
            v[b, :, :n[b] + P[b]] = _exact_row(s, "v", b, n[b] + P[b])
        return {"k": k, "v": v}
    if op == "attend":
        out, G, parent, perm = s["out"].double(), case["Hq"] // case["Hk"], t["parent"].cpu(), t["perm"].cpu()
        for b in range(case["B"]):
            K, V = (_exact_row(s, x, b, n[b] + P[b]) for x in ("k", "v"))
            see = torch.zeros(n[b], n[b] + P[b], dtype=torch.bool)
            see[:, :P[b]] = True
            for i in range(n[b]):                         # up the tree from i, by the parents
                a = i
                while a >= 0:
                    see[i, P[b] + a] = True
                    a = int(parent[b, a])
            hide = ~see.to(DEV)
            ids = perm[b, :n[b]].long().to(DEV)
            for h in range(case["Hq"]):
                x = s["q"][b, ids, h].double() @ K[h // G].T / math.sqrt(case["d"])
                out[b, ids, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ V[h // G]
        return out
    # commit moves values: an element-wise statement of the moves
    got = {}
    path, dfs = t["path"].cpu(), t["dfs_of"].cpu()
    for name, key in (("ks", "k_scale"), ("vs", "v_scale")):
        x = s[name].double()
        y = x.clone()
        for b in range(case["B"]):
            for i in range(int(t["count"][b])):
                a, z = P[b] + int(dfs[b, path[b, i]]), P[b] + i
                f = (lambda r: (b, r)) if s["bt"] is None else (lambda r: (int(s["bt"][b, r // PAGE]), r % PAGE))  # noqa: B023
                y[f(z)[0], :, f(z)[1]] = x[f(a)[0], :, f(a)[1]]
        got[key] = y
    return {"k": None, "v": None, **got, "prefix": None}
