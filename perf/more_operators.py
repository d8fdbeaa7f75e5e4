"""What is timed and checked of a decode step on the paged cache: one new token a request.

Four operators, in the order a step calls them:

  pages   kv_pages_build          pages from a pool of free ones to requests that grow, back from those that shrink;
                                  block table, and the slot of every new row
  append  kv_append_slots         K and V rows of new tokens (a prompt's, or one a request) into pages by their slots
  decode  decode_attention_paged  attention of one new token a request over its pages, grouped query heads
  sample  sample_tokens           a token a row from logits and a uniform number: temperature, top-k, top-p, min-p; the
                                  filtered distribution or the filtered logits beside it

With `own` false, `run` computes them by elementary torch operations; with `own` true it makes the library's calls.
Lengths follow from the case alone (so the work does), everything else from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE = 64                       # rows of a cache page
DROPPED = -1e30                 # a filtered logit that is not kept


def listed():
    def c(name, op, **kw):
        base = {"pages": {"new": 1, "Pmin": 0, "mix": "decode", "short": False},
                "append": {"d": 128, "prompt": False, "pad": 0},
                "decode": {"d": 128, "Pmin": 0, "empty": False},
                "sample": {"dtype": "f32", "filter": "mixed", "out": "none", "padded": False, "masked": False}}[op]
        return {"name": name, "op": op, **base, **kw}
    return [
        # one new token for each of eight requests in the middle of their contexts: latency
        c("pages_tokens", "pages", B=8, Pmin=1000, P=2048),
        # a batch of long prompts enters an empty cache: slots of some two million rows
        c("pages_prompts", "pages", B=256, new=0, Pmin=512, P=16384, mix="prompts"),
        # the new tokens' rows of the same eight requests, 32 heads
        c("append_tokens", "append", T=8, H=32),
        # a prompt batch of 16384 rows, 32 heads, with padding at its end
        c("append_prompts", "append", T=16384, H=32, prompt=True, pad=100),
        # one request at its start, small grouped heads: latency
        c("decode_start", "decode", B=1, Hq=16, Hk=4, d=64, Pmin=100, P=100),
        # the LLaMA-7B-shaped prefix with grouped heads
        c("decode_gqa", "decode", B=8, Hq=32, Hk=8, Pmin=2048, P=2048),
        # the merge-based layer's ragged prefixes, one key/value head a query head, some requests not started
        c("decode_ragged", "decode", B=16, Hq=32, Hk=32, Pmin=512, P=4096, empty=True),
        # the long-context layer with grouped heads: 4 requests of 64 / 8 heads
        c("decode_long", "decode", B=4, Hq=64, Hk=8, Pmin=16384, P=16384),
        # the OPT-30B-shaped layer: 64 requests of 56 heads over 1024 keys
        c("decode_opt30b", "decode", B=64, Hq=56, Hk=56, Pmin=1024, P=1024),
        # one row of bf16 logits (many equal ones), top-k and top-p: latency
        c("sample_one_bf16", "sample", R=1, V=32000, dtype="bf16", filter="topk"),
        # a batch's rows drawn from the whole distribution, temperature only
        c("sample_temperature", "sample", R=64, V=50272, filter="none"),
        # drafted rows with their filtered distributions, every row with settings of its own, some tokens masked
        c("sample_probs", "sample", R=1024, V=50272, out="probs", masked=True),
    ]


def draw(rng):
    """Sizes between the listed ones, of one of the four operators."""
    logint = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["pages", "append", "decode", "decode", "sample", "sample"])
    if op == "pages":
        P = logint(1, 16384)
        c = {"P": P, "Pmin": max(0, P - logint(1, P + 1)), "new": rng.choice([1, 1, logint(2, 256)]),
             "mix": rng.choice(["decode", "prompts", "mixed", "mixed"]), "short": rng.random() < 0.3}
        c["B"] = logint(1, max(1, min(1024, 2_000_000 // (P + c["new"]))))
    elif op == "append":
        T, d = logint(1, 16384), rng.choice([64, 128])
        c = {"T": T, "d": d, "H": logint(1, max(1, min(64, 16384 * 32 * 128 // (T * d)))), "prompt": rng.random() < 0.5,
             "pad": rng.choice([0, logint(1, 200)])}
    elif op == "decode":
        P, G, Hk = logint(1, 16384), rng.choice([1, 1, 2, 4, 7, 8, 16, 32]), logint(1, 56)
        Hk = max(1, min(Hk, 128 // G))
        c = {"Hk": Hk, "Hq": Hk * G, "d": rng.choice([64, 128, 128]), "P": P, "Pmin": max(0, P - logint(1, P + 1)),
             "empty": rng.random() < 0.2, "B": logint(1, max(1, min(256, 3_000_000 // ((P + PAGE) * Hk * max(1, G // 4)))))}
    else:
        V = logint(200, 160000)
        c = {"V": V, "R": logint(1, max(1, min(2000, 50_000_000 // V))), "dtype": rng.choice(["f32", "f32", "bf16"]),
             "filter": rng.choice(["none", "topk", "topp", "minp", "mixed", "mixed"]),
             "out": rng.choice(["none", "probs", "kept"]), "padded": rng.random() < 0.3, "masked": rng.random() < 0.3}
    return {"op": op, **c}


def _ceil(a, b):
    return (a + b - 1) // b


def _spread(c, b):
    """Row counts from Pmin to P, from the case alone."""
    return c["P"] - (b * 977) % (c["P"] - c["Pmin"] + 1)


def _requests(c):
    """Of a pages case: rows before and after the call, and pages held before it."""
    b = np.arange(c["B"])
    rows = _spread(c, b)
    kind = {"decode": np.zeros_like(b), "prompts": np.ones_like(b), "mixed": (b * 5) % 3}[c["mix"]]
    begin = np.where(kind == 0, rows, 0)
    end = np.where(kind == 0, rows + c["new"], np.where(kind == 1, rows, 0))
    # one in four holds a page more than its rows need, as after a rejected tree; finished requests (kind 2) give all back
    held = np.where(kind == 0, _ceil(rows, PAGE) + (b % 4 == 3), np.where(kind == 1, 0, _ceil(rows, PAGE)))
    return begin.astype(np.int64), end.astype(np.int64), held.astype(np.int64)


def _lengths(c):
    """Keys of every request of a decode case."""
    b = np.arange(c["B"])
    n = _spread(c, b)
    return np.where((b % 5 == 3) & c["empty"], 0, n).astype(np.int64)


def work(c):
    """Every input read once, every output written once; products and sums of the definition."""
    if c["op"] == "pages":
        begin, end, held = _requests(c)
        want = _ceil(end, PAGE)
        moved = int(np.abs(want - held).sum())
        new = int((end - begin).sum())
        # lengths and counts; a slot each row; the pages that the new rows touch; moved ids, read and written
        return {"bytes": 24 * c["B"] + 4 * new + 4 * int((want - begin // PAGE).clip(0).sum()) + 8 * moved, "flops": 0}
    if c["op"] == "append":
        return {"bytes": c["T"] * (c["H"] * c["d"] * 2 * 2 * 2 + 4), "flops": 0}
    if c["op"] == "decode":
        n = int(_lengths(c).sum())
        return {"bytes": n * c["Hk"] * c["d"] * 2 * 2 + 2 * c["B"] * c["Hq"] * c["d"] * 2, "flops": 4 * n * c["Hq"] * c["d"]}
    es = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": c["R"] * c["V"] * (es + (0 if c["out"] == "none" else 4)) + c["R"] * 24, "flops": 4 * c["R"] * c["V"]}


# ------------------------------------------------------------------ inputs ----
def _cu(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).to(DEV)


def _prepare_pages(c, rng, s):
    begin, end, held = _requests(c)
    want = _ceil(end, PAGE)
    takes = int((want - held).clip(0).sum())
    free = takes // 2 if c["short"] else takes + 5
    num = int(held.sum()) + max(free, 1)
    ids = rng.permutation(num)
    table = rng.integers(0, num, (c["B"], int(max(want.max(), held.max(), 1)) + 2)).astype(np.int32)   # stale behind held
    at = 0
    for b, k in enumerate(held):
        table[b, :k], at = ids[at:at + k], at + int(k)
    free_ids = ids[at:at + free]
    head = int(rng.integers(0, num))                      # the ring has been in use: its free part starts anywhere
    ring = rng.integers(0, num, num).astype(np.int32)
    ring[(head + np.arange(len(free_ids))) % num] = free_ids
    s["begin"], s["end"], s["held"] = _cu(begin), _cu(end), _cu(held)
    s["table"], s["ring"], s["state"] = _cu(table), _cu(ring), _cu([head, len(free_ids), 0])
    s["new_held"], s["new_state"] = torch.zeros_like(s["held"]), torch.zeros_like(s["state"])
    s["slot"] = torch.zeros(max(1, int((end - begin).sum())) + 7, dtype=torch.int32, device=DEV)
    s["offset"] = torch.zeros(c["B"] + 1, dtype=torch.int32, device=DEV)


def _prepare_append(c, rng, g, s):
    T, H, d, pad = c["T"], c["H"], c["d"], min(c["pad"], c["T"] - 1)
    if c["prompt"]:                                       # runs of rows in pages of any order, the last ones part full
        pages = _ceil(T, PAGE) + 9
        p = np.repeat(rng.permutation(pages), PAGE)
        start = int(rng.integers(0, PAGE))
        slot = (p * PAGE + np.tile(np.arange(PAGE), pages))[start:start + T]
    else:                                                 # a row each, in pages of its own
        pages = T + 3
        slot = rng.permutation(pages)[:T] * PAGE + rng.integers(0, PAGE, T)
    slot[T - pad:] = -1
    qkv = torch.randn(T, 3 * H, d, generator=g, device=DEV).to(torch.bfloat16)        # one projection's output
    s["k"], s["v"], s["slot"] = qkv[:, H:2 * H], qkv[:, 2 * H:], _cu(slot)
    for name in ("kp", "vp"):
        s[name] = torch.randn(pages, H, PAGE, d, generator=g, device=DEV).to(torch.bfloat16)


def _prepare_decode(c, rng, g, s):
    n, Hk, d = _lengths(c), c["Hk"], c["d"]
    need = _ceil(n, PAGE)
    ids, at = rng.permutation(int(need.sum()) + 3), 0
    table = np.full((c["B"], max(1, int(need.max()))), -1, np.int32)
    for b, k in enumerate(need):
        table[b, :k], at = ids[at:at + k], at + int(k)
    for name in ("kp", "vp"):
        x = torch.empty(len(ids), Hk, PAGE, d, dtype=torch.bfloat16, device=DEV)
        for i in range(0, len(ids), 512):
            y = torch.randn(x[i:i + 512].shape, generator=g, device=DEV)
            if name == "kp":
                y[..., 3] *= 4.0                          # keys have a few strong channels
            x[i:i + 512] = y
        s[name] = x
    qkv = torch.randn(c["B"], c["Hq"] + 2 * Hk, d, generator=g, device=DEV)
    s["q"] = qkv.to(torch.bfloat16)[:, :c["Hq"]]
    s["out"] = torch.zeros(c["B"], c["Hq"], d, dtype=torch.bfloat16, device=DEV)
    s["table"], s["len"] = _cu(table), _cu(n)


def _prepare_sample(c, rng, g, s):
    R, V = c["R"], c["V"]
    wide = _ceil(V, 64) * 64 + 64 if c["padded"] else V
    x = 3.0 * torch.randn(R, wide, generator=g, device=DEV)
    if c["masked"]:                                       # tokens that a grammar forbids, in some of the rows
        forbidden = torch.rand(R, wide, generator=g, device=DEV) < 0.4 * torch.rand(R, 1, generator=g, device=DEV) - 0.1
        forbidden[:, V // 2] = False
        x.masked_fill_(forbidden, -math.inf)
    s["logits"] = x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)[:, :V]
    s["u"] = torch.rand(R, generator=g, device=DEV)
    pick = lambda *a: torch.tensor(a, device=DEV)[torch.randint(len(a), (R,), generator=g, device=DEV)]  # noqa: E731
    f = c["filter"]
    s["temperature"] = pick(0.0, 0.6, 0.8, 1.0, 1.0, 1.3) if f == "mixed" else pick(0.7, 1.0)
    s["top_k"] = (pick(0, 0, 1, 20, 50, 1000, V + 5) if f == "mixed" else pick(50)).to(torch.int32) if f in ("topk", "mixed") else None
    s["top_p"] = pick(0.5, 0.9, 0.95, 0.99, 1.0) if f == "mixed" else pick(0.9) if f in ("topk", "topp") else None
    s["min_p"] = pick(0.0, 0.0, 0.02, 0.1) if f == "mixed" else pick(0.05) if f == "minp" else None
    s["token"] = torch.zeros(R, dtype=torch.int32, device=DEV)
    s["rows"] = None if c["out"] == "none" else torch.zeros(R, V, device=DEV)


def prepare(case, seed):
    """A decode step's tensors as a serving program holds them: the pool's state, projections' output (one buffer whose
    parts are slices), pages and block table, logits and settings a row; with `own` the library's handles."""
    rng, g = np.random.default_rng(seed), torch.Generator(DEV).manual_seed(int(seed))
    c, op = case, case["op"]
    s = {"case": case}
    if op == "pages":
        _prepare_pages(c, rng, s)
    elif op == "append":
        _prepare_append(c, rng, g, s)
    elif op == "decode":
        _prepare_decode(c, rng, g, s)
    else:
        _prepare_sample(c, rng, g, s)
    if own:
        from tree_speculative_verification_gb300 import api
        s["api"] = api
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op == "pages":
            s["pool"] = api.PagePool(s["table"], s["held"], s["ring"], s["state"])
        if op in ("append", "decode"):
            table = s["table"] if op == "decode" else torch.zeros(1, 1, dtype=torch.int32, device=DEV)
            s["kv"] = api.PagedKV(s["kp"], s["vp"], table)
        if op == "decode":
            s["ws"] = api.decode_workspace(c["B"], c["Hq"], c["Hk"], c["d"], DEV)
    return s


# --------------------------------------------------------------- plain form ----
def _plain_pages(s):
    """Counts and running sums over the requests; then every table entry, ring entry and slot by itself."""
    begin, end, held = (s[x].long() for x in ("begin", "end", "held"))
    table, ring, num = s["table"], s["ring"], s["ring"].numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    B, width = table.shape
    want = (end + PAGE - 1) // PAGE
    take = (want - held).clamp_min(0)
    upto = take.cumsum(0)
    ok = (take == 0) | (upto <= count)                    # in order: none gets pages that an earlier one needs
    taken = torch.where(ok, upto, 0).amax()
    back = torch.where(ok, (held - want).clamp_min(0), 0)
    back_at = back.cumsum(0) - back
    p = torch.arange(width, device=DEV)
    got = ok[:, None] & (p >= held[:, None]) & (p < want[:, None])
    source = (head + (upto - take)[:, None] + p - held[:, None]) % num
    given = ok[:, None] & (p >= want[:, None]) & (p < held[:, None])
    target = torch.where(given, (head + count + back_at[:, None] + p - want[:, None]) % num, num)
    ring_out = torch.cat((ring, ring.new_zeros(1)))
    ring_out[target.flatten()] = torch.where(given, table, 0).flatten()
    table.copy_(torch.where(got, ring[source], table))
    ring.copy_(ring_out[:num])
    s["new_held"].copy_(torch.where(ok, want, held))
    s["new_state"][0], s["new_state"][1] = (head + taken) % num, count - taken + back.sum()
    s["offset"][1:] = (end - begin).cumsum(0)
    i = torch.arange(s["slot"].numel(), device=DEV)
    b = (torch.searchsorted(s["offset"].long(), i, right=True) - 1).clamp_max(B - 1)
    r = (begin[b] + i - s["offset"][b]).clamp(0, width * PAGE - 1)
    slot = table[b, r // PAGE].long() * PAGE + r % PAGE
    s["slot"].copy_(torch.where(ok[b] & (i < s["offset"][-1]), slot, -1))
    return _pages_out(s)


def _pages_out(s):
    return {x: s[x] for x in ("table", "ring", "new_held", "new_state", "slot", "offset")}


def _plain_append(s):
    t = (s["slot"] >= 0).nonzero().squeeze(1)
    page, row = s["slot"][t].long() // PAGE, s["slot"][t].long() % PAGE
    s["kp"][page, :, row] = s["k"][t]
    s["vp"][page, :, row] = s["v"][t]
    return {"k": s["kp"], "v": s["vp"]}


def _plain_decode(s):
    c, at = s["case"], s["table"].clamp_min(0).long()
    B, Hq, Hk, d = c["B"], c["Hq"], c["Hk"], c["d"]
    K = s["kp"][at].transpose(1, 2).flatten(2, 3).float()                # [B][Hk][keys][d]
    x = torch.matmul(s["q"].float().reshape(B, Hk, Hq // Hk, d), K.transpose(2, 3)) / math.sqrt(d)
    del K
    hide = torch.arange(x.shape[-1], device=DEV) >= s["len"][:, None]
    x = x.masked_fill(hide[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    V = s["vp"][at].transpose(1, 2).flatten(2, 3).float()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, V) / torch.where(total > 0, total, 1.0)          # no key: zeros
    s["out"].copy_(o.reshape(B, Hq, d))
    return s["out"]


def _plain_sample(s):
    """In 64 bits: a running sum over a vocabulary decides which token's interval a uniform number falls into."""
    c, V = s["case"], s["case"]["V"]
    x, order = s["logits"].float().sort(dim=-1, descending=True, stable=True)   # equal values: the lower id first
    T = s["temperature"].double()[:, None]
    x = x.double()
    rank = torch.arange(V, device=DEV)
    keep = x > -math.inf
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
    if s["min_p"] is not None:
        m = s["min_p"].double()[:, None]
        keep &= (m <= 0) | (x >= x[:, :1] + T * torch.log(m.clamp(1e-300, 1.0)))
    keep &= (T > 0) | (rank < 1)
    w = torch.where(keep, torch.exp((x - x[:, :1]) / torch.where(T > 0, T, 1.0)), 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        keep &= (p >= 1) | (w.cumsum(-1) - w < p * w.sum(-1, keepdim=True)) | (rank < 1)
        w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)                        # by id
    C = w.cumsum(-1)
    token = (C <= s["u"].double()[:, None] * C[:, -1:]).sum(-1)
    last = torch.where(w > 0, rank, 0).amax(-1)
    s["token"].copy_(torch.minimum(token, last))
    if c["out"] == "none":
        return s["token"]
    if c["out"] == "probs":
        s["rows"].copy_(w / C[:, -1:])
    else:
        kept = torch.zeros_like(keep).scatter_(1, order, keep)
        s["rows"].copy_(torch.where(kept, s["logits"].float(), DROPPED))
    return {"token": s["token"], c["out"]: s["rows"]}


# -------------------------------------------------------------- the library ----
def _own(s):
    api, c, op = s["api"], s["case"], s["case"]["op"]
    if op == "pages":
        api.kv_pages_build(s["pool"], s["end"], s["begin"], s["slot"], s["offset"], s["new_held"], s["new_state"], s["status"])
        return _pages_out(s)
    if op == "append":
        api.kv_append_slots(s["kv"], s["k"], s["v"], s["slot"], s["status"])
        return {"k": s["kp"], "v": s["vp"]}
    if op == "decode":
        api.decode_attention_paged(s["out"], s["q"], s["kv"], s["len"], ws=s["ws"], status=s["status"])
        return s["out"]
    probs, kept = (s["rows"] if c["out"] == x else None for x in ("probs", "kept"))
    api.sample_tokens(s["token"], s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], probs, kept,
                      s["status"])
    return s["token"] if c["out"] == "none" else {"token": s["token"], c["out"]: s["rows"]}


def run(state):
    if own:
        return _own(state)
    return {"pages": _plain_pages, "append": _plain_append, "decode": _plain_decode,
            "sample": _plain_sample}[state["case"]["op"]](state)


# ------------------------------------------------- the definition in 64 bits ----
def _exact_row(x, T, k, p, m):
    """How many tokens of one row are kept, in the order of falling values, and that order."""
    order = torch.argsort(-x, stable=True)
    y = x[order]
    n = int((y > -math.inf).sum())
    if T == 0:
        return order, 1
    if k > 0:
        n = min(n, k)
    if m > 0:
        n = min(n, int((y >= float(y[0]) + T * math.log(min(m, 1.0))).sum()))
    if p < 1:
        mass = torch.cat((y.new_zeros(1), torch.softmax(y[:n] / T, 0).cumsum(0)[:-1]))
        n = max(1, int((mass < p).sum()))
    return order, n


def exact(case, seed):
    op = case["op"]
    if op in ("pages", "append"):
        return None                                       # whole numbers, and values that are only moved
    s = prepare(case, seed)
    if op == "decode":
        n, out, G = _lengths(case).tolist(), s["out"].double(), case["Hq"] // case["Hk"]
        for b in range(case["B"]):
            out[b] = 0.0
            if not n[b]:
                continue
            at = s["table"][b, :_ceil(n[b], PAGE)].long()
            for h in range(case["Hk"]):
                K, V = (s[x][at, h].reshape(-1, case["d"])[:n[b]].double() for x in ("kp", "vp"))
                x = s["q"][b, h * G:(h + 1) * G].double() @ K.T * case["d"] ** -0.5
                out[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ V
        return out
    if case["out"] != "probs":
        return None                                       # a token, or logits as they were
    probs = torch.zeros(case["R"], case["V"], dtype=torch.float64, device=DEV)
    get = lambda x, r, off: off if s[x] is None else s[x][r].item()      # noqa: E731
    for r in range(case["R"]):
        T = get("temperature", r, 1.0)
        x = s["logits"][r].double()
        order, n = _exact_row(x, T, get("top_k", r, 0), get("top_p", r, 1.0), get("min_p", r, 0.0))
        probs[r, order[:n]] = torch.softmax(x[order[:n]] / (T or 1.0), 0)
    return {"token": None, "probs": probs}
