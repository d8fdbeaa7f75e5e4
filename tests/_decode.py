"""Shared by the decode step's tests: the pool of pages as a plain list, attention and sampling in 64 bits."""
import math

import numpy as np
import torch

from tree_speculative_verification_gb300 import api

PK = api.PAGE_KEYS


def cu(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


class Pages:
    """The definition of kv_pages_build, one request after the other."""

    def __init__(self, table, held, free, num):
        self.table, self.held, self.free, self.num = np.array(table), list(held), list(free), num

    def build(self, begin, end, max_slots=None):
        B, width = self.table.shape
        free, back, stuck, status = list(self.free), [], False, 0
        slots, offset, ok = [], [0], []
        for b in range(B):
            want, h = -(-int(end[b]) // PK), self.held[b]
            good = 0 <= begin[b] <= end[b] and want <= width and 0 <= h <= width
            status |= 0 if good else api.STATUS_INDEX
            if good and want > h:
                stuck |= want - h > len(free)
                if stuck:
                    good, status = False, status | api.STATUS_NO_PAGES
                else:
                    self.table[b, h:want], free = free[:want - h], free[want - h:]
            elif good:
                back += list(self.table[b, want:h])
            if good:
                self.held[b] = want
            ok.append(good)
            rows = range(begin[b], end[b]) if end[b] > begin[b] else ()
            slots += [int(self.table[b, r // PK]) * PK + r % PK if good else -1 for r in rows]
            offset.append(len(slots))
        self.free = free + [int(x) for x in back]
        if max_slots is not None:
            status |= api.STATUS_INDEX if len(slots) > max_slots else 0
            slots = (slots + [-1] * max_slots)[:max_slots]
        return slots, offset, status


def device_pool(ref, head=0, stale=7):
    """The same pool on the GPU, its free pages from entry `head` of the ring on."""
    ring = np.full(ref.num, stale, np.int32)
    ring[(head + np.arange(len(ref.free))) % ref.num] = ref.free
    return api.PagePool(cu(ref.table), cu(ref.held), cu(ring), cu([head, len(ref.free), 0]))


def free_pages(pool, state=None):
    head, count, done = (pool.state if state is None else state).tolist()
    assert done == 0
    ring = pool.ring.cpu().numpy()
    return [int(x) for x in ring[(head + np.arange(count)) % pool.num_pages]]


class Cache:
    """Pages of random rows for requests of the given lengths, in shuffled order; every row behind them holds NaN."""

    def __init__(self, lens, H, d, seed=0, scale=1.0, extra=2, width=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // PK) for n in lens]
        ids = rng.permutation(sum(need) + extra)
        bt, at = np.full((len(lens), width or max(1, max(need))), -1, np.int32), 0
        g = torch.Generator("cuda").manual_seed(seed)
        self.k, self.v = (torch.full((len(ids), H, PK, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.rows = []
        for b, n in enumerate(lens):
            bt[b, :need[b]], at = ids[at:at + need[b]], at + need[b]
            kv = [(scale * torch.randn(H, n, d, generator=g, device="cuda")).to(torch.bfloat16) for _ in "kv"]
            self.rows.append(kv)
            for j in range(need[b]):
                r = slice(j * PK, min(n, j * PK + PK))
                for x, y in zip((self.k, self.v), kv):
                    x[int(bt[b, j]), :, :r.stop - r.start] = y[:, r]
        self.bt = bt
        self.kv = api.PagedKV(self.k, self.v, cu(bt))


def attention64(q, k, v, scale):
    """fp64 output [Hq][d] of one request's q [Hq][d] over k, v [H][n][d], and the tolerance of each entry.

    The stored output is half a step of bf16 off (2^-8 of it). The rest is fp32: a score of d products is off by at most
    2^-20 of its terms' sum (d + 3 roundings of 2^-24, d <= 128, times log2(e) and scale, two more), which moves its weight by
    that much of itself; a weight entering the sum over v may be rounded to 16 bits (2^-16), and up to 16384 of them are
    summed in at least 64 partial sums (2^-24 a step: 2^-15 at most). A weight error of e moves the normalised output by at
    most 2 e A, A = sum p |v|."""
    H, n, d = k.shape
    G = q.shape[0] // H
    if n == 0:
        return torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    x = q.double().view(H, G, d)
    K, V = k.double(), v.double()
    p = torch.softmax(x @ K.transpose(1, 2) * scale, -1)
    out = p @ V
    off = (2.0 ** -20 * scale * (x.abs() @ K.abs().transpose(1, 2))).amax(-1, keepdim=True)
    tol = 2.0 ** -8 * out.abs() + 2 * (2.0 ** -16 + 2.0 ** -15 + off) * (p @ V.abs()) + 1e-30
    return out.view(q.shape), tol.view(q.shape)


def check_attention(cache, q, out, lens, scale=None):
    d = q.shape[-1]
    for b, n in enumerate(lens):
        ref, tol = attention64(q[b], *cache.rows[b], scale or d ** -0.5)
        got = out[b].double()
        assert torch.isfinite(got).all(), f"request {b}"
        if n == 0:
            assert not got.any(), f"request {b}"
            continue
        worst = float(((got - ref).abs() / tol).max())
        assert worst <= 1.0, f"request {b}: error {worst:.2f} of its tolerance"


# Weights are whole numbers of 2^-36 of the largest, so off by 2^-37 each, as often up as down: 2^18 of them by 2^-26 of the
# largest within four standard deviations. Large ones (from 2^-6 of the largest on) by 2^-38 of themselves more; small ones
# by up to 2^-20 (roundings of an exponent of some 16 and of 2^x), as often up as down: their sum by a standard deviation of
# 2^-21 sqrt(sum w^2) <= 2^-21 sqrt(2^-6 sum w), and as the whole sum is 1 at least, by 2^-22 of that within four of these.
SUM_OFF = 2.0 ** -22


def sample64(x, T, k, p, m):
    """One row's order, weights in it (fp64), and how many are kept (before top-p, after it, and the range that the
    tolerance of sums leaves to the latter)."""
    order = np.argsort(-x.astype(np.float64), kind="stable")
    y = x.astype(np.float64)[order]
    n = int((y > -np.inf).sum())
    if T < 2.0 ** -100:
        return order, np.array([1.0]), 1, (1, 1)
    if k > 0:
        n = min(n, k)
    if m > 0:
        n = min(n, int((y >= y[0] + float(T) * math.log(min(float(m), 1.0))).sum()))
    w = np.exp((y[:n] - y[0]) / float(T))
    lo = hi = n
    if p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        S = w.sum()
        lo = max(1, int((before < (float(p) - SUM_OFF) * S).sum()))
        hi = max(1, int((before < (float(p) + SUM_OFF) * S).sum()))
    return order, w, n, (lo, hi)


def check_sample(logits, u, T, k, p, m, token, probs=None, kept=None):
    """Every row's token, distribution and kept logits against the definition in 64 bits. Rows at numpy float32."""
    R, V = logits.shape
    for r in range(R):
        row = logits[r]
        order, w, n, (lo, hi) = sample64(row, T[r], int(k[r]), p[r], m[r])
        got_n = None
        if probs is not None:
            got_n = int((probs[r] > 0).sum())
            # what underflows fp32 or has no weight in 2^-36 may be kept and read 0
            if not lo <= got_n <= hi:
                q = w[:hi] / w[:hi].sum()
                assert lo > got_n >= int((q > 1e-35).sum()), f"row {r}: {got_n} kept, {lo}..{hi} expected"
                got_n = lo
            ref = np.zeros(V)
            ref[order[:got_n]] = w[:got_n] / w[:got_n].sum()
            # fp32: the exponent's argument is good to 2^-22 of itself at |y| <= 150 by compensation, 2^x to 2^-22, the
            # reciprocal of the sum and the product 2^-23, the sum 2^-22
            err = np.abs(probs[r].astype(np.float64) - ref)
            assert (err <= 2.0 ** -20 * ref + 1e-37).all(), f"row {r}: {err.max()}"
        if kept is not None:
            is_kept = kept[r] != np.float32(api.DROPPED_LOGIT)
            same = order[:lo][row[order[:lo]] == np.float32(api.DROPPED_LOGIT)]
            is_kept[same] = True          # a logit that is DROPPED_LOGIT itself does not show that it is kept
            n2 = int(is_kept.sum())
            assert lo <= n2 <= hi, f"row {r}: {n2} kept, {lo}..{hi} expected"
            assert is_kept[order[:n2]].all() and (kept[r][is_kept] == row[is_kept]).all(), f"row {r}"
            got_n = n2 if got_n is None else got_n
        if token is None:
            continue
        t = int(token[r])
        assert 0 <= t < V, f"row {r}: token {t}"
        ok = False
        for n2 in range(lo, hi + 1) if got_n is None else [got_n]:
            c = np.zeros(V)
            c[order[:n2]] = w[:n2]
            S = c.sum()
            upto = c[:t].sum()
            ok |= c[t] > 0 and upto - SUM_OFF * S <= float(u[r]) * S <= upto + c[t] + SUM_OFF * S
        assert ok, f"row {r}: token {t}"
