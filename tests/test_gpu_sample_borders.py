"""sample_tokens where u and top_p are the fp32 numbers next to borders of the sums in 64 bits: tokens and cuts are equal to
the definition's, whichever layout the sizes choose. What 64 bits themselves leave open (1e-13 of the sum) is left out."""
import math

import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import cu
from test_gpu_sample import BF16, F32, run

pytestmark = pytest.mark.gpu
OPEN = 1e-13

#: rows, vocabulary, type, and filters that do not filter (they choose between a cluster and a CTA a row)
LAYOUTS = [(300, 50272, F32, {}), (60, 50272, F32, {}), (7, 32000, BF16, {}), (2000, 4001, F32, {}), (600, 300, F32, {}), (2000, 2000, BF16, {}),
           (320, 30001, F32, {"m": 0.0}), (320, 60002, BF16, {"k": 0})]


def row_of(V, dtype, kind, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(V, generator=g, device="cuda")
    x = {"normal": 3.0 * x, "flat": 0.05 * x, "peaked": 8.0 * x, "steps": (2.0 * x).round(), "offset": 3.0 * x - 1000.0}[kind]
    if kind == "peaked":
        x[V // 3] = 40.0
    return x.to(dtype)


def definition(x, T, k, m):
    """Order, weights in it and their running sums, of one row under top-k and min-p."""
    y = x.double().cpu().numpy()
    order = np.argsort(-y, kind="stable")
    z = y[order]
    n = len(z) if k <= 0 else min(len(z), k)
    if m > 0:
        n = min(n, int((z >= z[0] + float(T) * math.log(float(m))).sum()))
    w = np.exp((z[:n] - z[0]) / float(T)).astype(np.longdouble)
    return order, w, np.concatenate(([0.0], np.cumsum(w)))


def near(values, R, rng):
    """fp32 numbers in [0, 1) next to R of the values: the nearest, the one below or above it."""
    u = rng.choice(values, R).astype(np.float64).astype(np.float32)
    u = np.where(np.arange(R) % 3 == 1, np.nextafter(u, np.float32(0)), np.where(np.arange(R) % 3 == 2, np.nextafter(u, np.float32(1)), u))
    return np.clip(u, 0, np.float32(1 - 2.0 ** -24)).astype(np.float32)


def drawn(order, w, V, u):
    """The token of every u, and whether 64 bits tell."""
    ids = np.sort(order[:len(w)])
    by_id = np.zeros(V, np.longdouble)
    by_id[order[:len(w)]] = w
    C = np.cumsum(by_id[ids])
    C /= C[-1]
    u = u.astype(np.longdouble)
    at = np.searchsorted(C, u, side="right")
    gap = np.minimum(C[at] - u, np.where(at > 0, u - C[np.maximum(at - 1, 0)], 1.0))   # (before the first token there is no border)
    return ids[at], gap > OPEN


@pytest.mark.parametrize("R,V,dtype,none", LAYOUTS)
@pytest.mark.parametrize("kind", ["normal", "flat", "peaked", "steps", "offset"])
@pytest.mark.parametrize("kw", [{}, {"T": 0.6}, {"T": 1.3}, {"k": 50}, {"m": 0.01}, {"k": 1000}, {"k": 200, "m": 0.02}])
def test_token(R, V, dtype, none, kind, kw):
    x, rng = row_of(V, dtype, kind, V), np.random.default_rng(V + len(kind))
    T, k, m = np.float32(kw.get("T", 1.0)), kw.get("k", 0), np.float32(kw.get("m", 0.0))
    order, w, upto = definition(x, T, k, m)
    by_id = np.zeros(V, np.longdouble)
    by_id[order[:len(w)]] = w
    u = near(np.cumsum(by_id) / upto[-1], R, rng)
    want, sure = drawn(order, w, V, u)
    args = {n: [v] * R for n, v in {**none, **kw}.items()}
    got, status = run(x.expand(R, V).contiguous(), u, **args, want="token")
    assert status == 0 and sure.mean() > (0.2 if kind == "peaked" or dtype is BF16 else 0.99)   # (few borders, or some at u itself)
    token = got["token"].cpu().numpy()
    assert (token[sure] == want[sure]).all(), f"{(token != want)[sure].sum()} of {sure.sum()} rows"


@pytest.mark.parametrize("R,V,dtype,none", LAYOUTS)
@pytest.mark.parametrize("kind", ["normal", "flat", "peaked", "steps", "offset"])
@pytest.mark.parametrize("kw", [{}, {"T": 0.6}, {"k": 400}, {"k": 2000}, {"m": 0.001}])
def test_cut_of_top_p(R, V, dtype, none, kind, kw):
    """Kept logits, and the token that is drawn of them."""
    x, rng = row_of(V, dtype, kind, V + 1), np.random.default_rng(V + len(kind))
    T, k, m = np.float32(kw.get("T", 1.0)), kw.get("k", 0), np.float32(kw.get("m", 0.0))
    order, w, upto = definition(x, T, k, m)
    share = upto[:-1] / upto[-1]
    p = near(share[len(share) > 1:], R, rng)
    p = np.maximum(p, np.float32(1e-7))
    before = np.searchsorted(share, p.astype(np.longdouble), side="left")          # of those with less than p before them
    n = np.maximum(before, 1)
    gap = np.minimum(np.abs(share[np.minimum(before, len(share) - 1)] - p), np.abs(share[before - 1] - p))
    sure = (gap > OPEN) | (before == len(share))
    u = rng.random(R, dtype=np.float32)
    args = {name: [v] * R for name, v in {**none, **kw}.items()}
    got, status = run(x.expand(R, V).contiguous(), u, **args, p=p, want="token kept")
    assert status == 0 and sure.mean() > (0.2 if kind == "peaked" or dtype is BF16 else 0.99)
    kept = (got["kept"] != -1e30).cpu().numpy()
    count = kept.sum(1)
    assert (count[sure] == n[sure]).all(), f"{(count != n)[sure].sum()} of {sure.sum()} rows"
    token = got["token"].cpu().numpy()
    for r in np.flatnonzero(sure)[:40]:
        assert kept[r, order[:n[r]]].all()
        want, told = drawn(order, w[:n[r]], V, u[r:r + 1])
        assert token[r] == want[0] or not told[0], f"row {r}"


@pytest.mark.parametrize("R,V,dtype,none", LAYOUTS)
def test_cut_and_token_at_once(R, V, dtype, none):
    """u next to borders of what top_p next to a border keeps."""
    x, rng = row_of(V, dtype, "normal", V + 2), np.random.default_rng(V)
    order, w, upto = definition(x, np.float32(1.0), 0, 0.0)
    share = upto[:-1] / upto[-1]
    p = np.maximum(near(share[1:], R, rng), np.float32(1e-7))
    u, want, sure = np.zeros(R, np.float32), np.zeros(R, np.int64), np.zeros(R, bool)
    for r in range(0, R, max(1, R // 100)):
        before = int(np.searchsorted(share, np.longdouble(p[r]), side="left"))
        gap = min(abs(share[min(before, V - 1)] - p[r]), abs(share[before - 1] - p[r]))
        n = max(1, before)
        by_id = np.zeros(V, np.longdouble)
        by_id[order[:n]] = w[:n]
        u[r:r + 1] = near(np.cumsum(by_id) / upto[n], 1, rng)
        t, told = drawn(order, w[:n], V, u[r:r + 1])
        want[r], sure[r] = t[0], told[0] and gap > OPEN
    got, status = run(x.expand(R, V).contiguous(), u, p=p, **{name: [v] * R for name, v in none.items()}, want="token")
    assert status == 0
    token = got["token"].cpu().numpy()
    assert (token[sure] == want[sure]).all()


def test_smallest_numbers():
    """u = 0 is the first kept token, however light; so it is where the first ones have no weight in fp32."""
    for R, V, none in ((4, 1000, {}), (3, 50272, {}), (170, 30001, {"m": 0.0})):
        x = -torch.full((R, V), 30.0, device="cuda")
        x[:, V // 2] = 0.0
        x[:, :5] = -math.inf
        got, status = run(x, [0.0] * R, **{n: [v] * R for n, v in none.items()}, want="token")
        assert status == 0 and (got["token"] == 5).all()


@pytest.mark.parametrize("R,V,none", [(3, 2 ** 18, {}), (160, 2 ** 17, {"m": 0.0}), (5, 50272, {}), (700, 1000, {})])
@pytest.mark.parametrize("low", [-22.0, -25.3, -27.7])
def test_cut_in_a_flat_tail(R, V, none, low):
    """One token and V - 1 others of 2^-32 to 2^-40 of it each, all alike: top_p ends between some of them, thousands of tokens
    from where weights of few bits would end it."""
    x = torch.full((R, V), low, device="cuda")
    x[:, V // 3] = 0.0
    w = math.exp(low)
    S = 1.0 + (V - 1) * w
    p = np.float32(1.0) - (1 + np.arange(R) % 6).astype(np.float32) * np.float32(2.0 ** -24)
    n = [max(1, 1 + math.ceil((float(v) * S - 1.0) / w)) if float(v) * S > 1.0 else 1 for v in p]
    got, status = run(x, [0.999999] * R, p=p, **{name: [v] * R for name, v in none.items()}, want="kept")
    assert status == 0
    count = (got["kept"] != -1e30).sum(1).cpu().numpy()
    open_ = math.ceil(2.0 ** -43 * S / w)      # tokens by which 64 bits may be off
    assert (np.abs(count - np.asarray(n)) <= open_).all(), (count[:6], n[:6])


@pytest.mark.parametrize("R,V,none", [(3, 50272, {}), (200, 30001, {"m": 0.0}), (700, 1000, {}), (40, 3000, {})])
@pytest.mark.parametrize("T,low,high", [(1e-6, 9.9999, 10.0), (1e-7, 3.0, 3.000002), (1e-4, -512.0, -511.99), (1e-30, 1.0, 1.0), (3e4, -1e5, 3e5),
                                        (1e30, -3e30, 2e30), (2e31, -1e32, 3e31), (1e37, -3e38, 3e38), (3e38, -3e38, 3e38)])
def test_coldest_and_hottest_temperatures(R, V, none, T, low, high):
    """Temperatures that logits are millions of times, and those near the largest number."""
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.uniform(low, high, V).astype(np.float32)).cuda()
    x[V // 2] = high
    T = np.float32(T)
    order, w, upto = definition(x, T, 0, 0.0)
    w = w[w > 0]                                             # (what 64 bits have no weight for)
    u = near(np.cumsum(np.bincount(order[:len(w)], weights=w.astype(np.float64), minlength=V)) / float(w.sum()), R, rng)
    want, sure = drawn(order, w, V, u)
    X, full = x.expand(R, V).contiguous(), {name: [v] * R for name, v in none.items()}
    got, status = run(X, u, T=[T] * R, **full, want="token")
    token = got["token"].cpu().numpy()
    assert status == 0 and (token[sure] == want[sure]).all(), f"{(token != want)[sure].sum()} of {sure.sum()} rows"
    share = np.concatenate(([0.0], np.cumsum(w)[:-1])) / w.sum()
    p = np.maximum(near(share, R, rng), np.float32(1e-7))
    before = np.searchsorted(share, p.astype(np.longdouble), side="left")
    gap = np.minimum(np.abs(share[np.minimum(before, len(share) - 1)] - p), np.abs(share[before - 1] - p))
    told = (gap > OPEN) | (before == len(share))
    got, status = run(X, rng.random(R, dtype=np.float32), T=[T] * R, p=p, **full, want="kept")
    count = (got["kept"] != -1e30).sum(1).cpu().numpy()
    # (where the border is the last one that has a weight in 64 bits, tokens without one are kept or not)
    told &= before < len(share)
    assert status == 0 and (count[told] == np.maximum(before, 1)[told]).all()


@pytest.mark.parametrize("R,V,dtype,none", LAYOUTS)
def test_all_outputs_of_rows_at_a_border(R, V, dtype, none):
    """u and top_p next to borders: distributions and kept logits are those of the cut that is kept, each output alone too."""
    x, rng = row_of(V, dtype, "normal", V + 3), np.random.default_rng(V)
    order, w, upto = definition(x, np.float32(1.0), 0, 0.0)
    share = upto[:-1] / upto[-1]
    p = np.maximum(near(share[1:], R, rng), np.float32(1e-7))
    by_id = np.zeros(V, np.longdouble)
    by_id[order] = w
    u = near(np.cumsum(by_id) / upto[-1], R, rng)
    X, kw = x.expand(R, V).contiguous(), {"p": p, **{name: [v] * R for name, v in none.items()}}
    got, status = run(X, u, **kw)
    assert status == 0
    kept = (got["kept"] != -1e30).cpu().numpy()
    count, probs = kept.sum(1), got["probs"].cpu().numpy().astype(np.float64)
    for r in range(0, R, max(1, R // 40)):
        ref = np.zeros(V)
        ref[order[:count[r]]] = w[:count[r]] / upto[count[r]]
        assert kept[r, order[:count[r]]].all() and (np.abs(probs[r] - ref) <= 2.0 ** -20 * ref + 1e-37).all()
        assert kept[r, int(got["token"][r])]
    for name in got:
        alone, _ = run(X, u, want=name, **kw)
        assert torch.equal(alone[name], got[name])


@pytest.mark.parametrize("R,V,none", [(60, 50272, {}), (320, 30001, {"m": 0.0}), (2000, 2000, {})])
def test_kept_in_the_logits_place_at_a_border(R, V, none):
    """The row is weighed once more although the kept logits go where it was."""
    x, rng = row_of(V, F32, "normal", V + 4), np.random.default_rng(V)
    order, w, upto = definition(x, np.float32(1.0), 0, 0.0)
    share = upto[:-1] / upto[-1]
    by_id = np.zeros(V, np.longdouble)
    by_id[order] = w
    X, u = x.expand(R, V).contiguous(), near(np.cumsum(by_id) / upto[-1], R, rng)
    for p in (np.full(R, 1.0, np.float32), np.maximum(near(share[1:], R, rng), np.float32(1e-7))):
        f = lambda a: cu(a, np.float32)
        m = f([0.0] * R) if none else None
        want, _ = run(X, u, p=p, m=[0.0] * R if none else None)
        y, token = X.clone(), torch.zeros(R, dtype=torch.int32, device="cuda")
        api.sample_tokens(token, y, f(u), top_p=f(p), min_p=m, kept=y)
        assert torch.equal(y, want["kept"]) and torch.equal(token, want["token"])
