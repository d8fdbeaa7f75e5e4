"""sample_tokens against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import check_sample, cu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def run(x, u, T=None, k=None, p=None, m=None, want="token probs kept", stream=None):
    """x [R][V] on the GPU; settings as lists or None."""
    R, V = x.shape
    f = lambda a: None if a is None else cu(a, np.float32)
    out = {"token": torch.full((R,), -9, dtype=torch.int32, device="cuda"), "probs": torch.full((R, V), -9.0, device="cuda"),
           "kept": torch.full((R, V), -9.0, device="cuda")}
    got = {n: t if n in want else None for n, t in out.items()}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sample_tokens(got["token"], x, f(u), f(T), None if k is None else cu(k), f(p), f(m), got["probs"], got["kept"], status)
    return got, status.item()


def check(x, u, T=None, k=None, p=None, m=None, want="token probs kept"):
    R = x.shape[0]
    full = lambda a, v, t=np.float32: np.full(R, v, t) if a is None else np.asarray(a, t)
    got, status = run(x, u, T, k, p, m, want)
    assert status == 0
    n = lambda t: None if t is None else t.cpu().numpy()
    check_sample(x.float().cpu().numpy(), np.asarray(u, np.float32), full(T, 1.0), full(k, 0, np.int64), full(p, 1.0), full(m, 0.0),
                 n(got["token"]), n(got["probs"]), n(got["kept"]))
    return got


def logits(R, V, seed=0, dtype=F32, sigma=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (sigma * torch.randn(R, V, generator=g, device="cuda")).to(dtype)


def uniforms(R, seed=0):
    return np.random.default_rng(seed).random(R, dtype=np.float32)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 256, 1000, 4096, 32000, 50272, 131075, 2 ** 18])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_settings_by_row(V, dtype):
    """Rows of every kind of setting side by side, over vocabularies of all sizes."""
    grid = [(T, k, p, m) for T in (0.0, 0.7, 1.0) for k in (0, 1, 50, V + 3) for p in (1.0, 0.9) for m in (0.0, 0.05)]
    grid += [(1.3, 5, 0.5, 0.3), (0.3, 0, 0.99, 0.0), (1.0, 2000, 0.97, 0.0), (2.0, 3, 1.0, 1.0), (1.0, 0, 0.0, 0.0), (1.0, 0, -1.0, 2.0)]
    if V > 40000:
        grid = grid[::5]
    T, k, p, m = zip(*grid)
    check(logits(len(grid), V, V, dtype), uniforms(len(grid), V), T, k, p, m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V", [(200, 300), (7, 50272), (30, 20011)])
def test_whole_distribution(R, V, dtype):
    x, u = logits(R, V, 1, dtype), uniforms(R, 5)
    check(x, u, want="token")
    check(x, u, T=[0.8] * R, want="token probs")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p", [0.1, 0.6, 0.95, 0.999, 0.9999999])
def test_top_p_alone(p, dtype):
    R, V = 12, 30001
    check(logits(R, V, 2, dtype), uniforms(R), p=[p] * R)
    check(logits(R, V, 2, dtype, 0.01), uniforms(R), p=[p] * R)      # nearly flat: thousands kept
    check(logits(R, V, 2, dtype, 30.0), uniforms(R), p=[p] * R)      # nearly one


@pytest.mark.parametrize("k", [2, 64, 1024, 1025, 5000, 29999, 30000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_top_k_alone(k, dtype):
    """bf16 rows have many equal values where the cut falls: the lowest ids of them stay."""
    R, V = 6, 30001
    check(logits(R, V, 3, dtype), uniforms(R), k=[k] * R)
    check(logits(R, V, 3, dtype), uniforms(R), k=[k] * R, p=[0.8] * R)


@pytest.mark.parametrize("V", [1, 7, 1000, 33333])
def test_all_equal(V):
    """One value: filters keep the lowest ids, and a uniform number falls on id u * kept."""
    R = 9
    x, u = torch.full((R, V), 2.5, device="cuda"), np.arange(R, dtype=np.float32) / R
    k = [0, 0, 3, 1000, V, 1, 0, 0, 17]
    p = [1.0, 0.5, 1.0, 0.25, 0.75, 0.9, 1e-6, 0.999, 0.5]
    got = check(x, u, k=k, p=p)
    for r in range(R):
        n = min(k[r] or V, V)
        n = max(1, math.ceil(n * float(np.float32(p[r])))) if p[r] < 1 else n
        assert int((got["probs"][r] > 0).sum()) == n and int(got["token"][r]) == min(n - 1, int(float(u[r]) * n))


def test_few_values():
    """Rows of a handful of values, each held by thousands of tokens."""
    R, V = 10, 40000
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randint(0, 4, (R, V), generator=g, device="cuda").float()
    for kw in ({"p": [0.3] * R}, {"k": [15000] * R}, {"k": [9000] * R, "p": [0.5] * R}, {"m": [0.3] * R}, {"k": [30000] * R, "p": [0.99] * R}):
        check(x, uniforms(R), **kw)


def test_zeros_of_both_signs_are_equal():
    x = torch.zeros(2, 100, device="cuda")
    x[:, ::2] *= -1.0
    got = check(x, [0.3, 0.99], k=[10, 33])
    assert got["kept"][0, :10].abs().max() == 0 and (got["probs"][1] > 0).nonzero().flatten().tolist() == list(range(33))


def test_far_apart_values():
    """The type's largest and lowest values, and steps between them, at small and large temperatures."""
    top = torch.finfo(F32).max
    row = torch.tensor([top, -top, 0.0, 1e30, -1e30, top, 1.0, -1.0] * 5, device="cuda")
    x = row.repeat(6, 1)
    check(x, uniforms(6), T=[1.0, 1e-6, 1e30, 3e38, 1e-20, 0.0], want="token kept")
    x = torch.linspace(-300, 300, 4000, device="cuda").repeat(5, 1)
    check(x, uniforms(5), T=[1.0, 0.01, 100.0, 1e4, 1e-30])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_tokens(dtype):
    """-inf has no weight: never drawn, not kept, not counted by top-k; one token left; all but the last."""
    R, V = 8, 5000
    x = logits(R, V, 4, dtype)
    x[0, 1:] = -math.inf
    x[1, :-1] = -math.inf
    x[2, ::2] = -math.inf
    x[3, torch.randperm(V, device="cuda")[:V - 20]] = -math.inf
    for kw in ({}, {"k": [50] * R}, {"p": [0.9] * R}, {"k": [3000] * R, "p": [0.99] * R}, {"m": [0.1] * R}, {"T": [0.0] * R}):
        got = check(x, uniforms(R), **kw)
        assert (got["kept"][torch.isinf(x)] == api.DROPPED_LOGIT).all()
        assert got["token"][0] == 0 and got["token"][1] == V - 1


@pytest.mark.parametrize("V", [5, 999, 50272])
def test_rows_that_cannot_be_drawn(V):
    """NaN, +inf, nothing finite: token -1 and NaN rows, the others as ever."""
    R = 6
    x = logits(R, V, 7)
    clean = x.clone()
    x[1, V // 2], x[2, V - 1], x[4] = math.nan, math.inf, -math.inf
    got, status = run(x, uniforms(R), k=[4] * R)
    assert status == api.STATUS_NONFINITE
    ok = [0, 3, 5]
    ref, _ = run(clean, uniforms(R), k=[4] * R)
    for n, t in got.items():
        assert torch.equal(t[ok], ref[n][ok])
    for r in (1, 2, 4):
        assert got["token"][r] == -1 and torch.isnan(got["probs"][r]).all() and torch.isnan(got["kept"][r]).all()


@pytest.mark.parametrize("kw", [{"T": [-1.0]}, {"T": [math.nan]}, {"T": [math.inf]}, {"k": [-1]}, {"p": [math.nan]}, {"m": [math.nan]},
                                {"u": [1.0]}, {"u": [-0.1]}, {"u": [math.nan]}])
def test_settings_out_of_range(kw):
    x = logits(2, 300)
    u = list(uniforms(2))
    kw = dict(kw)
    u[0] = kw.pop("u", u)[0]
    got, status = run(x, u, **{n: a + [1] for n, a in kw.items()})
    assert status == api.STATUS_INDEX and got["token"][0] == -1 and torch.isnan(got["probs"][0]).all()
    assert 0 <= int(got["token"][1]) < 300 and torch.isfinite(got["probs"][1]).all()


@pytest.mark.parametrize("dtype,off,wide", [(F32, 0, 1003), (F32, 1, 1024), (BF16, 0, 1001), (BF16, 3, 1024), (BF16, 8, 1008)])
def test_strided_rows(dtype, off, wide):
    """Rows of a wider projection output, at any alignment; what stands behind them is not read."""
    R, V = 5, 990
    buf = torch.full((R, wide), math.nan, dtype=dtype, device="cuda")
    x = buf[:, off:off + V]
    x.copy_(logits(R, V, 11, dtype))
    check(x, uniforms(R), k=[0, 5, 0, 40, 0], p=[1.0, 0.9, 0.9, 1.0, 0.5])


def test_kept_in_the_logits_place():
    x = logits(20, 3000, 5)
    want, _ = run(x, uniforms(20), k=[30] * 20, p=[0.9] * 20)
    probs, token = torch.zeros_like(x), torch.zeros(20, dtype=torch.int32, device="cuda")
    y = x.clone()
    api.sample_tokens(token, y, cu(uniforms(20), np.float32), top_k=cu([30] * 20), top_p=cu([0.9] * 20, np.float32), probs=probs, kept=y)
    assert torch.equal(y, want["kept"]) and torch.equal(probs, want["probs"]) and torch.equal(token, want["token"])


def test_rows_only():
    x = logits(3, 500)
    got, status = run(x, [0.0] * 3, p=[0.9] * 3, want="probs")
    assert status == 0 and abs(float(got["probs"].sum(-1).sub(1).abs().max())) < 1e-5
    probs = torch.zeros(3, 500, device="cuda")
    api.sample_tokens(None, x, top_p=cu([0.9] * 3, np.float32), probs=probs)
    assert torch.equal(probs, got["probs"])


def test_drawn_as_often_as_its_probability():
    """20000 draws from one row: every token within five standard deviations."""
    n, V = 20000, 40
    row = logits(1, V, 3, sigma=1.5)
    x = row.expand(n, V).contiguous()
    u = (np.arange(n, dtype=np.float32) + 0.5) / n                      # a grid: each token's share to 1 / n
    for kw in ({}, {"k": [7] * n}, {"p": [0.8] * n}):
        got, _ = run(x, u, **kw, want="token probs")
        share = np.bincount(got["token"].cpu().numpy(), minlength=V) / n
        assert np.abs(share - got["probs"][0].double().cpu().numpy()).max() < 2.0 / n + 1e-6


def test_same_results_again_and_in_a_graph():
    x = logits(33, 20000, 5)
    u, p = cu(uniforms(33), np.float32), cu([0.9] * 33, np.float32)
    outs = [(torch.zeros(33, dtype=torch.int32, device="cuda"), torch.zeros_like(x)) for _ in range(3)]
    for t, pr in outs[:2]:
        api.sample_tokens(t, x, u, top_p=p, probs=pr)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        api.sample_tokens(outs[2][0], x, u, top_p=p, probs=outs[2][1])
    graph.replay()
    for t, pr in outs[1:]:
        assert torch.equal(t, outs[0][0]) and torch.equal(pr, outs[0][1])
    u.copy_(cu(uniforms(33, 9), np.float32))
    graph.replay()
    api.sample_tokens(outs[0][0], x, u, top_p=p, probs=outs[0][1])
    assert torch.equal(outs[0][0], outs[2][0])


def test_more_rows_than_a_grid_dimension():
    R, V = 70000, 5
    x, u = logits(R, V, 2), uniforms(R)
    got, status = run(x, u, want="token")
    assert status == 0
    rows = np.random.default_rng(0).integers(0, R, 300)
    one = np.ones(300)
    check_sample(x.cpu().numpy()[rows], u[rows], one, one * 0, one, one * 0, got["token"].cpu().numpy()[rows])
