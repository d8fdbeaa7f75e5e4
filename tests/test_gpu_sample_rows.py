"""sample_tokens where there are many rows: long ones, which a CTA reads again from L2 (fp32 from some 26000 tokens on, bf16 from
some 52000), and short ones, which a small CTA has."""
import math

import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import check_sample, cu
from test_gpu_sample import BF16, F32, check, logits, run, uniforms

pytestmark = pytest.mark.gpu
LONG = [(F32, 30001), (BF16, 60002)]
MANY = 168     # rows, more than there are SMs


def many(V):
    return MANY if V > 20000 else 680


def check_some(x, u, rows, T=None, k=None, p=None, m=None, want="token probs kept"):
    """All rows are run, some are compared."""
    R = x.shape[0]
    full = lambda a, v, t=np.float32: np.full(R, v, t) if a is None else np.asarray(a, t)
    got, status = run(x, u, T, k, p, m, want)
    assert status == 0
    n = lambda t: None if t is None else t[rows].cpu().numpy()
    check_sample(x[rows].float().cpu().numpy(), np.asarray(u, np.float32)[rows], full(T, 1.0)[rows], full(k, 0, np.int64)[rows],
                 full(p, 1.0)[rows], full(m, 0.0)[rows], n(got["token"]), n(got["probs"]), n(got["kept"]))
    return got


@pytest.mark.parametrize("dtype,V", LONG)
def test_settings_by_row(dtype, V):
    grid = [(T, k, p, m) for T in (0.0, 0.7, 1.0, 2.0) for k in (0, 1, 50, V + 3) for p in (1.0, 0.9, 0.99) for m in (0.0, 0.05)]
    grid += [(1.3, 5, 0.5, 0.3), (1.0, 4095, 0.97, 0.0), (1.0, 4096, 1.0, 0.0), (1.0, 9000, 0.999, 0.001), (2.0, 3, 1.0, 1.0), (1.0, 0, 0.0, 0.0)]
    grid += grid[:MANY - len(grid)]
    T, k, p, m = zip(*grid)
    check(logits(len(grid), V, V, dtype), uniforms(len(grid), V), T, k, p, m)


@pytest.mark.parametrize("V", [131072, 131075, 2 ** 18])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_longest_rows(dtype, V):
    R = MANY
    grid = [(0.8, 0, 1.0, 0.0), (1.0, 50, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 0.995, 0.0), (0.5, 3000, 0.99, 0.0), (1.0, 0, 1.0, 0.02),
            (0.0, 0, 1.0, 0.0), (1.0, 20000, 0.999, 0.0)]
    T, k, p, m = zip(*(grid * (R // len(grid))))
    rows = list(range(8)) + list(range(R - 8, R))
    check_some(logits(R, V, V, dtype), uniforms(R, V), rows, T, k, p, m)


@pytest.mark.parametrize("dtype,V", LONG)
@pytest.mark.parametrize("sigma", [0.01, 3.0, 30.0])
def test_top_p_alone(dtype, V, sigma):
    R = MANY
    check_some(logits(R, V, 2, dtype, sigma), uniforms(R), list(range(0, R, 3)), p=[0.1, 0.6, 0.95, 0.99, 0.999, 0.9999999, 0.3, 0.8] * (R // 8))


@pytest.mark.parametrize("dtype,V", LONG)
def test_top_k_alone(dtype, V):
    R = MANY
    k = [1, 2, 64, 1000, 4095, 4096, 6144, 6145, 20000, V - 1, V, 300, 1500, 2049]
    rows = list(range(28))
    check_some(logits(R, V, 3, dtype), uniforms(R), rows, k=k * 12)
    check_some(logits(R, V, 3, dtype), uniforms(R), rows, k=k * 12, p=[0.8] * R)


def test_equal_values():
    R, V = 180, 33333
    x, u = torch.full((R, V), -7.25, device="cuda"), np.arange(R, dtype=np.float32) / R
    k = [0, 0, 3, 1000, V, 1, 0, 0, 17] * 20
    p = [1.0, 0.5, 1.0, 0.25, 0.75, 0.9, 1e-6, 0.999, 0.5] * 20
    got, status = run(x, u, k=k, p=p)
    assert status == 0
    for r in range(R):
        n = min(k[r] or V, V)
        n = max(1, math.ceil(n * float(np.float32(p[r])))) if p[r] < 1 else n
        assert int((got["probs"][r] > 0).sum()) == n and int((got["kept"][r, :n] == -7.25).sum()) == n
        assert abs(int(got["token"][r]) - min(n - 1, int(float(u[r]) * n))) <= 0


def test_few_values():
    R, V = MANY, 40000
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randint(0, 4, (R, V), generator=g, device="cuda").float()
    for kw in ({"p": [0.3] * R}, {"k": [15000] * R}, {"k": [9000] * R, "p": [0.5] * R}, {"m": [0.3] * R}, {"k": [30000] * R, "p": [0.99] * R}):
        check_some(x, uniforms(R), [0, 7, 50, 99], **kw)


@pytest.mark.parametrize("dtype,V", LONG)
def test_masked_tokens(dtype, V):
    R = MANY
    x = logits(R, V, 4, dtype)
    x[0, 1:] = -math.inf
    x[1, :-1] = -math.inf
    x[2, ::2] = -math.inf
    x[3, torch.randperm(V, device="cuda")[:V - 20]] = -math.inf
    x[4, :V - 7000] = -math.inf
    for kw in ({}, {"k": [50] * R}, {"p": [0.9] * R}, {"p": [0.9999] * R}, {"k": [3000] * R, "p": [0.99] * R}, {"m": [0.1] * R}, {"T": [0.0] * R}):
        got = check_some(x, uniforms(R), list(range(6)), **kw)
        assert (got["kept"][torch.isinf(x)] == api.DROPPED_LOGIT).all()
        assert got["token"][0] == 0 and got["token"][1] == V - 1


@pytest.mark.parametrize("dtype,V", LONG + [(F32, 4001)])
def test_rows_that_cannot_be_drawn(dtype, V):
    R = many(V)
    x = logits(R, V, 7, dtype)
    clean = x.clone()
    x[1, V // 2], x[2, V - 1], x[4], x[150, 0] = math.nan, math.inf, -math.inf, math.nan
    set_p, set_T = [0.9, 1.0] * (R // 2), [1.0] * R
    set_T[9], set_p[10] = -1.0, math.nan
    got, status = run(x, uniforms(R), p=set_p, T=set_T)
    assert status == api.STATUS_NONFINITE | api.STATUS_INDEX
    set_T[9], set_p[10] = 1.0, 0.9
    ref, _ = run(clean, uniforms(R), p=set_p, T=set_T)
    bad = [1, 2, 4, 9, 10, 150]
    ok = [r for r in range(R) if r not in bad]
    for n, t in got.items():
        assert torch.equal(t[ok], ref[n][ok])
    assert (got["token"][bad] == -1).all() and torch.isnan(got["probs"][bad]).all() and torch.isnan(got["kept"][bad]).all()


@pytest.mark.parametrize("dtype,V,off,wide", [(F32, 30001, 1, 30003), (F32, 30002, 2, 30016), (BF16, 60001, 3, 60005), (BF16, 60007, 5, 60016),
                                              (F32, 777, 3, 781), (BF16, 4095, 1, 4097)])
def test_strided_rows(dtype, V, off, wide):
    """Rows at every alignment; what stands around them is not read."""
    R = many(V)
    buf = torch.full((R, wide), math.nan, dtype=dtype, device="cuda")
    x = buf[:, off:off + V]
    x.copy_(logits(R, V, 11, dtype))
    check_some(x, uniforms(R), list(range(16)), k=[0, 5, 0, 40, 0, 0, 700, 0] * (R // 8), p=[1.0, 0.9, 0.9, 1.0, 0.5, 0.999, 0.9, 0.99] * (R // 8))


@pytest.mark.parametrize("V", [30001, 4093, 4096])
def test_kept_in_the_logits_place(V):
    """Each kind of row: nothing dropped, few kept, many kept, one kept, some tokens masked."""
    R = many(V)
    x = logits(R, V, 5)
    x[::16, 7:900] = -math.inf
    k, p, T = [0, 30, 0, 0, 20000, 0, 1, 0] * (R // 8), [1.0, 0.9, 0.9, 0.9999, 0.99, 0.5, 1.0, 0.999] * (R // 8), [1.0, 1.0, 1.0, 1.0, 1.0, 0.0, 1.0, 1e30] * (R // 8)
    want, _ = run(x, uniforms(R), T, k, p)
    for again in range(3):
        y, token = x.clone(), torch.zeros(R, dtype=torch.int32, device="cuda")
        probs = torch.zeros_like(x)
        api.sample_tokens(token, y, cu(uniforms(R), np.float32), cu(T, np.float32), cu(k), cu(p, np.float32), probs=probs, kept=y)
        assert torch.equal(y, want["kept"]) and torch.equal(probs, want["probs"]) and torch.equal(token, want["token"])


@pytest.mark.parametrize("R,V", [(MANY, 30001), (6, 30001), (300, 1000)])
def test_hottest_temperatures(R, V):
    """Temperatures up to the largest number, over logits as far apart as they can be."""
    top = torch.finfo(F32).max
    x = torch.linspace(-top, top, V, device="cuda", dtype=torch.float64).float().repeat(R, 1)
    x[:, ::7] = 0.0
    x[:, 1::7] *= 1e-8
    T = [1e30, 1.3e30, 1e35, 1e37, 1e38, top] * R
    u = uniforms(R)
    check_some(x, u, list(range(6)), T=T[:R])
    check_some(x, u, list(range(6)), T=T[:R], p=[0.9] * R)
    check_some(x, u, list(range(6)), T=T[:R], k=[500] * R, p=[0.5] * R)
    check_some(x, u, list(range(6)), T=T[:R], m=[0.5] * R)


@pytest.mark.parametrize("R,V", [(MANY, 30001), (420, 2000)])
def test_same_results_again_and_in_a_graph(R, V):
    x = logits(R, V, 5)
    u, p, k = cu(uniforms(R), np.float32), cu([0.9, 0.99] * (R // 2), np.float32), cu([0, 0, 400, 5000] * (R // 4))
    outs = [(torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros_like(x)) for _ in range(3)]
    for t, pr in outs[:2]:
        api.sample_tokens(t, x, u, top_k=k, top_p=p, probs=pr)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        api.sample_tokens(outs[2][0], x, u, top_k=k, top_p=p, probs=outs[2][1])
    graph.replay()
    for t, pr in outs[1:]:
        assert torch.equal(t, outs[0][0]) and torch.equal(pr, outs[0][1])


@pytest.mark.parametrize("dtype,V", LONG + [(F32, 3999), (BF16, 4096)])
def test_outputs_alone(dtype, V):
    """Each output asked for alone is the one of all three; token alone is checked against the definition too."""
    R = many(V)
    x, u = logits(R, V, 9, dtype), uniforms(R, 3)
    kw = dict(T=[0.8, 1.0] * (R // 2), k=[0, 0, 40, 5000] * (R // 4), p=([1.0, 0.9, 0.9, 0.99, 0.97] * R)[:R])
    all_of, _ = run(x, u, **kw)
    for name in all_of:
        got, status = run(x, u, want=name, **kw)
        assert status == 0 and torch.equal(got[name], all_of[name])
    check_some(x, u, list(range(20)), want="token", **kw)


def test_rows_do_not_depend_on_one_another():
    """A row's results are the same whatever rows stand beside it: settings in other orders, more rows than are put in order."""
    R, V = 2100, 30001
    x, u = logits(R, V, 6), uniforms(R)
    rng = np.random.default_rng(3)
    kw = dict(T=rng.choice([0.0, 0.7, 1.0, 1.3], R), k=rng.choice([0, 0, 1, 50, 1000, 5000, V], R), p=rng.choice([0.5, 0.9, 0.99, 1.0], R),
              m=rng.choice([0.0, 0.0, 0.05], R))
    whole, status = run(x, u, **kw)
    assert status == 0
    for rows in (slice(0, 700), slice(700, 2100), slice(5, 200), slice(40, 90)):
        got, _ = run(x[rows], u[rows], **{n: v[rows] for n, v in kw.items()})
        for n in whole:
            assert torch.equal(got[n], whole[n][rows])
    back = np.arange(699, -1, -1)
    got, _ = run(x[:700].flip(0), u[back], **{n: v[back] for n, v in kw.items()})
    for n in whole:
        assert torch.equal(got[n].flip(0), whole[n][:700])
