"""decode_attention_paged over values of the type's largest numbers, infinities and NaN, at keys of every weight down to none."""
import math

import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import Cache, cu

pytestmark = pytest.mark.gpu
LARGEST = torch.finfo(torch.bfloat16).max


def run(lens, Hq, Hk, d, far, every, value, seed=0):
    """Keys whose score is that of their first dim alone (scale 1): -0.5 (j % 5), but `far` at every j with every(j), and there
    the first half of the value row is `value`. Out, and for every request out in 64 bits and its tolerance."""
    cache = Cache(lens, Hk, d, seed)
    refs = []
    for b, n in enumerate(lens):
        k, v = cache.rows[b]
        j = torch.arange(n, device="cuda")
        s = torch.where(every(j), far, -0.5 * (j % 5)).to(torch.bfloat16)
        k.zero_()
        k[:, :, 0] = s
        v[:, every(j), :d // 2] = value
        for page in range(-(-n // 64)):
            rows = slice(page * 64, min(n, page * 64 + 64))
            for x, y in ((cache.k, k), (cache.v, v)):
                x[int(cache.bt[b, page]), :, :rows.stop - rows.start] = y[:, rows]
        # A score is one product, exact, and two roundings of its exponent (2^-24 each); the rest as in attention64()
        s, V = s.double(), v.double()
        p = torch.softmax(s, 0)
        out = torch.einsum("j,hjd->hd", p, V)
        tol = 2.0 ** -8 * out.abs() + torch.einsum("j,hjd->hd", p * (2 * (2.0 ** -16 + 2.0 ** -15) + 2.0 ** -22 * s.abs()), V.abs()) + 1e-30
        refs.append([x.repeat_interleave(Hq // Hk, 0) for x in (out, tol)])
    q = torch.zeros(len(lens), Hq, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    out = torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.decode_attention_paged(out, q, cache.kv, cu(lens), 1.0, api.decode_workspace(len(lens), Hq, Hk, d), status)
    assert status.item() == 0
    return out.double(), refs


def third(j):
    return j % 3 == 1


def second(j):
    return j == 2


SHAPES = [([100], 4, 1, 64), ([100, 37, 300], 16, 2, 128), ([700] * 40, 8, 8, 64), ([5000], 20, 1, 128)]


@pytest.mark.parametrize("lens,Hq,Hk,d", SHAPES)
@pytest.mark.parametrize("far", [-110.0, -200.0, -1e4, -3e38])
@pytest.mark.parametrize("value", [LARGEST, -LARGEST, 1e36])
def test_no_weight_and_the_largest_values(lens, Hq, Hk, d, far, value):
    """Keys so far below that fp32 has no weight for them: what they hold does not show (e^-110 of 3e38 is 6e-10)."""
    out, ref = run(lens, Hq, Hk, d, far, third, value)
    for b in range(len(lens)):
        want, tol = ref[b]
        assert ((out[b] - want).abs() <= tol + 2e-6).all()


@pytest.mark.parametrize("lens,Hq,Hk,d", SHAPES)
@pytest.mark.parametrize("far", [-20.0, -60.0, -75.0, -83.0])
def test_small_weights_and_the_largest_values(lens, Hq, Hk, d, far):
    """Weights down to 2^-120 count as what they are (2^-133 more at most: 2^-13 of them)."""
    out, ref = run(lens, Hq, Hk, d, far, second, LARGEST)
    for b in range(len(lens)):
        want, tol = ref[b]
        assert ((out[b] - want).abs() <= tol + 2.0 ** -13 * want.abs()).all()


@pytest.mark.parametrize("lens,Hq,Hk,d", SHAPES)
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("at", [0.0, -0.5, -3.0, -40.0, -70.0])
def test_infinite_values(lens, Hq, Hk, d, value, at):
    """An infinite value of a key that has a weight is the output; the other dims are as ever."""
    out, ref = run(lens, Hq, Hk, d, at, second, value)
    for b in range(len(lens)):
        assert (out[b][:, :d // 2] == value).all()
        want, tol = ref[b]
        assert torch.isfinite(out[b][:, d // 2:]).all()
        assert ((out[b] - want).abs() <= tol)[:, d // 2:].all()


@pytest.mark.parametrize("lens,Hq,Hk,d", SHAPES)
def test_nan_values(lens, Hq, Hk, d):
    out, ref = run(lens, Hq, Hk, d, -1.0, second, math.nan)
    for b in range(len(lens)):
        assert torch.isnan(out[b][:, :d // 2]).all() and torch.isfinite(out[b][:, d // 2:]).all()
