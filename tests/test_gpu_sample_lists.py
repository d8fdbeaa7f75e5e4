"""sample_tokens of many long rows whose kept tokens are listed and are more than a CTA's threads."""
import numpy as np
import pytest
import torch

from test_gpu_sample import BF16, F32, logits, uniforms
from test_gpu_sample_rows import LONG, MANY, check_some

pytestmark = pytest.mark.gpu


def above(x, n, T):
    """min_p [R] with which rows x keep the n tokens of the highest values (fp32: between the n-th one's value and the next)."""
    y = x.double().sort(dim=-1, descending=True).values
    return torch.exp((0.5 * (y[:, n - 1] + y[:, n]) - y[:, 0]) / T).float().cpu().numpy()


@pytest.mark.parametrize("dtype,V", LONG)
@pytest.mark.parametrize("n", [513, 700, 999, 1000, 1001, 3000])
def test_min_p_keeps_about_as_many_as_top_k(dtype, V, n):
    """More than 512 kept by min-p, beside a top_k of more, as many and fewer; with top-p and without."""
    R, T = MANY, 1.3
    x = logits(R, V, 21, dtype)
    k = [1000, n, n + 1, n - 1, 0, V] * (R // 6)
    for p in (1.0, 0.97):
        check_some(x, uniforms(R, n), list(range(24)), T=[T] * R, k=k, p=[p] * R, m=above(x, n, T))
    check_some(x, uniforms(R, n + 1), list(range(24)), T=[T] * R, k=k, m=above(x, n, T), want="token")


def test_min_p_and_top_k_of_every_row():
    """One top_k for all, min-p by row: every row's token."""
    R, V, T = MANY, 50272, 1.3
    x = logits(R, V, 22)
    check_some(x, uniforms(R, 5), list(range(R)), T=[T] * R, k=[1000] * R, m=[0.02] * R, want="token")
    check_some(x, np.full(R, 0.5, np.float32), list(range(R)), T=[T] * R, k=[1000] * R, m=[0.02] * R, want="token probs")


def far_rows(R, V, finite, values, dtype, seed=0):
    """Rows of -inf but for `finite` tokens anywhere, which hold values(generator, number) in any order."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.full((R, V), -np.inf, device="cuda")
    for r in range(R):
        ids = torch.randperm(V, generator=g, device="cuda")[:finite]
        x[r, ids] = values(g, finite)
    return x.to(dtype)


@pytest.mark.parametrize("dtype,V", LONG)
@pytest.mark.parametrize("p", [1.0, 0.9])
def test_top_k_ends_far_below_the_top(dtype, V, p):
    """513 to 4096 finite tokens, as a grammar leaves them, and top-k ending among those far below the top, which count in one
    class whatever their distance."""
    R = MANY
    rows = list(range(0, R, 7))
    wide = far_rows(R, V, 3000, lambda g, n: 10.0 * torch.randn(n, generator=g, device="cuda"), dtype, 1)
    check_some(wide, uniforms(R, 1), rows, T=[0.2] * R, k=[1500] * R, p=[p] * R)
    check_some(wide, uniforms(R, 2), rows, T=[0.2] * R, k=[2999] * R, p=[p] * R)

    def steps(g, n):   # 600 near the top, the others from 129 to 2000 below it
        near = 9.0 * torch.rand(600, generator=g, device="cuda") - 9.0
        near[0] = 0.0
        return torch.cat((near, -129.0 - 1871.0 * torch.rand(n - 600, generator=g, device="cuda")))
    x = far_rows(R, V, 3000, steps, dtype, 2)
    for k in (700, 601, 600, 2500, 3000):
        check_some(x, uniforms(R, k), rows, k=[k] * R, p=[p] * R)


@pytest.mark.parametrize("dtype,V", LONG)
def test_top_k_ends_among_masks_of_low_numbers(dtype, V):
    """Masks of finite numbers: -1e30, the lowest of the type, and -1e4, beside 600 ordinary tokens."""
    R = MANY
    low = float(torch.finfo(dtype).min)

    def values(g, n):
        y = 3.0 * torch.randn(n, generator=g, device="cuda")
        y[600:1500], y[1500:2400], y[2400:] = -1e30, low, -1e4
        return y
    x = far_rows(R, V, 3000, values, dtype, 3)
    for k in (700, 1300, 2000, 2999):
        check_some(x, uniforms(R, k), list(range(0, R, 7)), k=[k] * R, want="token kept")
        check_some(x, uniforms(R, k), list(range(0, R, 7)), k=[k] * R, p=[0.95] * R, want="token probs")
