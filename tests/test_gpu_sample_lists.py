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
