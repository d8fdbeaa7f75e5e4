"""sample_tokens where u falls among tokens of next to no weight: some token of the row all the same, never -1."""
import numpy as np
import pytest
import torch

from test_gpu_sample import BF16, F32, run

pytestmark = pytest.mark.gpu

#: rows and vocabularies of each of the kernel's layouts: a cluster a row, a CTA a row from L2, a small CTA a row
LAYOUTS = [(40, 1000), (7, 50272), (168, 30001), (168, 60002), (680, 900)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V", LAYOUTS)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_token_and_the_others_far_below(R, V, dtype, where):
    """One token holds nearly everything, the others are 25 to 27 nats below it, 1/8 to 1/2 of 2^-36 each: u = 0 and the smallest
    numbers that a generator of 24 bits gives, and those around the large token."""
    g = torch.Generator("cuda").manual_seed(V)
    for low, high in ((25.3, 26.5), (25.0, 25.2), (26.0, 26.0), (27.0, 29.0)):
        x = -(low + (high - low) * torch.rand(R, V, generator=g, device="cuda"))
        big = {"first": 0, "middle": V // 2, "last": V - 1}[where]
        x[:, big] = 0.0
        u = (np.arange(R) % 8).astype(np.float32) * np.float32(2.0 ** -24)
        u[3::5] = 1 - 2.0 ** -24
        for kw in ({}, {"T": [1.0] * R}, {"p": [0.99999] * R}, {"m": [1e-13] * R}):
            got, status = run(x.to(dtype), u, **kw, want="token")
            token = got["token"].cpu().numpy()
            assert status == 0 and (token >= 0).all() and (token < V).all()
            # the others' mass is V 2^-36 at most: u 2^-24 and above is past all of them that stand before the large one
            sure = u > 2 * V * 2.0 ** -36
            assert (token[sure] >= big).all()
