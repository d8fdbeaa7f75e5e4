"""sample_tokens: which status bit says what, where a setting is out of range in a row whose logits are finite, and the other way."""
import math

import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api

from test_gpu_sample import BF16, F32, logits, run, uniforms

pytestmark = pytest.mark.gpu
SHAPES = [(4, 300, F32), (3, 50272, F32), (168, 30001, F32), (168, 60002, BF16), (680, 900, BF16)]


@pytest.mark.parametrize("R,V,dtype", SHAPES)
@pytest.mark.parametrize("bad", [{"T": math.nan}, {"T": -1.0}, {"T": math.inf}, {"T": -math.inf}, {"k": -1}, {"m": math.nan}, {"u": math.nan}])
def test_settings_beside_top_p(R, V, dtype, bad):
    """Rows under top-p alone, and a setting out of range in one of them: its logits are as good as the others'."""
    kw = {"T": [1.0] * R, "k": [0] * R, "m": [0.0] * R, "p": [0.9] * R, "u": list(uniforms(R))}
    for name, value in bad.items():
        kw[name][1] = value
    u = kw.pop("u")
    got, status = run(logits(R, V, 3, dtype), u, **kw)
    assert status == api.STATUS_INDEX
    assert got["token"][1] == -1 and torch.isnan(got["probs"][1]).all() and torch.isnan(got["kept"][1]).all()
    assert (got["token"][[0, 2]] >= 0).all() and torch.isfinite(got["probs"][[0, 2]]).all()


@pytest.mark.parametrize("R,V,dtype", SHAPES)
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_logits_beside_top_p(R, V, dtype, value):
    """A bad logit is that alone; with a bad setting in the same row it is both."""
    x = logits(R, V, 4, dtype)
    x[1, V // 3] = value
    p, T = [0.9] * R, [1.0] * R
    assert run(x, uniforms(R), T=T, p=p)[1] == api.STATUS_NONFINITE
    T[1] = math.nan
    assert run(x, uniforms(R), T=T, p=p)[1] == api.STATUS_NONFINITE | api.STATUS_INDEX
