"""Heads that are rotated without a norm: the norm's weights, though given, are left out."""
import pytest
import torch

from _kv8 import Setup, get, norm_rope64
from tree_speculative_verification_gb300 import api

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 64, True), (64, 32, False), (64, 0, False)])
def test_weights_without_a_norm(d, rot, inter, dtype):
    s = Setup([13, 5], [100, 3000], seed=d + rot)
    q, k, v = [s.randn(2, 13, H, d, dtype=dtype) for H in (6, 2, 2)]
    inv = api.QKRope.frequencies(rot) if rot else None
    w = [1.0 + 0.3 * s.randn(d, dtype=torch.float32) for _ in "qk"]
    given, bare = (api.QKRope(inv, *x, norm=False, interleaved=inter) for x in (w, (None, None)))
    outs = []
    for r in (given, bare):
        qo, ko, qa = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q)
        api.tree_qk_norm_rope(qo, ko, q, k, r, s.tree, s.status)
        kv = api.KV8.dense(2, 2, 3020, d)
        kv.bt = None
        api.kv8_append(kv, k, v, s.prefix, s.tree, r, q, qa, s.status)
        outs.append([qo, ko, qa] + [x for b in range(2) for x in get(kv, b, s.P[b] + s.n[b])])
    assert all(same(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][0], outs[0][2])
    # rotations off by 8 steps of fp32 of |a| + |b| (angle, sine and cosine, two products and a sum), then rounded
    ref = dict(inv=inv, rot=rot, norm=False, interleaved=inter)
    eps = torch.finfo(dtype).eps / 2
    for x, y in ((q, outs[0][0]), (k, outs[0][1])):
        for b in range(2):
            pos = [s.P[b] + int(s.depth[b, s.dfs[b, u]]) for u in range(s.n[b])]
            z, mag = norm_rope64(x[b, :s.n[b]], None, pos, ref, d)
            assert ((y[b, :s.n[b]].double() - z).abs() <= eps * z.abs() + 8 * 2.0 ** -24 * (1 + eps) * mag).all()
    assert s.status.item() == 0
