"""tree_attention_kv8 against the definition in 64 bits, over head layouts,
lengths from one key on, ragged and rejected requests, pages that end inside a
tile, poisoned rows in masked and in unused places."""
import math

import pytest
import torch

from _kv8 import Setup, check_attention, get
from tree_speculative_verification_gb300 import api

pytestmark = pytest.mark.gpu


def run(s, Hq, Hk, d, paged=False, scale=0.0, q=None, kv=None, q_scale=1.0, ws=None, cache_scale=1.0):
    kv = kv or s.cache(Hk, d, paged, scale=cache_scale)
    q = q if q is not None else s.randn(s.B, s.n_max, Hq, d, scale=q_scale)
    out = torch.full((s.B, s.n_max, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    before = out.clone()
    ws = ws if ws is not None else api.kv8_workspace(s.B, Hq, Hk, s.n_max, d, kv.L_max)
    api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, scale, ws, s.status)
    return q, kv, out, before, ws


CASES = [  # n_nodes, prefix, Hq, Hk
    ([1], [0], 1, 1),                                # a single token over itself
    ([1], [1], 4, 1),
    ([1, 1, 1], [126, 127, 128], 8, 2),              # the key axis ends before, at and after a 128-key tile
    ([3, 5, 2], [0, 61, 64], 3, 3),
    ([16, 17, 15], [112, 111, 300], 2, 2),           # 128 keys in all; row counts around 16
    ([47, 12, 0, 31], [513, 1024, 40, 77], 4, 2),    # a rejected request among others
    ([64, 65], [190, 255], 2, 2),                    # row counts around 64
    ([21] * 9, [5, 1000, 64, 128, 700, 3, 2, 1, 0], 14, 2),   # seven query heads to a key head
    ([128, 100], [257, 1], 2, 2),
    ([129, 256], [640, 30], 1, 1),
    ([33, 8], [2000, 4100], 16, 2),                  # eight query heads to a key head, rows over several blocks
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n,P,Hq,Hk", CASES)
def test_attention(n, P, Hq, Hk, d, paged):
    s = Setup(n, P, seed=len(n) + Hq + d)
    q, kv, out, before, _ = run(s, Hq, Hk, d, paged)
    check_attention(s, q, kv, out, before)
    assert s.status.item() == 0


@pytest.mark.parametrize("n,P,H", [([1], [40000], 1), ([21], [16384], 2), ([5, 1], [9000, 20011], 3)])
def test_long_axis_and_few_rows(n, P, H):
    s = Setup(n, P, seed=5)
    q, kv, out, before, _ = run(s, H, H, 128)
    check_attention(s, q, kv, out, before)


def test_more_items_than_multiprocessors():
    s = Setup([4, 30, 11, 47, 1, 9, 2, 25] * 3, [300, 17, 900, 64, 1500, 31, 128, 2] * 3, seed=8)
    q, kv, out, before, _ = run(s, 24, 12, 128)
    check_attention(s, q, kv, out, before)


@pytest.mark.parametrize("q_scale,cache_scale", [(30.0, 1.0), (1e-3, 1.0), (1.0, 1e-6), (1e4, 1e-4), (1e-20, 1e20), (4.0, 4.0)])
def test_magnitudes(q_scale, cache_scale):
    s = Setup([9, 20], [400, 260], seed=2)
    q, kv, out, before, _ = run(s, 4, 2, 128, q_scale=q_scale, cache_scale=cache_scale)
    check_attention(s, q, kv, out, before)


@pytest.mark.parametrize("scale", [1.0, 0.02])
def test_scale(scale):
    s = Setup([9, 20], [400, 260], seed=2)
    q, kv, out, before, _ = run(s, 2, 2, 64, scale=scale)
    check_attention(s, q, kv, out, before, scale)


@pytest.mark.parametrize("where", ["first", "late", "rising"])
def test_scores_that_grow_along_the_axis(where):
    """One key far above all others (a sink at the front, or found late), and scores that rise from tile to tile: the
    running maximum moves, and the small weights still count. V's scales grow by 2^10 along the axis too."""
    s = Setup([13, 40], [1500, 2100], seed=4)
    kv = s.cache(2, 128)
    q = s.randn(2, 40, 4, 128)
    q[..., 0] = 8.0
    for b in range(2):
        L = s.P[b]
        k = kv.k[b].float()
        if where == "first":
            kv.k_scale[b, :, 0] *= 1.0
            k[:, 0] = 0.0
            k[:, 0, 0] = 16.0
            kv.k_scale[b, :, 0] = 1.0                 # a score of 128 / sqrt(128) = 11.3 above the rest
        elif where == "late":
            k[:, L - 5] = 0.0
            k[:, L - 5, 0] = 60.0
            kv.k_scale[b, :, L - 5] = 1.0
        else:
            k[:, :L, 0] = (torch.arange(L, device="cuda") / L * 400.0)
            kv.k_scale[b, :, :L] = 0.05
        kv.k[b] = k.to(torch.float8_e4m3fn)
        kv.v_scale[b, :, :L] *= 2.0 ** torch.linspace(-5, 5, L, device="cuda")
    q, kv, out, before, _ = run(s, 4, 2, 128, q=q, kv=kv)
    check_attention(s, q, kv, out, before)


def test_many_small_weights_behind_a_sink():
    """A key that takes half the weight against 60000 others of about 2^-17 each."""
    s = Setup([2], [60000], seed=9)
    kv = s.cache(1, 128)
    q = s.randn(1, 2, 1, 128, scale=0.05)
    q[..., 0] = 8.0
    k = kv.k[0].float()
    k[:, 3] = 0.0
    k[:, 3, 0] = 15.5                                 # a score of 11, e^11 = 60000
    kv.k_scale[0, :, 3] = 1.0
    k[:, 4:, 0] = 0.0
    kv.k[0] = k.to(torch.float8_e4m3fn)
    q, kv, out, before, _ = run(s, 1, 1, 128, q=q, kv=kv)
    check_attention(s, q, kv, out, before)


def test_poisoned_rows_reach_only_those_who_see_them():
    """NaN in one node's key and in another's value: only the nodes below them turn NaN; a poisoned query its own row."""
    s = Setup([40, 40], [100, 20], seed=6)
    kv = s.cache(2, 128)
    k, v, q = s.randn(2, 40, 2, 128), s.randn(2, 40, 2, 128), s.randn(2, 40, 2, 128)
    k[0, 5, 0, 3], v[0, 9, 1, 0], v[1, 39, 0, 0] = math.nan, math.inf, math.nan
    api.kv8_append(kv, k, v, s.prefix, s.tree, status=s.status)
    assert s.status.item() == api.STATUS_NONFINITE
    q, kv, out, before, _ = run(s, 2, 2, 128, kv=kv, q=q)
    check_attention(s, q, kv, out, before)
    assert torch.isnan(out[0]).any() and not torch.isnan(out[0, 0]).any()
    q[1, 7, 1, 100] = math.nan
    out2 = torch.zeros_like(out)
    api.tree_attention_kv8(out2, q, kv, s.prefix, s.tree, ws=api.kv8_workspace(2, 2, 2, 40, 128, kv.L_max))
    assert torch.isnan(out2[1, 7, 1]).all()
    out2[1, 7, 1] = out[1, 7, 1]
    assert torch.equal(torch.nan_to_num(out2), torch.nan_to_num(out))


def test_requests_that_do_not_fit_and_bad_pages():
    s = Setup([4, 6, 5], [100, 130, 70], seed=1)
    kv = s.cache(2, 64, paged=True)
    q = s.randn(3, 6, 4, 64)
    good = run(s, 4, 2, 64, q=q, kv=kv)[2]
    old = s.prefix.clone()
    s.prefix[1] = kv.L_max - 5
    s.prefix[2] = -3
    bad = run(s, 4, 2, 64, q=q, kv=kv)[2]
    assert s.status.item() == api.STATUS_INDEX
    assert torch.equal(bad[0], good[0]) and (bad[1:] == 7.0).all()
    s.prefix.copy_(old)
    s.status.zero_()
    table = kv.block_table.clone()
    table[1, 0] = kv.k.shape[0] + 7
    other = run(s, 4, 2, 64, q=q, kv=api.KV8(kv.k, kv.v, kv.k_scale, kv.v_scale, table))[2]
    assert s.status.item() == api.STATUS_INDEX
    assert torch.equal(other[0], good[0]) and torch.equal(other[2], good[2])


def test_same_call_twice_and_captured():
    """Two calls on one workspace, another stream, and a replayed graph give the same bits; new lengths and a new cache
    content are picked up by the replay."""
    s = Setup([21, 13, 40], [3000, 64, 700], seed=11)
    q, kv, out, before, ws = run(s, 8, 2, 128)
    again = run(s, 8, 2, 128, q=q, kv=kv, ws=ws)[2]
    assert torch.equal(out, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = torch.full_like(out, 7.0)
    api.tree_attention_kv8(third, q, kv, s.prefix, s.tree, ws=ws, status=s.status, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, third)
    g, held = torch.cuda.CUDAGraph(), torch.full_like(out, 7.0)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        api.tree_attention_kv8(held, q, kv, s.prefix, s.tree, ws=ws, status=s.status)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, held)
    s.prefix[0] = 1500
    s.P[0] = 1500
    q.copy_(s.randn(*q.shape))
    held.fill_(7.0)
    g.replay()
    check_attention(s, q, kv, held, before)
    assert s.status.item() == 0


def test_dense_and_paged_agree():
    s = Setup([30, 7], [200, 450], seed=12)
    kv = s.cache(2, 128, paged=True)
    dense = api.KV8.dense(2, 2, kv.L_max, 128)
    for b in range(2):
        kc, vc, ks, vs = get(kv, b, s.P[b] + s.n[b])
        m = kc.shape[1]
        dense.k.view(torch.uint8)[b, :, :m], dense.v.view(torch.uint8)[b, :, :m] = kc, vc
        dense.k_scale[b, :, :m], dense.v_scale[b, :, :m] = ks, vs
    q = s.randn(2, 30, 6, 128)
    assert torch.equal(run(s, 6, 2, 128, q=q, kv=kv)[2], run(s, 6, 2, 128, q=q, kv=dense)[2])
