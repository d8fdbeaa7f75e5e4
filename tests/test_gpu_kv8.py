"""tree_qk_norm_rope, and append, read-back and commit of the 8-bit cache,
against their definitions in 64 bits (fp32 where the definition says fp32)."""
import math

import numpy as np
import pytest
import torch

from _kv8 import F8, PK, Setup, get, norm_rope64, quantised, values
from tree_speculative_verification_gb300 import api

pytestmark = pytest.mark.gpu

# fp32 steps between a head's values and its rotated ones, in units of 2^-24 of |a| + |b|: the sum of squares (13
# additions, halved by the root), mean and eps (2), rsqrt (4), two products, the angle's rounding and sincos (8), the
# rotation's products and sum (3): below 32
F32_OFF = 32 * 2.0 ** -24


def step(dtype):
    return torch.finfo(dtype).eps / 2


def rotary(s, d, rot, norm=True, weights=True, interleaved=False, theta=10000.0):
    inv = api.QKRope.frequencies(rot, theta) if rot else None
    w = [1.0 + 0.3 * s.randn(d, dtype=torch.float32) if weights and norm else None for _ in "qk"]
    return (api.QKRope(inv, w[0], w[1], 1e-6, norm, interleaved),
            dict(inv=inv, rot=rot, norm=norm, eps=1e-6, interleaved=interleaved), w)


def projection(s, Hq, Hk, d, dtype, sliced):
    """q, k, v: slices of one projection output, or tensors of their own."""
    if sliced:
        x = s.randn(s.B, s.n_max, Hq + 2 * Hk, d, dtype=dtype)
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    return [s.randn(s.B, s.n_max, H, d, dtype=dtype) for H in (Hq, Hk, Hk)]


ROPE = [  # n_nodes, prefix, Hq, Hk, d, rot, norm, weights, interleaved, sliced
    ([1], [0], 1, 1, 128, 128, True, True, False, False),
    ([1, 1, 1], [131071, 5, 1 << 30], 8, 2, 64, 64, True, False, True, True),
    ([7, 0, 21, 3], [100, 3, 4096, 0], 5, 3, 128, 64, True, True, False, True),
    ([256, 13], [17, 1000], 3, 1, 64, 16, False, False, True, False),
    ([33, 40], [70000, 9], 56, 56, 128, 0, True, True, False, True),
    ([11], [64], 7, 0, 128, 96, True, True, False, False),
    ([11], [64], 0, 4, 64, 32, True, True, False, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,P,Hq,Hk,d,rot,norm,weights,inter,sliced", ROPE)
def test_norm_rope(n, P, Hq, Hk, d, rot, norm, weights, inter, sliced, dtype):
    s = Setup(n, P, seed=len(P) * 7 + d)
    q, k, _ = projection(s, Hq, Hk, d, dtype, sliced)
    r, ref, w = rotary(s, d, rot, norm, weights, inter)
    outs = [torch.full((s.B, s.n_max, H, d), 7.0, dtype=dtype, device="cuda") for H in (Hq, Hk)]
    api.tree_qk_norm_rope(outs[0] if Hq else None, outs[1] if Hk else None, q if Hq else None, k if Hk else None, r, s.tree,
                          s.status)
    for x, wt, out in ((q, w[0], outs[0]), (k, w[1], outs[1])):
        for b in range(s.B):
            m = s.n[b]
            assert (out[b, m:] == 7.0).all()
            if not m or not x.shape[2]:
                continue
            pos = [s.P[b] + int(s.depth[b, s.dfs[b, v]]) for v in range(m)]
            y, mag = norm_rope64(x[b, :m], wt, pos, ref, d)
            err = (out[b, :m].double() - y).abs()
            assert (err <= step(dtype) * y.abs() + F32_OFF * (1 + step(dtype)) * mag + 1e-30).all(), float((err / mag).max())
    assert s.status.item() == 0


def test_norm_rope_in_place():
    s = Setup([9, 5], [50, 60])
    q = s.randn(2, 9, 6, 128)
    r, _, _ = rotary(s, 128, 128)
    out = q.clone()
    api.tree_qk_norm_rope(out, None, out, None, r, s.tree)
    other = q.clone()
    api.tree_qk_norm_rope(other, None, q, None, r, s.tree)
    assert torch.equal(out, other)


APPEND = [  # n_nodes, prefix, Hq, Hk, d, paged, sliced
    ([1], [0], 1, 1, 128, False, False),
    ([5, 0, 64, 3], [63, 10, 100, 0], 6, 3, 64, True, True),
    ([21, 21], [1000, 47], 8, 8, 128, False, True),
    ([256, 130, 1], [1, 62, 640], 2, 1, 128, True, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,P,Hq,Hk,d,paged,sliced", APPEND)
def test_append_is_the_definition_bit_for_bit(n, P, Hq, Hk, d, paged, sliced, dtype):
    s = Setup(n, P, seed=d + len(n))
    _, k, v = projection(s, Hq, Hk, d, dtype, sliced)
    k[0, 0, 0] = 0.0                                 # a row of zeros
    k[0, 0, -1, 1:] = 0.0                            # one value alone
    v[0, 0, 0] = v[0, 0, 0] * 1e-33                  # below the smallest scale
    v[0, 0, -1] = v[0, 0, -1] * 1e30
    kv = s.cache(Hk, d, paged)
    before = [get(kv, b, s.P[b] + s.n[b]) for b in range(s.B)]
    whole = [x.clone() for x in (kv.k.view(torch.uint8), kv.v.view(torch.uint8))]
    api.kv8_append(kv, k, v, s.prefix, s.tree, status=s.status)
    changed = 0
    for b in range(s.B):
        m, p = s.n[b], s.P[b]
        got = get(kv, b, p + m)
        for x, code, scale in ((k, 0, 2), (v, 1, 3)):
            y, z = quantised(x[b, :m].float())       # [m][H][d]
            row = torch.from_numpy(p + s.dfs[b, :m].astype(np.int64)).cuda()
            assert torch.equal(got[code][:, row], y.view(torch.uint8).transpose(0, 1))
            assert torch.equal(got[scale][:, row], z.transpose(0, 1))
            assert torch.equal(got[code][:, :p], before[b][code][:, :p])
            assert torch.equal(got[scale][:, :p], before[b][scale][:, :p])
        changed += m * Hk * d
    for x, y in zip(whole, (kv.k, kv.v)):            # no more bytes than the nodes' rows
        assert int((x != y.view(torch.uint8)).sum()) <= changed
    assert s.status.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,P,Hq,Hk,d,paged,sliced", APPEND)
@pytest.mark.parametrize("inter,rot,with_q", [(False, 1.0, True), (True, 0.5, False)])
def test_append_with_norm_and_rotation(n, P, Hq, Hk, d, paged, sliced, inter, rot, with_q, dtype):
    s = Setup(n, P, seed=d + len(n))
    q, k, v = projection(s, Hq, Hk, d, dtype, sliced)
    r, ref, w = rotary(s, d, int(d * rot), interleaved=inter)
    kv, q_out, q_two = s.cache(Hk, d, paged), *[torch.full((s.B, s.n_max, Hq, d), 7.0, dtype=dtype, device="cuda") for _ in "ab"]
    api.kv8_append(kv, k, v, s.prefix, s.tree, r, q if with_q else None, q_out if with_q else None, s.status)
    if with_q:                                       # the queries are those of the separate call
        api.tree_qk_norm_rope(q_two, None, q, None, r, s.tree)
        assert torch.equal(q_out, q_two)
    for b in range(s.B):
        m = s.n[b]
        if not m:
            continue
        kc, vc, ks, vs = get(kv, b, s.P[b] + m)
        row = torch.from_numpy(s.P[b] + s.dfs[b, :m].astype(np.int64)).cuda()
        pos = [s.P[b] + int(s.depth[b, s.dfs[b, u]]) for u in range(m)]
        y, mag = norm_rope64(k[b, :m], w[1], pos, ref, d)
        z = y.abs().amax(-1) / 448.0
        big = F32_OFF * mag.amax(-1)
        assert ((ks[:, row].T.double() - z).abs() <= big / 448.0 + 2.0 ** -23 * z).all()
        # half a step of e4m3 (2^-4 of a normal value, 2^-10 scales of a smaller one), and the fp32 steps before it
        err = (values(kc[:, row], ks[:, row]).transpose(0, 1) - y).abs()
        tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * z[..., None]) + 2 * big[..., None] + 2.0 ** -20 * y.abs()
        assert (err <= tol).all(), float((err / tol).max())
        vy, vz = quantised(v[b, :m].float())
        assert torch.equal(vc[:, row], vy.view(torch.uint8).transpose(0, 1)) and torch.equal(vs[:, row], vz.T)
    assert s.status.item() == 0


def test_append_of_nonfinite_rows():
    s = Setup([6], [10])
    k, v = s.randn(1, 6, 2, 64), s.randn(1, 6, 2, 64)
    k[0, 2, 1, 5], v[0, 3, 0, 63] = math.nan, -math.inf
    kv = s.cache(2, 64)
    api.kv8_append(kv, k, v, s.prefix, s.tree, status=s.status)
    kc, vc, ks, vs = get(kv, 0, 16)
    r2, r3 = 10 + int(s.dfs[0, 2]), 10 + int(s.dfs[0, 3])
    assert torch.isnan(ks[1, r2]) and (kc[1, r2] == 0).all() and torch.isnan(vs[0, r3]) and (vc[0, r3] == 0).all()
    assert int(torch.isnan(ks).sum()) == 1 and int(torch.isnan(vs).sum()) == 1
    assert s.status.item() == api.STATUS_NONFINITE


def test_append_skips_requests_that_do_not_fit():
    s = Setup([4, 4, 4], [10, 61, 3])
    k, v = s.randn(3, 4, 2, 64), s.randn(3, 4, 2, 64)
    kv = s.cache(2, 64)
    s.prefix[1] = kv.L_max - 3                        # four rows from the third last on
    s.prefix[2] = -1
    whole = kv.k.view(torch.uint8).clone()
    r, _, _ = rotary(s, 64, 64)
    q, q_out = s.randn(3, 4, 2, 64), torch.full((3, 4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    api.kv8_append(kv, k, v, s.prefix, s.tree, r, q, q_out, s.status)
    assert s.status.item() == api.STATUS_INDEX
    assert torch.equal(whole[1:], kv.k.view(torch.uint8)[1:]) and not torch.equal(whole[0], kv.k.view(torch.uint8)[0])
    assert (q_out[1:] == 7.0).all() and not (q_out[0] == 7.0).any()


def test_append_skips_a_request_with_a_bad_page():
    s = Setup([70, 70], [30, 30])
    kv = s.cache(2, 64, paged=True)
    bad = kv.block_table.clone()
    bad[0, 1] = kv.k.shape[0]
    broken = api.KV8(kv.k, kv.v, kv.k_scale, kv.v_scale, bad)
    k, v = s.randn(2, 70, 2, 64), s.randn(2, 70, 2, 64)
    old = get(kv, 0, 100)
    api.kv8_append(broken, k, v, s.prefix, s.tree, status=s.status)
    assert s.status.item() == api.STATUS_INDEX
    assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(old, get(kv, 0, 100)))
    y, _ = quantised(k[1].float())
    assert torch.equal(get(kv, 1, 100)[0][:, torch.from_numpy(30 + s.dfs[1].astype(np.int64)).cuda()],
                       y.view(torch.uint8).transpose(0, 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,H,d,paged", [([1], 1, 128, False), ([64, 0, 65, 130], 3, 64, True), ([500, 1, 333], 2, 128, True),
                                            ([200, 63, 7], 5, 64, False)])
@pytest.mark.parametrize("begin", [False, True])
def test_read_is_the_product(rows, H, d, paged, begin, dtype):
    s = Setup([1] * len(rows), [max(0, r - 1) for r in rows])
    kv = s.cache(H, d, paged)
    first = [min(r, 3 * i) for i, r in enumerate(rows)] if begin else [0] * len(rows)
    L_out = max(rows) + 2
    k, v = [torch.full((s.B, H, L_out, d), 7.0, dtype=dtype, device="cuda") for _ in "kv"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    api.kv8_read(k, v, kv, i32(rows), i32(first) if begin else None, s.status)
    for b, (lo, hi) in enumerate(zip(first, rows)):
        kc, vc, ks, vs = get(kv, b, max(1, hi))
        for out, c, z in ((k, kc, ks), (v, vc, vs)):
            ref = (c.view(F8).float() * z[..., None])[:, lo:hi].to(dtype)
            assert torch.equal(out[b, :, :hi - lo], ref)
            assert (out[b, :, hi - lo:] == 7.0).all()
    assert s.status.item() == 0


def test_read_refuses_ranges_and_pages():
    s = Setup([1] * 5, [99] * 5)
    kv = s.cache(2, 64, paged=True)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    new = lambda: [torch.full((5, 2, 100, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = new()
    api.kv8_read(k, v, kv, i32([100, 129, 50, 128, 40]), i32([0, 60, 60, 0, -1]), s.status)
    assert s.status.item() == api.STATUS_INDEX
    assert (k[1:] == 7.0).all() and (v[1:] == 7.0).all() and not (k[0] == 7.0).all()
    s.status.zero_()
    bad = kv.block_table.clone()
    bad[0, 0] = -1
    k2, v2 = new()
    api.kv8_read(k2, v2, api.KV8(kv.k, kv.v, kv.k_scale, kv.v_scale, bad), i32([100, 0, 0, 0, 0]), None, s.status)
    assert s.status.item() == api.STATUS_INDEX
    assert (k2[0, :, :64] == 7.0).all() and torch.equal(k2[0, :, 64:], k[0, :, 64:])


@pytest.mark.parametrize("n,P,H,d,paged", [([1], [0], 1, 128, False), ([21, 0, 40, 9], [60, 5, 127, 0], 9, 64, True),
                                           ([256, 128], [33, 700], 3, 128, True), ([47] * 3, [64, 100, 3], 56, 128, False)])
def test_commit_moves_the_path(n, P, H, d, paged):
    s = Setup(n, P, seed=3)
    kv = s.cache(H, d, paged)
    path, count = np.full((s.B, s.n_max + 1), -1, np.int32), np.zeros(s.B, np.int32)
    for b in range(s.B):
        u, up = s.n[b] - 1, []
        while u >= 0:
            up.append(u)
            u = int(s.par[b, u])
        path[b, :len(up)], count[b] = up[::-1], len(up)
    before = [get(kv, b, s.P[b] + s.n[b]) for b in range(s.B)]
    new = torch.full((s.B,), -5, dtype=torch.int32, device="cuda")
    api.kv8_commit(kv, s.prefix, new, torch.from_numpy(path).cuda(), torch.from_numpy(count).cuda(), s.tree, s.status)
    assert new.tolist() == [p + int(c) for p, c in zip(s.P, count)] and s.status.item() == 0
    for b in range(s.B):
        c = int(count[b])
        src = torch.tensor([s.P[b] + int(s.dfs[b, u]) for u in path[b, :c]], dtype=torch.long, device="cuda")
        for x, y in zip(before[b], get(kv, b, s.P[b] + s.n[b])):
            assert torch.equal(y[:, s.P[b]:s.P[b] + c], x[:, src])
            assert torch.equal(y[:, :s.P[b]], x[:, :s.P[b]])
            assert torch.equal(torch.nan_to_num(y[:, s.P[b] + c:].float()), torch.nan_to_num(x[:, s.P[b] + c:].float()))


def test_commit_refuses_paths_that_are_none():
    s = Setup([5, 5, 5], [10, 10, 10])
    kv = s.cache(2, 64)
    path = torch.full((3, 6), -1, dtype=torch.int32, device="cuda")
    path[0, :2] = torch.tensor([0, 7])               # no such node
    path[1, :1] = 0
    path[2, :1] = 0
    count = torch.tensor([2, 6, 1], dtype=torch.int32, device="cuda")     # more tokens than nodes in request 1
    old = kv.k.view(torch.uint8).clone()
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    api.kv8_commit(kv, s.prefix, new, path, count, s.tree, s.status)
    assert new.tolist() == [10, 10, 11] and s.status.item() == api.STATUS_INDEX
    assert torch.equal(old, kv.k.view(torch.uint8))


def test_binding_checks_tensors():
    s = Setup([4, 4], [10, 10])
    kv, q = s.cache(2, 64), s.randn(2, 4, 4, 64)
    k = s.randn(2, 4, 2, 64)
    r, _, _ = rotary(s, 64, 64)
    r128, _, _ = rotary(s, 128, 64)
    ws = api.kv8_workspace(2, 4, 2, 4, 64, kv.L_max)
    out = torch.zeros_like(q)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = [
        lambda: api.kv8_append(kv, k.float(), k, s.prefix, s.tree),                     # two types
        lambda: api.kv8_append(kv, k[:, :3], k, s.prefix, s.tree),                      # too few nodes
        lambda: api.kv8_append(kv, k.transpose(1, 2), k, s.prefix, s.tree),
        lambda: api.kv8_append(kv, k.repeat(1, 1, 1, 2)[..., ::2], k, s.prefix, s.tree),
        lambda: api.kv8_append(kv, k, k, one, s.tree),                                  # too few prefix lengths
        lambda: api.kv8_append(kv, k, k, s.prefix.long(), s.tree),
        lambda: api.kv8_append(kv, k, k, s.prefix.cpu(), s.tree),
        lambda: api.kv8_append(kv, k, k, s.prefix, s.tree, r128),                       # weights of another head size
        lambda: api.kv8_append(kv, k, k, s.prefix, s.tree, None, q, out),
        lambda: api.kv8_append(kv, k, k, s.prefix, s.tree, r, q),
        lambda: api.kv8_append(kv, k.half(), k.half(), s.prefix, s.tree),
        lambda: api.kv8_append(kv, k, k, s.prefix, api.Tree(3, 4)),
        lambda: api.kv8_append(kv, k, k, s.prefix, s.tree, status=one.float()),
        lambda: api.tree_qk_norm_rope(out[:, :, :2], None, q, None, r, s.tree),
        lambda: api.tree_qk_norm_rope(out, None, q.cpu(), None, r, s.tree),
        lambda: api.kv8_read(k, k, kv, s.prefix),
        lambda: api.kv8_read(torch.zeros(2, 2, 8, 64, device="cuda"), torch.zeros(2, 2, 9, 64, device="cuda"), kv, s.prefix),
        lambda: api.kv8_read(*[torch.zeros(2, 2, 8, 64, device="cuda", dtype=torch.half)] * 2, kv, s.prefix),
        lambda: api.tree_attention_kv8(out, q, kv, s.prefix, s.tree),                   # no workspace
        lambda: api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, ws=ws[:16]),
        lambda: api.tree_attention_kv8(out, q.float(), kv, s.prefix, s.tree, ws=ws),
        lambda: api.tree_attention_kv8(out[:, :, :3], q[:, :, :3], kv, s.prefix, s.tree, ws=ws),
        lambda: api.tree_attention_kv8(out.view(2, 4, 2, 128), q.view(2, 4, 2, 128), kv, s.prefix, s.tree, ws=ws),
        lambda: api.kv8_commit(kv, s.prefix, s.prefix, one, one, s.tree),
        lambda: api.KV8(kv.k, kv.v, kv.k_scale, kv.v_scale, torch.zeros(2, 1, dtype=torch.int32, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(api.TreespecError):
            f()
            raise AssertionError(f"call {i} was taken")
