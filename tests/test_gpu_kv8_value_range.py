"""tree_attention_kv8 where value rows differ in size by far more than their weights do: rows of a branch a query does
not see, rows of no weight, rows of zeros, whole and in parts that are joined."""
import math

import pytest
import torch

from _kv8 import PK, Setup, attention64, get
from tree_speculative_verification_gb300 import api

pytestmark = pytest.mark.gpu

FAR = -60.0                                           # a key's only value, against a query's 8: 42 nats below the rest
TINY = 2.0 ** -100                                    # the scale of a row of zeros


def at(kv, b, row):
    """Where cache row `row` of request b is: (strip or page, row in it)."""
    return (b, row) if kv.block_table is None else (int(kv.bt[b, row // PK]), row % PK)


def scale_value(kv, b, row, factor, h=slice(None)):
    i, r = at(kv, b, row)
    kv.v_scale[i, h, r] *= factor


def set_key(kv, b, row, first, h=slice(None)):
    """A key of zeros but for its first value."""
    i, r = at(kv, b, row)
    code = torch.zeros(kv.d, device="cuda")
    code[0] = first
    kv.k.view(torch.uint8)[i, h, r] = code.to(torch.float8_e4m3fn).view(torch.uint8)
    kv.k_scale[i, h, r] = 1.0


def zero_value(kv, b, row):
    i, r = at(kv, b, row)
    kv.v.view(torch.uint8)[i, :, r] = 0
    kv.v_scale[i, :, r] = TINY


def floor64(s, b, q, kv, G, scale):
    """What the smallest step of a weight may move each output: a weight times its row's value scale is off by at most
    2^-24 of the largest such product of its query row, however small it is; that times the codes it meets."""
    n, P = s.n[b], s.P[b]
    kc, vc, ks, vs = get(kv, b, P + n)
    see = torch.zeros(n, P + n, dtype=torch.bool)
    see[:, :P] = True
    for v in range(n):
        u = v
        while u >= 0:
            see[v, P + int(s.dfs[b, u])] = True
            u = int(s.par[b, u])
    see = see.to(q.device)
    out = torch.zeros(n, q.shape[2], kv.d, dtype=torch.float64, device=q.device)
    for h in range(q.shape[2]):
        K = kc[h // G].view(torch.float8_e4m3fn).double() * ks[h // G].double()[:, None]
        p = torch.softmax((q[b, :n, h].double() @ K.T * scale).masked_fill(~see, -math.inf), -1)
        top = (p * vs[h // G].double()).amax(-1, keepdim=True)
        out[:, h] = 2.0 ** -24 * top * (see.double() @ vc[h // G].view(torch.float8_e4m3fn).double().abs())
    return out


def check(s, q, kv):
    """The call's outputs against the definition, every node of every request."""
    Hq, d = q.shape[2], q.shape[3]
    out = torch.full_like(q, 7.0)
    api.tree_attention_kv8(out, q, kv, s.prefix, s.tree, ws=api.kv8_workspace(s.B, Hq, kv.H, s.n_max, d, kv.L_max),
                           status=s.status)
    assert s.status.item() == 0
    for b in range(s.B):
        ref, tol = attention64(s, b, q, kv, Hq // kv.H, 1.0 / math.sqrt(d))
        tol = tol + floor64(s, b, q, kv, Hq // kv.H, 1.0 / math.sqrt(d))
        worst = ((out[b, :s.n[b]].double() - ref).abs() / tol).amax()
        assert worst <= 1.0, f"request {b}: error {float(worst):.2f} of its tolerance"   # NaN fails too
    return out


def setup(n, P, Hq, Hk, d, paged=False, seed=3):
    s = Setup(n, P, seed=seed)
    q = s.randn(s.B, s.n_max, Hq, d)
    q[..., 0] = 8.0
    kv = s.cache(Hk, d, paged)
    for b in range(s.B):                              # first values of zero: set_key's rows alone use that channel
        for row in range(s.P[b] + s.n[b]):
            i, r = at(kv, b, row)
            kv.k.view(torch.uint8)[i, :, r, 0] = 0
    return s, q, kv


# rows a unit: 16 to 64 query rows; one item, or parts that are joined
SHAPES = [([40], [300], 4, 2, 128), ([9, 31], [100, 5], 3, 3, 64), ([5], [9000], 2, 2, 128), ([47], [4000], 1, 1, 64),
          ([3] * 130, [150] * 130, 2, 1, 128)]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("factor", [2.0 ** 10, 1e6, 1e20])
@pytest.mark.parametrize("n,P,Hq,Hk,d", SHAPES[:4])
def test_a_large_value_in_another_branch(n, P, Hq, Hk, d, factor, paged):
    s, q, kv = setup(n, P, Hq, Hk, d, paged)
    for b in range(s.B):
        scale_value(kv, b, s.P[b] + int(s.dfs[b, s.n[b] - 1]), factor)
    check(s, q, kv)


@pytest.mark.parametrize("factor", [1e6, 1e20])
@pytest.mark.parametrize("n,P,Hq,Hk,d", SHAPES)
def test_a_large_value_of_no_weight(n, P, Hq, Hk, d, factor):
    s, q, kv = setup(n, P, Hq, Hk, d)
    for b in range(s.B):
        row = s.P[b] * 3 // 4
        set_key(kv, b, row, FAR)
        scale_value(kv, b, row, factor if factor < 1e9 else 1e15)   # e^-42 is 2^-61: the product stays far below the rest
    check(s, q, kv)


@pytest.mark.parametrize("n,P,Hq,Hk,d", SHAPES)
def test_zero_rows_of_most_weight(n, P, Hq, Hk, d):
    """A sink whose value is zero, among ordinary rows, and the same beside a value that is far larger than theirs."""
    s, q, kv = setup(n, P, Hq, Hk, d)
    for b in range(s.B):
        zero_value(kv, b, 3)
        set_key(kv, b, 3, 12.0)
    check(s, q, kv)
    for b in range(s.B):
        scale_value(kv, b, s.P[b] - 1, 1e20)
    check(s, q, kv)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n,P,Hq,Hk,d", SHAPES)
def test_half_the_weight_on_zeros_beside_large_values(n, P, Hq, Hk, d, first):
    """One half of the prefix rows zeros, the other 1e30 times its size: the zeros count in the sums all the same."""
    s, q, kv = setup(n, P, Hq, Hk, d)
    for b in range(s.B):
        half = s.P[b] // 2
        zero, large = (slice(0, half), slice(half, s.P[b])) if first else (slice(half, s.P[b]), slice(0, half))
        kv.v.view(torch.uint8)[b, :, zero] = 0
        kv.v_scale[b, :, zero] = TINY
        kv.v_scale[b, :, large] *= 1e30
    check(s, q, kv)


@pytest.mark.parametrize("n,P,Hq,Hk,d", SHAPES)
def test_values_that_grow_and_shrink_along_the_axis(n, P, Hq, Hk, d):
    s, q, kv = setup(n, P, Hq, Hk, d)
    for b in range(s.B):
        L, sign = s.P[b] + s.n[b], 1 if b % 2 == 0 else -1
        kv.v_scale[b, :, :L] *= 2.0 ** (sign * torch.linspace(-50, 50, L, device="cuda"))
    check(s, q, kv)


def test_a_cache_of_zeros():
    s, q, kv = setup([9, 31], [100, 700], 4, 2, 128)
    for scale in (TINY, 0.0):
        kv.v.view(torch.uint8).zero_()
        kv.v_scale.fill_(scale)
        assert (check(s, q, kv)[0, :9] == 0).all()


@pytest.mark.parametrize("up", [2.0 ** 5, 2.0 ** 7, 2.0 ** 10])
def test_small_weights_beside_a_larger_value(up):
    """A sink of half the weight, 60000 keys of 2^-17 each behind it, and one value row of no weight 2^5 to 2^10 times
    the others': the small weights keep their bits (values of one sign, so that what they lose does not cancel)."""
    # more requests than are planned: the long one is one item, whose tail meets the large value's tile
    s, q, kv = setup([2] + [1] * 129, [60000] + [1] * 129, 1, 1, 128, paged=True, seed=9)
    q *= 0.05
    q[..., 0] = 8.0
    kv.v.view(torch.uint8).bitwise_and_(0x7f)
    set_key(kv, 0, 3, 15.5)
    set_key(kv, 0, 700, FAR)
    scale_value(kv, 0, 700, up)
    check(s, q, kv)
