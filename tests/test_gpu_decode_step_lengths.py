"""DecodeStep.begin with lengths that its rows do not bear out: nothing of such a request is taken over."""
import pytest
import torch

from tree_speculative_verification_gb300 import api
from tree_speculative_verification_gb300.step import DecodeStep

from _decode import PK, attention64, cu

pytestmark = pytest.mark.gpu
B, Hq, Hk, d = 4, 4, 2, 64


def fresh(num_pages=12):
    return DecodeStep(B, Hq, Hk, d, num_pages, 4)


def rows(n, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(n, Hk, d, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv"]


def step(s, seed=1):
    """A step of every request that takes part; its q, k and v."""
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v = (torch.randn(B, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
    s.run(q, k, v, torch.randn(B, 100, generator=g, device="cuda"), torch.full((B,), 0.5, device="cuda"))
    return q, k, v


def check(s, held, q, k, v):
    """held[b]: the (k, v) rows [n][Hk][d] that request b had before the step."""
    for b, (K, V) in enumerate(held):
        if K.shape[0] == 0:
            assert not s.out[b].any()
            continue
        K, V = torch.cat((K, k[b:b + 1])), torch.cat((V, v[b:b + 1]))
        ref, tol = attention64(q[b], K.transpose(0, 1), V.transpose(0, 1), d ** -0.5)
        assert ((s.out[b].double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("lengths,fits", [([3, 70, 40, 0], 3), ([3, 200, 1, 1], 1), ([113, 0, 0, 1], 1), ([114, 0, 5, 0], 0)])
def test_more_rows_than_there_are(lengths, fits):
    """113 rows: requests up to those whose rows end past them are taken over, the others stay empty, now and in the next step."""
    s, (k, v) = fresh(), rows(113)
    s.begin(cu(lengths), k, v)
    want = [n if sum(lengths[:b + 1]) <= 113 else 0 for b, n in enumerate(lengths)]
    assert sum(n > 0 for n in want) == fits
    assert s.len.tolist() == want and s.status.item() == (api.STATUS_INDEX if sum(lengths) > 113 else 0)
    at = [sum(lengths[:b]) for b in range(B)]
    held = [(k[a:a + n], v[a:a + n]) for a, n in zip(at, want)]
    check(s, held, *step(s))
    assert s.len.tolist() == [n + (n > 0) for n in want]


def test_negative_lengths():
    """A length below 0 does not take rows away."""
    s, (k, v) = fresh(), rows(100)
    s.begin(cu([60, 40, 0, 0]), k, v)
    assert s.status.item() == 0
    more = rows(5, 3)
    s.begin(cu([-1, 0, 5, -7]), *more)
    assert s.len.tolist() == [60, 40, 5, 0] and s.status.item() == api.STATUS_INDEX
    check(s, [(k[:60], v[:60]), (k[60:], v[60:]), more, (k[:0], v[:0])], *step(s))


def test_pages_of_what_was_not_taken_over_come_back():
    """All pages are free again once every request has ended."""
    s, (k, v) = fresh(8), rows(10)
    s.begin(cu([4, 200, 0, 0]), k, v)
    assert s.len.tolist() == [4, 0, 0, 0]
    s.end(torch.ones(B, dtype=torch.bool, device="cuda"))
    assert s.pool.state.tolist()[1] == 8 and not s.pool.held.any()
    s.begin(cu([0, 2 * PK, 0, 0]), *rows(2 * PK))
    assert s.len.tolist() == [0, 2 * PK, 0, 0]
