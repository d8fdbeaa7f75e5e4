"""decode_attention_paged against its definition in 64 bits."""
import math

import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import PK, Cache, check_attention, cu

pytestmark = pytest.mark.gpu


def queries(B, Hq, d, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed + 1)
    return (scale * torch.randn(B, Hq, d, generator=g, device="cuda")).to(torch.bfloat16)


def attend(cache, q, lens, scale=0.0, ws=None, status=None, out=None):
    B, Hq, d = q.shape
    out = torch.full((B, Hq, d), math.nan, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = api.decode_workspace(B, Hq, cache.kv.H, d) if ws is None else ws
    api.decode_attention_paged(out, q, cache.kv, cu(lens), scale, ws, status)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (3, 1), (4, 2), (2, 3), (8, 4), (2, 7), (1, 8), (2, 9), (1, 16), (1, 17), (2, 32), (1, 71)])
def test_heads(Hk, G, d):
    """Every grouping of heads, over lengths about the sizes of pages and tiles."""
    lens = [1, 16, 63, 64, 65, 0, 130, 513]
    c = Cache(lens, Hk, d, seed=G)
    q = queries(len(lens), Hk * G, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(c, q, attend(c, q, lens, status=status), lens)
    assert status.item() == 0


@pytest.mark.parametrize("lens", [[0], [1], [2], [15], [17], [0, 0, 0], [4097], [0, 8000, 0], [1000, 1, 300, 2049, 64]])
@pytest.mark.parametrize("d,Hk,G", [(128, 8, 4), (64, 1, 1), (128, 2, 16)])
def test_lengths(lens, d, Hk, G):
    c = Cache(lens, Hk, d, seed=len(lens))
    q = queries(len(lens), Hk * G, d)
    check_attention(c, q, attend(c, q, lens), lens)


@pytest.mark.parametrize("B,n,Hk,G,d", [(1, 16384, 1, 8, 128), (1, 16384, 8, 1, 64), (300, 70, 2, 1, 128), (2, 16001, 4, 20, 128),
                                        (70, 129, 40, 1, 128)])
def test_work_cut_over_the_keys_and_joined(B, n, Hk, G, d):
    lens = [max(0, n - 37 * b) for b in range(B)]
    c = Cache(lens, Hk, d, seed=n)
    q = queries(B, Hk * G, d)
    check_attention(c, q, attend(c, q, lens), lens)


def test_many_requests():
    """More requests than a CTA has threads, most of them empty."""
    lens = [(b * 13) % 90 if b % 7 == 0 else 0 for b in range(2100)]
    c = Cache(lens, 1, 64, seed=3)
    q = queries(len(lens), 2, 64)
    check_attention(c, q, attend(c, q, lens), lens)


@pytest.mark.parametrize("scale", [0.01, 0.5])
def test_scale_and_strided_queries(scale):
    lens = [200, 3]
    c = Cache(lens, 2, 128, seed=1)
    x = torch.cat((queries(2, 8, 128), queries(2, 4, 128, 5)), 1)
    out = attend(c, x[:, :8], lens, scale)
    check_attention(c, x[:, :8], out, lens, scale)
    assert torch.equal(out, attend(c, x[:, :8].clone(), lens, scale))


def test_large_scores():
    """Scores in the thousands: all weight on a few keys."""
    lens = [500, 64, 4000]
    c = Cache(lens, 2, 128, seed=1, scale=20.0)
    q = queries(3, 8, 128, scale=20.0)
    check_attention(c, q, attend(c, q, lens), lens)


def test_equal_and_lowest_keys():
    """All scores equal, and scores of the type's lowest value next to others."""
    lens = [300, 70]
    c = Cache(lens, 1, 64, seed=1)
    lowest = torch.finfo(torch.bfloat16).min
    for b, (k, _) in enumerate(c.rows):
        k.zero_()
        if b == 1:
            k[:, 5:40, 0] = lowest
        for j in range(-(-lens[b] // PK)):
            r = slice(j * PK, min(lens[b], j * PK + PK))
            c.k[int(c.bt[b, j]), :, :r.stop - r.start] = k[:, r]
    q = queries(2, 4, 64)
    q[..., 0] = 1.0 / 16
    check_attention(c, q, attend(c, q, lens), lens)


def test_values_that_are_seen_and_not_finite():
    """NaN and infinities of seen rows reach the outputs of their requests and no others."""
    lens = [100, 100, 100, 100]
    c = Cache(lens, 1, 64, seed=1)
    q = queries(4, 2, 64)
    ref = attend(c, q, lens)
    c.v[int(c.bt[1, 0]), 0, 7, 3] = math.nan
    c.v[int(c.bt[2, 1]), 0, 0, 5] = math.inf
    c.k[int(c.bt[3, 0]), 0, 1, 1] = math.nan
    out = attend(c, q, lens)
    assert torch.equal(out[0], ref[0])
    assert torch.isnan(out[1, :, 3]).all() and torch.equal(out[1, :, :3], ref[1, :, :3]) and torch.equal(out[1, :, 4:], ref[1, :, 4:])
    assert torch.isinf(out[2, :, 5]).all() and torch.isfinite(out[2, :, :5]).all()
    assert torch.isnan(out[3]).all()


@pytest.mark.parametrize("n", [-1, 2 * PK + 1, 2 ** 31 - 1])
def test_lengths_past_the_pages(n):
    """The request's rows stay, the others are computed."""
    lens = [128, 40, 128]
    c = Cache(lens, 2, 128, seed=1, width=2)
    q = queries(3, 4, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((3, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    attend(c, q, [128, n, 128], status=status, out=out)
    assert status.item() == api.STATUS_INDEX and (out[1] == 5.0).all()
    c.rows = [c.rows[0], c.rows[2]]
    check_attention(c, q[[0, 2]], out[[0, 2]], [128, 128])


@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_pages_outside_the_cache_read_as_zeros(bad):
    lens = [200, 150]
    c = Cache(lens, 2, 64, seed=2)
    q = queries(2, 4, 64)
    bt = c.bt.copy()
    bt[0, 1] = bad
    c.kv = api.PagedKV(c.k, c.v, cu(bt))
    for x in c.rows[0]:
        x[:, PK:2 * PK] = 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(c, q, attend(c, q, lens, status=status), lens)
    assert status.item() == api.STATUS_INDEX


def test_same_results_again_and_workspace_shared_by_sizes():
    """Bit-equal outputs call after call, and one workspace for calls of several sizes in turn."""
    cases = []
    for lens, Hk, G, d in (([5000, 100], 2, 4, 128), ([64], 1, 1, 64), ([9000], 1, 16, 128), ([300] * 40, 8, 2, 64)):
        c = Cache(lens, Hk, d, seed=len(lens))
        q = queries(len(lens), Hk * G, d)
        cases.append((c, q, lens, attend(c, q, lens)))
    ws = torch.zeros(max(api.decode_workspace(len(x[2]), x[1].shape[1], x[0].kv.H, x[1].shape[2]).numel() for x in cases),
                     dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for c, q, lens, ref in cases:
            assert torch.equal(attend(c, q, lens, ws=ws), ref)


def test_two_streams_and_a_graph():
    lens = [700, 2000, 1]
    c = Cache(lens, 4, 128, seed=8)
    qs = [queries(3, 8, 128, s) for s in range(2)]
    ref = [attend(c, q, lens) for q in qs]
    outs = [torch.zeros_like(q) for q in qs]
    ws = [api.decode_workspace(3, 8, 4, 128) for _ in qs]
    n = cu(lens)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):                                        # at once, each with a workspace of its own
        for i, s in enumerate(streams):
            api.decode_attention_paged(outs[i], qs[i], c.kv, n, ws=ws[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        for i in range(2):
            api.decode_attention_paged(outs[i], qs[i], c.kv, n, ws=ws[0])
    for _ in range(3):
        for o in outs:
            o.fill_(math.nan)
        graph.replay()
        assert all(torch.equal(o, r) for o, r in zip(outs, ref))
    n.copy_(cu([64, 2000, 0]))                                  # lengths are read on the GPU
    graph.replay()
    c.rows = [[x[:, :m] for x in kv] for kv, m in zip(c.rows, (64, 2000, 0))]
    check_attention(c, qs[0], outs[0], [64, 2000, 0])


def test_pages_past_32_bits():
    """A cache of more than 2^31 values, whose requests hold its last pages."""
    H, d = 32, 128
    pages = 2 ** 31 // (H * PK * d) + 3
    c = Cache([100, 60], H, d, seed=4)
    big = [torch.empty(pages, H, PK, d, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    bt = c.bt.copy()
    for b, m in enumerate((2, 1)):
        for j in range(m):
            page = pages - 1 - 2 * b - j
            for x, y in zip(big, (c.k, c.v)):
                x[page] = y[int(c.bt[b, j])]
            bt[b, j] = page
    c.kv = api.PagedKV(*big, cu(bt))
    q = queries(2, H, d)
    check_attention(c, q, attend(c, q, [100, 60]), [100, 60])


def test_agrees_with_tree_attention_of_one_node():
    """The same step as a tree of one node over the same pages: outputs within the two kernels' roundings."""
    lens = [100, 1, 700]
    c = Cache(lens, 4, 128, seed=6)
    q = queries(3, 4, 128)
    out = attend(c, q, lens)
    t = api.Tree(3, 1)
    api.tree_build(t, cu([[0]] * 3), cu([[-1]] * 3), cu([1] * 3))
    ref = torch.zeros(3, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
    L = c.bt.shape[1] * PK
    for x in (c.k, c.v):
        x.nan_to_num_(0.0)
    api.tree_attention_paged(ref, q[:, None].contiguous(), c.kv, cu([n - 1 for n in lens]), t,
                             ws=api.workspace(api.TS_OP_ATTENTION, 3, 4, 1, 128, L, 1))
    assert (out.float() - ref[:, 0].float()).abs().max() < 2e-2


def test_more_tiles_than_32_bits_count():
    """2^31 tiles in all: told, and only the rows without a key are written (no page is read)."""
    B, H, d, pages = 16385, 256, 64, 512
    kv = api.PagedKV(torch.zeros(1, H, PK, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, H, PK, d, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(B, pages, dtype=torch.int32, device="cuda"))
    lens = torch.full((B,), pages * PK, dtype=torch.int32, device="cuda")
    lens[77] = 0
    q = torch.zeros(B, H, d, dtype=torch.bfloat16, device="cuda")
    out = torch.ones_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.decode_attention_paged(out, q, kv, lens, 0.0, api.decode_workspace(B, H, H, d), status)
    assert status.item() == api.STATUS_INDEX
    assert not out[77].any() and (out[:77] == 1).all() and (out[78:] == 1).all()


@pytest.mark.parametrize("B,Hk,G,d,n", [(3, 8, 4, 128, 600), (7, 4, 1, 64, 900), (11, 8, 2, 128, 3000), (32, 1, 8, 128, 2000), (31, 12, 1, 64, 300),
                                        (33, 8, 1, 128, 700), (2, 2, 9, 128, 8000), (1, 5, 3, 64, 12000)])
def test_unlike_lengths(B, Hk, G, d, n):
    """Batches of all lengths, some empty, cut into parts of their items."""
    g = torch.Generator().manual_seed(B)
    for again in range(3):
        lens = torch.randint(0, n + 1, (B,), generator=g).tolist()
        if again == 1:
            lens[B // 2] = 0
        if again == 2:
            lens = [n - n // 50 * (b % 2) for b in range(B)]
        c = Cache(lens, Hk, d, seed=again)
        q = queries(B, Hk * G, d, again)
        check_attention(c, q, attend(c, q, lens), lens)
