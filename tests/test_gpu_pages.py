"""kv_pages_build and kv_append_slots against plain definitions: whole numbers and moved values, so everything is equal."""
import numpy as np
import pytest
import torch

from tree_speculative_verification_gb300 import api

from _decode import PK, Pages, cu, device_pool, free_pages

pytestmark = pytest.mark.gpu


def scene(B, seed, P=400, new=70, width=None, short=0):
    """Requests that go on, begin, end, and stay; a pool with `short` pages fewer than they need (or some to spare)."""
    rng = np.random.default_rng(seed)
    rows = rng.integers(0, P, B)
    kind = rng.integers(0, 4, B)
    begin = np.where(kind == 0, rows, np.where(kind == 3, rows, 0))
    end = np.where(kind == 0, rows + rng.integers(1, new + 1, B), np.where(kind == 1, rng.integers(0, P, B), np.where(kind == 3, rows, 0)))
    held = np.where(kind == 1, 0, -(-rows // PK) + (rng.random(B) < 0.3))
    want = -(-end // PK)
    need = int(np.maximum(want - held, 0).sum())
    free = max(0, need - short) if short else need + 3
    num = int(held.sum()) + max(free, 1)
    ids = rng.permutation(num)
    table = rng.integers(-5, num + 5, (B, width or int(max(held.max(), want.max())) + 1))
    at = 0
    for b in range(B):
        table[b, :held[b]], at = ids[at:at + held[b]], at + held[b]
    return Pages(table, held, ids[at:at + free], num), begin, end


def run(ref, begin, end, in_place=True, head=0, extra=5, align=0, max_slots=None, offsets=True):
    pool = device_pool(ref, head)
    n = max(1, int(np.maximum(np.array(end) - begin, 0).sum())) + extra if max_slots is None else max_slots
    room = torch.full((n + align,), -9, dtype=torch.int32, device="cuda")
    slot, off = room[align:], torch.full((pool.B + 1,), -9, dtype=torch.int32, device="cuda")
    held = pool.held if in_place else torch.full_like(pool.held, -9)
    state = pool.state if in_place else torch.zeros_like(pool.state)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = {} if in_place else {"new_held": held, "new_state": state}
    for _ in range(1 if in_place else 3):     # apart from the pool's own: again, with the same outcome
        api.kv_pages_build(pool, cu(end), cu(begin), slot, off if offsets else None, status=status, **args)
    slots, offset, bits = ref.build(begin, end, n)
    assert status.item() == bits
    assert held.tolist() == ref.held
    for b, h in enumerate(ref.held):
        assert pool.block_table[b, :max(h, 0)].tolist() == ref.table[b, :max(h, 0)].tolist(), f"request {b}"
    assert torch.equal(pool.block_table.cpu(), torch.from_numpy(ref.table.astype(np.int32)))     # what is not held: as it was
    assert free_pages(pool, state) == ref.free
    assert slot.tolist() == slots
    assert not offsets or off.tolist() == offset
    return pool


@pytest.mark.parametrize("B", [1, 2, 33, 300, 512, 513, 1300])
@pytest.mark.parametrize("in_place", [True, False])
def test_pages(B, in_place):
    ref, begin, end = scene(B, B)
    run(ref, begin, end, in_place, head=ref.num - 1)


@pytest.mark.parametrize("short", [1, 3, 40])
@pytest.mark.parametrize("B", [7, 600])
def test_pool_runs_out(B, short):
    """Requests are served in order; from the first that is not, none that needs pages is."""
    ref, begin, end = scene(B, 100 + B + short, short=short)
    run(ref, begin, end, head=2)


@pytest.mark.parametrize("B,P,align", [(3, 9000, 0), (40, 3000, 1), (700, 200, 3)])
def test_many_slots(B, P, align):
    """Several CTAs, whose ranges end inside requests and, unaligned, inside 16 bytes."""
    for in_place in (True, False):
        ref, begin, end = scene(B, 7 * B, P=P, new=3000)
        run(ref, begin, end, in_place, head=5, align=align)


def test_slots_past_the_room():
    ref, begin, end = scene(20, 3, P=900)
    total = int(np.maximum(end - begin, 0).sum())
    run(ref, begin, end, max_slots=total - 1)
    ref, begin, end = scene(20, 4, P=9000)
    run(ref, begin, end, max_slots=1)


def test_nothing_to_do():
    run(Pages([[3, 4]], [2], [], 5), [128], [128])
    run(Pages([[3, 4]], [0], [], 5), [0], [0], max_slots=1, offsets=False)


def test_lengths_that_do_not_fit():
    """They keep their pages and get no slots; the others are served."""
    ref, begin, end = scene(12, 9, width=20)
    begin[1], end[4], begin[6], end[8] = -1, -3, end[6] + 1, 20 * PK + 1
    ref.held[10] = 21
    run(ref, begin, end)


def test_ring_that_does_not_fit():
    for head, count in ((-1, 2), (5, 1), (0, 6), (0, -1), (0, 4)):
        pool = api.PagePool(cu([[1, 2], [0, 0]]), cu([2, 0]), cu([3, 4, 0, 0, 0]), cu([head, count, 0]))
        slot, status = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        api.kv_pages_build(pool, cu([0, 2]), cu([0, 0]), slot, status=status)       # one gives two pages back
        assert status.item() == api.STATUS_INDEX and slot.tolist() == [-1, -1, -1]
        assert pool.held.tolist() == [2, 0] and pool.state.tolist() == [head, count, 0] and pool.ring.tolist() == [3, 4, 0, 0, 0]


def test_ids_outside_the_pool():
    pool = api.PagePool(cu([[1, 9]]), cu([2]), cu([-4, 0, 0]), cu([0, 1, 0]))
    slot, status = torch.zeros(200, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(api.TreespecError, match="slots need"):
        api.kv_pages_build(pool, cu([70]), None, slot)
    api.kv_pages_build(pool, cu([70]), cu([0]), slot, status=status)
    assert slot.tolist() == [64 + r for r in range(64)] + [-1] * 136 and status.item() == api.STATUS_INDEX


def test_tables_only():
    ref, begin, end = scene(50, 21)
    pool = device_pool(ref)
    api.kv_pages_build(pool, cu(end))
    begin[end < begin] = 0
    ref.build(np.minimum(begin, end), end)
    assert pool.held.tolist() == ref.held and free_pages(pool) == ref.free


def test_steps_in_a_graph():
    """A captured call brings the pool up to date at every replay: four requests grow by a row a step across pages."""
    rng = np.random.default_rng(2)
    ref = Pages(np.full((4, 6), -1), [0] * 4, rng.permutation(30), 30)
    pool = device_pool(ref, head=28)
    begin, slot = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(600, dtype=torch.int32, device="cuda")
    end = torch.zeros_like(begin)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        api.kv_pages_build(pool, end, begin, slot, status=status)
    rows = np.array([60, 1, 0, 130])
    for step in range(12):
        at = np.zeros(4, int) if step == 0 else rows.copy()
        rows = rows if step == 0 else rows + 1
        if step == 7:
            at[3] = rows[3] = 0                                  # a request ends, and its pages come back
        begin.copy_(cu(at)), end.copy_(cu(rows))
        graph.replay()
        slots, _, bits = ref.build(at, rows, 600)
        assert slot.tolist() == slots and pool.held.tolist() == ref.held and free_pages(pool) == ref.free and bits == 0
    assert status.item() == 0


@pytest.mark.parametrize("T,H,d", [(1, 1, 64), (1, 8, 128), (3, 5, 128), (65, 2, 64), (1025, 3, 128), (1300, 1, 64)])
@pytest.mark.parametrize("strided", [True, False])
def test_rows_into_their_slots(T, H, d, strided):
    rng = np.random.default_rng(T)
    pages = T // PK + 3
    slot = rng.permutation(pages * PK)[:T]
    slot[rng.random(T) < 0.1] = -1
    x = torch.randn(T, 3 * H, d, device="cuda").to(torch.bfloat16)
    k, v = (x[:, H:2 * H], x[:, 2 * H:]) if strided else (x[:, :H].clone(), x[:, H:2 * H].clone())
    kv = api.PagedKV(*(torch.randn(pages, H, PK, d, device="cuda").to(torch.bfloat16) for _ in "kv"), cu([[0]]))
    want = kv.k_pages.clone(), kv.v_pages.clone()
    for t, s in enumerate(slot):
        if s >= 0:
            want[0][s // PK, :, s % PK], want[1][s // PK, :, s % PK] = k[t], v[t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_append_slots(kv, k, v, cu(slot), status)
    assert torch.equal(kv.k_pages, want[0]) and torch.equal(kv.v_pages, want[1]) and status.item() == 0


@pytest.mark.parametrize("bad", [-2, 3 * PK, 2 ** 31 - 1, -2 ** 31])
def test_slots_outside_the_pages(bad):
    kv = api.PagedKV(*(torch.zeros(3, 2, PK, 64, device="cuda", dtype=torch.bfloat16) for _ in "kv"), cu([[0]]))
    x = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_append_slots(kv, x, x, cu([5, bad, 70]), status)
    assert status.item() == api.STATUS_INDEX
    for p in (kv.k_pages, kv.v_pages):
        assert p.sum().item() == 2 * 2 * 64 and p[0, :, 5].all() and p[1, :, 6].all()


def test_rows_past_32_bits():
    """Pages of more than 2^31 values: the last one's rows."""
    pages, H, d = 2 ** 31 // (32 * PK * 128) + 2, 32, 128
    kv = api.PagedKV(*(torch.empty(pages, H, PK, d, device="cuda", dtype=torch.bfloat16) for _ in "kv"), cu([[0]]))
    for p in (kv.k_pages, kv.v_pages):
        p[0] = 0
        p[-1] = 0
    x = torch.randn(2, H, d, device="cuda").to(torch.bfloat16)
    api.kv_append_slots(kv, x, x, cu([(pages - 1) * PK + 63, 1]))
    for p in (kv.k_pages, kv.v_pages):
        assert torch.equal(p[-1, :, 63], x[0]) and torch.equal(p[0, :, 1], x[1])
        assert not p[-1, :, :63].any() and not p[0, :, 2:].any() and not p[0, :, 0].any()


def test_most_slots_there_can_be():
    """A slot array of 2^31 - 1 entries: the last request's rows, and -1 on to the end."""
    n, B = 2 ** 31 - 1, 3
    pool = device_pool(Pages(np.zeros((B, 4), dtype=np.int64), [0] * B, [3, 1, 2, 0], 4))
    slot = torch.full((n,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_pages_build(pool, cu([64, 1, 2]), cu([0, 0, 0]), slot, None, status=status)
    assert status.item() == 0
    assert slot[:64].tolist() == list(range(192, 256)) and slot[64:67].tolist() == [64, 128, 129]
    for at in range(67, n, 1 << 28):
        assert int(slot[at:at + (1 << 28)].max()) == -1 and int(slot[at:at + (1 << 28)].min()) == -1


def test_ring_after_a_request_that_is_not_served():
    """What the pool cannot serve takes nothing from the ring, also where requests that need no pages follow: the start and the
    count are those of the pages that were handed out (none here, one in the second call)."""
    i32 = lambda *a: cu(list(a))
    pool = api.PagePool(cu([[-1, -1, -1], [2, -1, -1], [-1, -1, -1]]), i32(0, 1, 0), i32(0, 1, 3, 0), i32(2, 1, 0))
    slot, status = torch.full((104,), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_pages_build(pool, i32(100, 11, 0), i32(0, 10, 0), slot, None, status=status)
    assert status.item() == api.STATUS_NO_PAGES
    assert pool.state.tolist() == [2, 1, 0] and pool.held.tolist() == [0, 1, 0]
    assert slot.tolist() == [-1] * 100 + [2 * PK + 10] + [-1] * 3
    status.zero_()
    api.kv_pages_build(pool, i32(60, 100, 0), i32(0, 100, 0), slot, None, status=status)   # the first takes it, the second gets none
    assert status.item() == api.STATUS_NO_PAGES
    assert pool.state.tolist() == [3, 0, 0] and pool.held.tolist() == [1, 1, 0] and int(pool.block_table[0, 0]) == 3
    assert slot[:60].tolist() == list(range(3 * PK, 3 * PK + 60)) and slot[60:].max() == -1
