"""Refusals of the decode step's entry points, on the host and before anything is launched: through the C ABI with
pointers that are never followed, and through the binding's own checks of tensors."""
import ctypes as C

import pytest
import torch

from tree_speculative_verification_gb300 import api, build

P = C.c_void_p
OK, BAD = P(0x10000), P(0x10008)      # BAD: 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def pool(**kw):
    f = dict(block_table=0x10000, held=0x10000, ring=0x10000, ring_state=0x10000, B=2, max_pages=4, num_pages=9)
    f.update(kw)
    return C.byref(api.ts_page_pool(*[f[n] for n, _ in api.ts_page_pool._fields_]))


def pages(**kw):
    f = dict(k_pages=0x10000, v_pages=0x10000, block_table=0x10000, num_pages=9, max_pages=4)
    f.update(kw)
    return C.byref(api.ts_paged_kv(*[f[n] for n, _ in api.ts_paged_kv._fields_]))


@pytest.mark.parametrize("kw,word", [
    (dict(pool=None), b"pool"), (dict(pool=pool(held=None)), b"NULL"), (dict(pool=pool(ring=None)), b"NULL"),
    (dict(pool=pool(B=0)), b"B="), (dict(pool=pool(B=65536)), b"B="), (dict(pool=pool(num_pages=0)), b"num_pages"),
    (dict(pool=pool(num_pages=1 << 25)), b"num_pages"), (dict(pool=pool(max_pages=0)), b"max_pages"),
    (dict(end=None), b"NULL"), (dict(new_held=None), b"NULL"), (dict(new_state=None), b"NULL"), (dict(begin=None), b"row_begin"),
    (dict(n=0), b"max_slots"), (dict(slot=None), b"slot_offset"), (dict(slot=P(0x10002)), b"4-byte"),
    (dict(pool=pool(held=0x10001)), b"4-byte"), (dict(end=P(0x10002)), b"4-byte"),
])
def test_pages_refusals(lib, kw, word):
    a = {**dict(pool=pool(), new_held=OK, new_state=OK, slot=OK, n=8, off=OK, begin=OK, end=OK), **kw}
    rc = lib.kv_pages_build(a["pool"], a["new_held"], a["new_state"], a["slot"], a["n"], a["off"], a["begin"], a["end"], None, None)
    assert rc == api.TS_ERR_INVALID_ARG and word in lib.treespec_last_error() and b"kv_pages_build" in lib.treespec_last_error()


BAD_PAGES = [(dict(kv=None), 1, b"NULL"), (dict(kv=pages(k_pages=None)), 1, b"NULL"), (dict(kv=pages(v_pages=0x10008)), 1, b"aligned"),
             (dict(kv=pages(num_pages=0)), 1, b"num_pages"), (dict(d=96), 3, b"head_dim"), (dict(H=0), 1, b"H="), (dict(H=65536), 1, b"H=")]


@pytest.mark.parametrize("kw,rc,word", BAD_PAGES + [
    (dict(kv=pages(num_pages=1 << 25)), 1, b"num_pages"), (dict(T=0), 1, b"T="), (dict(slot=None), 1, b"slot"), (dict(k=None), 1, b"k_new"),
    (dict(v=BAD), 1, b"v_new"), (dict(ks=511), 1, b"stride"), (dict(vs=504), 1, b"stride"), (dict(ks=516), 1, b"stride"),
    (dict(vs=(1 << 31) + 8), 1, b"stride"), (dict(slot=P(0x10002)), 1, b"4-byte")])
def test_append_refusals(lib, kw, rc, word):
    a = {**dict(kv=pages(), k=OK, v=OK, ks=512, vs=512, slot=OK, T=3, H=4, d=128), **kw}
    got = lib.kv_append_slots(a["kv"], a["k"], a["v"], a["ks"], a["vs"], a["slot"], a["T"], a["H"], a["d"], None, None)
    assert got == rc and word in lib.treespec_last_error() and b"kv_append_slots" in lib.treespec_last_error()


@pytest.mark.parametrize("kw,rc,word", BAD_PAGES + [
    (dict(kv=pages(block_table=None)), 1, b"block table"), (dict(kv=pages(max_pages=0)), 1, b"block table"), (dict(out=None), 1, b"NULL"),
    (dict(n=None), 1, b"NULL"), (dict(out=BAD), 1, b"out"), (dict(q=BAD), 1, b"q must"), (dict(q=None), 1, b"q is NULL"),
    (dict(Hq=6), 1, b"multiple"), (dict(Hq=0), 1, b"multiple"), (dict(B=0), 1, b"B="), (dict(B=65536), 1, b"B="), (dict(qs=1000), 1, b"stride"),
    (dict(qs=1028), 1, b"stride"), (dict(scale=float("inf")), 1, b"scale"), (dict(scale=3e38), 1, b"scale"), (dict(ws=None), 1, b"workspace"),
    (dict(wn=16), 1, b"workspace"), (dict(ws=BAD), 1, b"workspace"), (dict(out=OK), 1, b"place of its own"),
    (dict(n=P(0x10001)), 1, b"4-byte")])
def test_attention_refusals(lib, kw, rc, word):
    a = {**dict(out=P(0x20000), q=OK, qs=1024, kv=pages(), n=OK, B=2, Hq=8, H=4, d=128, scale=0.0, ws=OK, wn=1 << 40), **kw}
    got = lib.decode_attention_paged(a["out"], a["q"], a["qs"], a["kv"], a["n"], a["B"], a["Hq"], a["H"], a["d"], a["scale"], a["ws"],
                                     a["wn"], None, None)
    assert got == rc and word in lib.treespec_last_error() and b"decode_attention_paged" in lib.treespec_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(logits=None), b"logits"), (dict(logits=P(0x10002)), b"aligned"), (dict(logits=P(0x10001), dt=1), b"aligned"), (dict(dt=2), b"dtype"),
    (dict(R=0), b"R="), (dict(V=0), b"V="), (dict(V=(1 << 18) + 1, stride=1 << 20), b"V="), (dict(stride=99), b"stride"),
    (dict(stride=(1 << 31) + 1), b"stride"), (dict(token=None), b"no output"), (dict(u=None), b"needs u"),
    (dict(probs=OK), b"place of its own"), (dict(probs=P(0x30000), kept=P(0x30000)), b"place of its own"),
    (dict(kept=OK, dt=1), b"place"), (dict(kept=OK, stride=101), b"place"), (dict(probs=P(0x30002)), b"4-byte"),
    (dict(u=P(0x30001)), b"4-byte"), (dict(token=P(0x30002)), b"4-byte"),
    (dict(token=P(0x30000), u=P(0x30000)), b"place of its own"), (dict(token=OK), b"place of its own")])
def test_sample_refusals(lib, kw, word):
    a = {**dict(token=P(0x20000), probs=None, kept=None, logits=OK, stride=100, dt=0, u=OK, R=2, V=100), **kw}
    rc = lib.sample_tokens(a["token"], a["probs"], a["kept"], a["logits"], a["stride"], a["dt"], a["u"], None, None, None, None, a["R"],
                           a["V"], None, None)
    assert rc == api.TS_ERR_INVALID_ARG and word in lib.treespec_last_error() and b"sample_tokens" in lib.treespec_last_error()


def test_workspace_size(lib):
    f = lib.treespec_decode_workspace_size
    assert f(2, 8, 4, 128) > 0
    for a in ((0, 8, 4, 128), (2, 6, 4, 128), (2, 0, 4, 128), (2, 8, 0, 128), (2, 8, 4, 96), (65536, 8, 4, 128)):
        assert f(*a) == 0, a


def test_binding_refuses_tensors_on_the_host():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    x = torch.zeros(3, 2, 64, 64, dtype=torch.bfloat16)
    kv = api.PagedKV(x, x.clone(), i32(2, 2))
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: api.PagePool(i32(2, 3), i32(2), i32(9), i32(3)), lambda: api.kv_append_slots(kv, q, q, i32(2)),
                 lambda: api.decode_attention_paged(q, q, kv, i32(2), ws=i32(9)),
                 lambda: api.sample_tokens(i32(2), torch.zeros(2, 9), torch.zeros(2))):
        with pytest.raises(api.TreespecError):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers would be followed")
def test_calls_that_pass_without_a_device(lib):
    """An error code comes back, whatever is left out of the call."""
    X = P(0x20000)
    for slot, off in ((OK, OK), (OK, None), (None, None)):
        assert lib.kv_pages_build(pool(), OK, OK, slot, 70000, off, OK, OK, None, None) == api.TS_ERR_CUDA
    for d in (64, 128):
        for T in (1, 2000):
            assert lib.kv_append_slots(pages(), OK, OK, 1024, 1024, OK, T, 4, d, None, None) == api.TS_ERR_CUDA
        for Hq in (4, 32, 64, 128):
            assert lib.decode_attention_paged(X, OK, 128 * Hq, pages(), OK, 2, Hq, 4, d, 0.0, OK, 1 << 40, None, None) == api.TS_ERR_CUDA
    for dt in (0, 1):
        for V in (1, 300, 32001, 50272, 1 << 18):
            for R in (1, 100, 5000):
                for outs in ((X, None, None), (None, X, None), (X, P(0x30000), P(0x40000))):
                    assert lib.sample_tokens(*outs, OK, V, dt, OK, None, OK, OK, None, R, V, None, None) == api.TS_ERR_CUDA
