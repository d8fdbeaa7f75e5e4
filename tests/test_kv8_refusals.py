"""Refusals of the 8-bit cache's entry points and of tree_qk_norm_rope, on the
host and before anything is launched: through the C ABI with pointers that are
never followed, and through the binding's own checks of tensors."""
import ctypes as C

import pytest
import torch

from tree_speculative_verification_gb300 import api, build

P = C.c_void_p
OK = P(0x10000)
BAD = P(0x10008)      # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def tree(B=2, n_max=8, **null):
    t = api.ts_tree(B, n_max, *([0x10000] * 9))
    for name in null:
        setattr(t, name, None)
    return t


def cache(**kw):
    f = dict(k=0x10000, v=0x10000, k_scale=0x10000, v_scale=0x10000, block_table=None, B=2, H=4, d=128, L_max=64,
             num_pages=0, max_pages=0)
    f.update(kw)
    return api.ts_kv8(*[f[n] for n, _ in api.ts_kv8._fields_])


def rope(**kw):
    f = dict(inv_freq=0x10000, q_weight=0x10000, k_weight=0x10000, eps=1e-6, norm=1, rot_dim=64, interleaved=0)
    f.update(kw)
    return api.ts_qk_rope(*[f[n] for n, _ in api.ts_qk_rope._fields_])


def call_rope(lib, t=None, r=None, Hq=8, Hk=4, d=128, qs=None, ks=None, q=OK, k=OK, qo=P(0x20000), ko=P(0x20000), dt=1):
    t, r = t or tree(), r or rope()
    return lib.tree_qk_norm_rope(qo, ko, q, k, Hq, Hk, d, Hq * d if qs is None else qs, Hk * d if ks is None else ks,
                                 C.byref(r), C.byref(t), dt, None, None)


@pytest.mark.parametrize("kw,rc,word", [
    (dict(t=tree(n_max=257)), 1, b"n_max"), (dict(t=tree(B=0)), 1, b"B="), (dict(t=tree(dfs_of=1)), 1, b"NULL"),
    (dict(d=96), 3, b"head_dim"), (dict(dt=5), 1, b"dtype"), (dict(r=rope(rot_dim=8)), 3, b"rot_dim"),
    (dict(r=rope(rot_dim=144)), 3, b"rot_dim"), (dict(r=rope(rot_dim=-16)), 3, b"rot_dim"),
    (dict(r=rope(inv_freq=None)), 1, b"inv_freq"), (dict(t=tree(pos=1)), 1, b"positions"),
    (dict(r=rope(eps=-1.0)), 1, b"eps"), (dict(r=rope(eps=float("nan"))), 1, b"eps"),
    (dict(Hq=0, Hk=0), 1, b"Hq"), (dict(Hq=-1), 1, b"Hq"), (dict(q=BAD), 1, b"aligned"), (dict(qo=None), 1, b"NULL"),
    (dict(k=None), 1, b"NULL"), (dict(qs=8 * 128 - 8), 1, b"stride"), (dict(ks=4 * 128 + 4), 1, b"stride"),
    (dict(qs=2048, qo=OK), 1, b"in place"), (dict(ks=2048, ko=OK), 1, b"in place"),
])
def test_rope_refusals(lib, kw, rc, word):
    assert call_rope(lib, **kw) == rc
    assert word in lib.treespec_last_error() and b"tree_qk_norm_rope" in lib.treespec_last_error()


BAD_CACHES = [
    (dict(k=None), 1, b"NULL"), (dict(v_scale=None), 1, b"NULL"), (dict(d=80), 3, b"head_dim"),
    (dict(H=0), 1, b"H="), (dict(v=0x10008), 1, b"aligned"), (dict(k_scale=0x10002), 1, b"aligned"),
    (dict(L_max=0), 1, b"L_max"), (dict(L_max=1 << 30), 1, b"rows"),
    (dict(block_table=0x10000, num_pages=0, max_pages=4), 1, b"num_pages"),
    (dict(block_table=0x10000, num_pages=4, max_pages=0), 1, b"num_pages"),
    (dict(block_table=0x10000, num_pages=1 << 24, max_pages=4), 1, b"rows"),
]
TREE_CACHES = BAD_CACHES + [(dict(B=3), 1, b"B="), (dict(L_max=7), 1, b"n_max")]


def calls(lib, kv, t):
    """Every call that takes a cache and a tree, with otherwise good arguments."""
    r = C.byref(kv)
    return {
        "kv8_append": lambda: lib.kv8_append(r, OK, OK, 512, 512, None, None, None, 0, 0, OK, C.byref(t), 1, None, None),
        "tree_attention_kv8": lambda: lib.tree_attention_kv8(OK, OK, r, 8, OK, C.byref(t), 0.0, OK, 1 << 40, None, None),
        "kv8_commit": lambda: lib.kv8_commit(r, OK, P(0x20000), OK, OK, C.byref(t), None, None),
    }


@pytest.mark.parametrize("kw,rc,word", TREE_CACHES)
@pytest.mark.parametrize("name", ["kv8_append", "tree_attention_kv8", "kv8_commit"])
def test_cache_refusals(lib, name, kw, rc, word):
    assert calls(lib, cache(**kw), tree())[name]() == rc
    assert word in lib.treespec_last_error() and name.encode() in lib.treespec_last_error()


@pytest.mark.parametrize("name", ["kv8_append", "tree_attention_kv8", "kv8_commit"])
def test_tree_refusals(lib, name):
    for t, word in ((tree(n_max=0), b"n_max"), (tree(perm=1), b"NULL"), (tree(sub_end=1), b"NULL")):
        assert calls(lib, cache(), t)[name]() == 1 and word in lib.treespec_last_error()


@pytest.mark.parametrize("kw,rc,word", BAD_CACHES)
def test_read_cache_refusals(lib, kw, rc, word):
    kv = cache(**kw)
    assert lib.kv8_read(OK, OK, C.byref(kv), None, OK, 16, 1, None, None) == rc
    assert word in lib.treespec_last_error() and b"kv8_read" in lib.treespec_last_error()


def test_read_refusals(lib):
    kv = C.byref(cache())
    for a, word in (((None, OK, kv, None, OK, 16, 1), b"NULL"), ((OK, OK, kv, None, None, 16, 1), b"NULL"),
                    ((BAD, OK, kv, None, OK, 16, 1), b"aligned"), ((OK, OK, kv, None, OK, 0, 1), b"L_out"),
                    ((OK, OK, kv, None, OK, 16, 2), b"dtype"), ((OK, OK, None, None, OK, 16, 1), b"NULL")):
        assert lib.kv8_read(*a, None, None) == 1 and word in lib.treespec_last_error()


def test_append_refusals(lib):
    kv, t, r = cache(), tree(), rope()
    good = dict(k=OK, v=OK, ks=512, vs=512, r=None, qo=None, q=None, Hq=0, qs=0, p=OK, dt=1)
    for kw, word in ((dict(k=None), b"k_new"), (dict(v=BAD), b"v_new"), (dict(ks=511), b"stride"), (dict(vs=500), b"stride"),
                     (dict(p=None), b"prefix_len"), (dict(dt=7), b"dtype"), (dict(Hq=4), b"without rope"),
                     (dict(r=rope(rot_dim=24)), b"rot_dim"), (dict(r=r, Hq=8, qs=1024, q=OK), b"q_out"),
                     (dict(r=r, Hq=8, qs=1024, qo=OK), b"q is NULL"), (dict(r=r, Hq=8, q=OK, qo=OK, qs=2048), b"in place"),
                     (dict(r=r, Hq=-2), b"Hq")):
        a = {**good, **kw}
        rc = lib.kv8_append(C.byref(kv), a["k"], a["v"], a["ks"], a["vs"], None if a["r"] is None else C.byref(a["r"]),
                            a["qo"], a["q"], a["Hq"], a["qs"], a["p"], C.byref(t), a["dt"], None, None)
        assert rc in (1, 3) and word in lib.treespec_last_error(), (kw, lib.treespec_last_error())


def test_attention_refusals(lib):
    kv, t = cache(), tree()
    good = dict(out=OK, q=OK, Hq=8, p=OK, scale=0.0, ws=OK, n=1 << 40)
    for kw, word in ((dict(out=None), b"NULL"), (dict(q=BAD), b"aligned"), (dict(Hq=6), b"multiple"), (dict(Hq=0), b"multiple"),
                     (dict(p=None), b"NULL"), (dict(ws=None), b"workspace"), (dict(n=16), b"workspace"),
                     (dict(ws=BAD), b"workspace"), (dict(scale=float("inf")), b"scale")):
        a = {**good, **kw}
        rc = lib.tree_attention_kv8(a["out"], a["q"], C.byref(kv), a["Hq"], a["p"], C.byref(t), a["scale"], a["ws"], a["n"],
                                    None, None)
        assert rc == 1 and word in lib.treespec_last_error(), (kw, lib.treespec_last_error())


def test_commit_refusals(lib):
    kv, t = C.byref(cache()), C.byref(tree())
    assert lib.kv8_commit(kv, OK, OK, OK, OK, t, None, None) == 1 and b"aliases" in lib.treespec_last_error()
    assert lib.kv8_commit(kv, OK, None, OK, OK, t, None, None) == 1 and b"NULL" in lib.treespec_last_error()


def test_workspace_size(lib):
    f = lib.treespec_kv8_workspace_size
    assert f(2, 8, 4, 8, 128, 64) > 0
    for a in ((0, 8, 4, 8, 128, 64), (2, 6, 4, 8, 128, 64), (2, 8, 0, 8, 128, 64), (2, 8, 4, 0, 128, 64),
              (2, 8, 4, 257, 128, 512), (2, 8, 4, 8, 96, 64), (2, 8, 4, 8, 128, 7)):
        assert f(*a) == 0, a


def test_binding_refuses_tensors_that_are_not_a_cache():
    f8, f32 = torch.float8_e4m3fn, torch.float32
    k, s = torch.zeros(2, 4, 64, 128, dtype=f8), torch.zeros(2, 4, 64, dtype=f32)
    for a in ((k.view(torch.uint8), k, s, s), (k, k[:1], s, s), (k, k, s[..., :63], s), (k, k, s, s.double()), (k, k, s, s)):
        with pytest.raises(api.TreespecError):      # the last one: not on a CUDA device
            api.KV8(*a)
    with pytest.raises(api.TreespecError):
        api.QKRope(torch.zeros(32))
    with pytest.raises(api.TreespecError):
        api.tree_qk_norm_rope(None, None, None, None, api.QKRope(), None)


def test_rope_frequencies():
    f = api.QKRope.frequencies(64, 10000.0, device="cpu")
    assert f.shape == (32,) and f[0] == 1.0
    assert abs(float(f[16]) * 100.0 - 1.0) < 1e-6
