"""Calls of the 8-bit cache's entry points that pass every check, where there is no device to launch on: an error code
comes back, whatever is left out of the call (the pointers are never followed)."""
import ctypes as C

import pytest
import torch

from tree_speculative_verification_gb300 import api, build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers would be followed")
X = C.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def tree(B=2, n_max=8):
    return C.byref(api.ts_tree(B, n_max, *([0x10000] * 9)))


def cache(d):
    return C.byref(api.ts_kv8(*([0x10000] * 4), None, 2, 4, d, 64, 0, 0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (4, 0), (0, 2)])
def test_norm_rope(lib, d, Hq, Hk):
    r = C.byref(api.ts_qk_rope(0x10000, None, None, 1e-6, 1, 64, 0))
    assert lib.tree_qk_norm_rope(X, X, X, X, Hq, Hk, d, max(1, Hq) * d, max(1, Hk) * d, r, tree(), api.TS_BF16, None,
                                 None) == api.TS_ERR_CUDA


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [0, 8])
def test_append(lib, d, Hq):
    r = C.byref(api.ts_qk_rope(0x10000, None, None, 1e-6, 1, 64, 0))
    assert lib.kv8_append(cache(d), X, X, 4 * d, 4 * d, r, X, X, Hq, 8 * d, X, tree(), api.TS_F32, None,
                          None) == api.TS_ERR_CUDA


@pytest.mark.parametrize("d", [64, 128])
def test_read_commit_attention(lib, d):
    assert lib.kv8_read(X, X, cache(d), None, X, 64, api.TS_BF16, None, None) == api.TS_ERR_CUDA
    assert lib.kv8_commit(cache(d), X, C.c_void_p(0x20000), X, X, tree(), None, None) == api.TS_ERR_CUDA
    assert lib.tree_attention_kv8(X, X, cache(d), 8, X, tree(), 0.0, X, 1 << 30, None, None) == api.TS_ERR_CUDA
