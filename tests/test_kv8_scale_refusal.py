"""tree_attention_kv8 refuses a scale whose scores, as exponents of 2, would be infinite or NaN whatever the keys."""
import ctypes as C

import pytest
import torch

from tree_speculative_verification_gb300 import api, build

X = C.c_void_p(0x10000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def call(lib, scale):
    kv = api.ts_kv8(*([0x10000] * 4), None, 2, 4, 128, 64, 0, 0)
    t = api.ts_tree(2, 8, *([0x10000] * 9))
    return lib.tree_attention_kv8(X, X, C.byref(kv), 8, X, C.byref(t), scale, X, 1 << 30, None, None)


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, float("inf")])
def test_refused(lib, scale):
    assert call(lib, scale) == api.TS_ERR_INVALID_ARG
    assert b"scale" in lib.treespec_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers would be followed")
@pytest.mark.parametrize("scale", [0.0, -1.0, float("nan"), 1e-30, 2.3e38])
def test_taken(lib, scale):
    assert call(lib, scale) == api.TS_ERR_CUDA        # every check passed; there is no device
