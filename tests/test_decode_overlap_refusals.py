"""sample_tokens refuses an output that lies, whole or in part, on u or on a row's settings; pointers are never followed."""
import ctypes as C

import pytest
import torch

from tree_speculative_verification_gb300 import api, build

P = C.c_void_p
SETTINGS = ("u", "temperature", "top_k", "top_p", "min_p")
R, V = 6, 100


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def call(lib, **at):
    """Arrays far apart, but for those whose place is given."""
    names = ("token", "probs", "kept", "logits") + SETTINGS
    a = {n: at.get(n, 0x100000 * (i + 1)) for i, n in enumerate(names)}
    return lib.sample_tokens(*[P(a[n]) for n in ("token", "probs", "kept", "logits")], V, 0, *[P(a[n]) for n in SETTINGS], R, V, None, None)


@pytest.mark.parametrize("setting", SETTINGS)
@pytest.mark.parametrize("output,entries", [("token", R), ("probs", R * V), ("kept", R * V)])
def test_outputs_on_settings(lib, setting, output, entries):
    for off in (0, 4, 4 * (R - 1), -4, -4 * (entries - 1), -4 * (entries // 2)):
        assert call(lib, **{output: 0x4000000, setting: 0x4000000 - off}) == api.TS_ERR_INVALID_ARG, off
        assert output.encode() in lib.treespec_last_error() and b"place of its own" in lib.treespec_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers would be followed")
def test_arrays_next_to_one_another(lib):
    """Ends that touch are apart, and inputs may be one array."""
    for setting in SETTINGS:
        for output, entries in (("token", R), ("probs", R * V), ("kept", R * V)):
            for off in (4 * R, -4 * entries):
                assert call(lib, **{output: 0x4000000, setting: 0x4000000 - off}) == api.TS_ERR_CUDA, (setting, output, off)
    assert call(lib, u=0x4000000, temperature=0x4000000, top_p=0x4000000, min_p=0x4000000) == api.TS_ERR_CUDA
