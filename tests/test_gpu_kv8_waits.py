"""The waits of the 8-bit cache's attention, in a kernel of their own: one that nothing ends gives up after the library's
limit."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from tree_speculative_verification_gb300 import build

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "kv8_wait.cuh"
using namespace ts;
__global__ void k_waits(int *verdict, long long *cycles) {
    __shared__ unsigned long long bars[2];
    const unsigned never = (unsigned)__cvta_generic_to_shared(&bars[0]), there = (unsigned)__cvta_generic_to_shared(&bars[1]);
    if (threadIdx.x == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(never));
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(there));
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(there) : "memory");
    }
    __syncthreads();
    const int warp = threadIdx.x / 32;
    const long long t0 = clock64();
    const bool found = wait_warp(there, 0);
    const long long t1 = clock64();
    const bool ended = wait_warp(never, 0);   // three warps wait for what nobody does
    const long long t2 = clock64();
    if (threadIdx.x % 32 == 0) {
        verdict[warp * 2] = found;
        verdict[warp * 2 + 1] = ended;
        cycles[warp * 3] = t1 - t0;
        cycles[warp * 3 + 1] = t2 - t1;
        cycles[warp * 3 + 2] = kWaitCycles;
    }
}
extern "C" int run_waits(void *verdict, void *cycles, cudaStream_t s) {
    k_waits<<<1, 96, 0, s>>>((int *)verdict, (long long *)cycles);
    return (int)cudaGetLastError();
}
"""


def test_a_wait_that_nothing_ends(tmp_path):
    src, lib = tmp_path / "waits.cu", tmp_path / "waits.so"
    src.write_text(SOURCE)
    subprocess.run([build.nvcc(), *build._flags(False), f"-I{build.CSRC}", "-shared", "-o", str(lib), str(src)], check=True)
    assert os.path.exists(lib)
    f = C.CDLL(str(lib)).run_waits
    f.argtypes = [C.c_void_p] * 3
    verdict = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    cycles = torch.zeros((3, 3), dtype=torch.int64, device="cuda")
    assert f(verdict.data_ptr(), cycles.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    limit = int(cycles[0, 2])
    assert verdict.tolist() == [[1, 0]] * 3
    # the library's limit, some 2 s, within a factor of two (a wait counts tries, which the hardware suspends)
    assert (cycles[:, 0] < limit / 1000).all(), cycles.tolist()
    assert (cycles[:, 1] >= limit / 2).all() and (cycles[:, 1] < limit * 2).all(), cycles.tolist()
