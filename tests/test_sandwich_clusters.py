"""How many clusters the sandwich norm's backward launches for rows of more than 4096 columns, and what it answers when the
question of how many the GPU holds fails.  The library's compiled host code runs against a CUDA runtime made for this test
(CPU only: nothing reaches a GPU)."""
import ctypes
import os
import subprocess

import pytest

from gaussian_splatting_tile_gb300 import build_lib, rs

FAKE = r"""
#include <cstddef>
extern "C" {
int most = 0, failures = 0, launches = 0;
unsigned first_grid = 0;
int cudaOccupancyMaxActiveClusters(int* n, const void*, const void*) {
    if (failures > 0) return --failures, 999;
    *n = most;
    return 0;
}
int cudaLaunchKernelExC(const unsigned* cfg, const void*, void**) {
    if (launches++ == 0) first_grid = cfg[0];
    return 0;
}
int cudaFuncSetAttribute(const void*, int, int) { return 0; }
int cudaMemsetAsync(void*, int, size_t, void*) { return 0; }
int __cudaGetKernel(void** k, const void* f) { return *k = const_cast<void*>(f), 0; }
int __cudaLaunchKernel() { return 1; }
int __cudaPopCallConfiguration() { return 1; }
void** __cudaRegisterFatBinary(void*) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaRegisterFunction() {}
void __cudaUnregisterFatBinary(void**) {}
}
"""


@pytest.fixture
def L(tmp_path):
    build_lib.build()
    src, lib = str(tmp_path / "fake.cpp"), str(tmp_path / "fake.so")
    with open(src, "w") as f:
        f.write(FAKE)
    # every symbol is the library's own: torch brings a CUDA runtime into the process
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-o", lib, src,
                    os.path.join(build_lib.BUILD, "sandwich_bwd.o")], check=True)
    L = ctypes.CDLL(lib)
    L.rs_sandwich_norm_bwd.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    return L


def call(L, rows, cols):
    """(answer, first launch's CTAs)"""
    p, q = 0x10000, 0x20000
    block = rs.rs_sandwich(rows=rows, cols=cols, dtype=rs.RS_BF16, gate_cols=0, d_x=p,
                           x_stride=cols, d_r=p, r_stride=cols, d_post_weight=p, d_pre_weight=p)
    grads = rs.rs_sandwich_grads(d_rstd_r=p, d_rstd_s=p, d_dL_dy=p, dy_stride=cols, d_dL_dx=q, dx_stride=cols, d_dL_dr=p,
                                 dr_stride=cols)
    ctypes.c_int.in_dll(L, "launches").value = 0
    got = L.rs_sandwich_norm_bwd(ctypes.byref(block), ctypes.byref(grads), None, 0, None)
    return got, ctypes.c_uint.in_dll(L, "first_grid").value if ctypes.c_int.in_dll(L, "launches").value else 0


@pytest.mark.parametrize("cols,ctas", [(5000, 2), (8192, 2), (9000, 4), (16384, 4)])
def test_a_failed_question_costs_one_call(L, cols, ctas):
    ctypes.c_int.in_dll(L, "most").value = 10
    ctypes.c_int.in_dll(L, "failures").value = 1
    assert call(L, 1000, cols) == (rs.RS_ERR_CUDA, 0)
    assert call(L, 1000, cols) == (rs.RS_OK, 10 * ctas)
    assert call(L, 3, cols) == (rs.RS_OK, 3 * ctas)


def test_each_call_goes_by_its_own_device(L):
    """A GPU that holds fewer clusters than the one before."""
    for most, want in ((38, 38), (7, 7), (0, None), (1000, 38)):
        ctypes.c_int.in_dll(L, "most").value = most
        got = call(L, 1000, 16384)
        assert got == ((rs.RS_OK, want * 4) if want else (rs.RS_ERR_CUDA, 0)), most
