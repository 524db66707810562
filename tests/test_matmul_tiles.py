"""The 8-bit matrix product on 256-column tiles, element by element: both scale forms, every output type, relu, NaN, ragged
edges, several tiles to a pair of CTAs, more blocks than the ring of scales holds, and split sums.  Which kernel a size takes
is asked of the library's own plan, so that a change of its rules shows here.

The tolerance is that of the sums: products of 8 significant bits are exact, a block's 128 of them and then ceil(k / 128)
blocks are added one after another, each addition and scaling losing at most 2u = 2^-23 of the sum of magnitudes:
(128 + k / 128 + 4) 2u, and half an ulp of the stored type."""
import ctypes
import os
import subprocess

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

from . import test_gpu_wide as W

# m, n, k, tiles of 256 x 256, stretches
TILES = [(10000, 300, 200, 80, 1),       # some pairs take a second tile
         (5000, 700, 1300, 60, 1),       # one tile a pair, fewer tiles than pairs
         (10000, 700, 1300, 120, 1),     # two tiles of 11 blocks to a pair: the scales' ring of 16 wraps across tiles
         (9729, 257, 97, 78, 1),         # one ragged block, one column in the second tile
         (20001, 513, 640, 237, 1),      # four tiles a pair
         (10000, 256, 4100, 40, 1),      # 33 blocks to a tile
         (2000, 700, 10000, 24, 3)]      # split, and joined by one group
SMALL = (9800, 300, 200)                 # 78 tiles, for what depends on no sums


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = str(d / "plan.cpp"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write('#include "matmul_plan.h"\nextern "C" void plan(int m, int n, int k, int* o) {\n'
                "  const rs::Plan p = rs::plan_matmul(m, n, k);\n"
                "  o[0] = p.rows, o[1] = p.bn, o[2] = p.splits, o[3] = p.tiles, o[4] = p.workspace() > 0;\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build_lib.CSRC, "-I", build_lib.INCLUDE, "-o", lib,
                    src], check=True)
    L = ctypes.CDLL(lib)

    def ask(m, n, k):
        o = (ctypes.c_int * 5)()
        L.plan(m, n, k, o)
        return dict(zip(("rows", "bn", "splits", "tiles", "workspace"), o))

    return ask


def test_sizes_reach_the_kernels_they_are_meant_for(plan):
    for m, n, k, tiles, splits in TILES:
        assert plan(m, n, k) == dict(rows=0, bn=256, splits=splits, tiles=tiles, workspace=int(splits > 1)), (m, n, k)
    assert plan(*SMALL)["bn"] == 256
    # the measured sizes take the same kernel
    assert plan(160000, 512, 512)["bn"] == plan(65536, 2048, 2048)["bn"] == 256
    # and the sizes of the older tests the other two
    for m, n, k in W.SIZES:
        p = plan(m, n, k)
        assert p["rows"] == (0 if m > 64 else 16 if m <= 16 else 32 if m <= 32 else 64) and p["bn"] == 128, (m, n, k)


def test_every_kernel_is_used_by_some_size(plan):
    got = {(p["rows"], p["bn"], p["splits"] > 1, p["splits"] >= 10)
           for p in (plan(*s[:3]) for s in [*W.SIZES, *TILES, (70, 50, 80001)])}
    assert {(0, 256, False, False), (0, 256, True, False), (0, 128, False, False), (0, 128, True, False),
            (0, 128, True, True)} <= got and {16, 32, 64} <= {g[0] for g in got}


def test_plan_agrees_with_the_librarys_workspace(plan):
    build_lib.build()
    for m, n, k in [*W.SIZES, *(t[:3] for t in TILES)]:
        p = plan(m, n, k)
        need = rs.rs_matmul_fp8_workspace_size(m, n, k)
        assert need == (p["splits"] * p["tiles"] * 2 * p["bn"] * 128 * 4 if p["workspace"] else 0)


@pytest.fixture(scope="module")
def built():
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [t[:3] for t in TILES])
@pytest.mark.parametrize("blocks", [True, False])
def test_wide_tiles(built, m, n, k, blocks):
    g = W.gen(m + n * 3 + k * 5)
    a, sa, b, sb = W.operands(g, m, n, k, blocks)
    want, mags = W.product(a, sa, b, sb)
    sums = (128 + k / 128 + 4) * 2 * W.U
    got = W.matmul(a, sa, b, sb)
    W.close(got, want, sums * mags)
    assert torch.equal(got, W.matmul(a, sa, b, sb))
    assert torch.equal(W.matmul(a, sa, b, sb, relu=True), got.clamp_min(0))
    shrink = 100 / max(1.0, float(want.abs().max()))             # inside float16's range
    small = sb * shrink
    want, mags = W.product(a, sa, b, small)
    for dt in ("f16", "bf16"):
        tol = sums * mags + W.HALF_ULP[dt] * 1.01 * want.abs() + 2.0 ** -24
        got = W.matmul(a, sa, b, small, dt)
        W.close(got, want, tol)
        assert torch.equal(W.matmul(a, sa, b, small, dt, relu=True), got.clamp_min(0))


@pytest.mark.gpu
@pytest.mark.parametrize("blocks", [True, False])
def test_wide_tiles_keep_nan_in_its_row_and_column(built, blocks):
    m, n, k = SMALL
    a, sa, b, sb = W.operands(W.gen(32), m, n, k, blocks)
    base = W.matmul(a, sa, b, sb)
    a.view(torch.uint8)[777, 100] = 0x7f
    b.view(torch.uint8)[290, 199] = 0x7f
    out = W.matmul(a, sa, b, sb, relu=True)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[777], bad[:, 290] = True, True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], base.clamp_min(0)[~bad])
