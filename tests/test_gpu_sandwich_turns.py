"""The sandwich norm's backward where a block takes many rows one after another: its ring of copies is filled again and again, and
the vectors' gradients are sums over long chains of rows.  How many rows a block takes is asked of the library's own rule, so that
a change of it shows here.

Tolerance of the vectors' gradients: a thread adds its rows' shares one after another, the rows of a block are joined, then 32
threads add every 32nd block's sum, and five exchanges add those: no chain of additions is longer than turns + rows a block +
ceil(blocks / 32) + 5, each step off by 2^-24 of the terms' magnitudes.  The terms' own errors and everything else are those
of test_gpu_sandwich."""
import ctypes
import subprocess

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

from . import test_gpu_sandwich as S

# rows, columns: at least six turns a block (twice the stages of the ring), whatever the type and the handing over
RAGGED = [(25000, 77), (16000, 129), (10000, 257), (12000, 450), (4000, 777), (2000, 1203), (2000, 2045), (1000, 2601),
          (1000, 4095), (600, 8193), (600, 4801)]
WHOLE = [(25000, 64), (16000, 136), (4000, 768), (2000, 1536), (1000, 3000), (600, 8192)]
U = S.U


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = str(d / "plan.cpp"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write('#include "sandwich_plan.h"\nextern "C" void ask(int rows, int cols, int f32, int* o) {\n'
                "  o[0] = rs::bwd_rows(cols, f32), o[1] = rs::bwd_blocks(rows, cols, f32);\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build_lib.CSRC, "-I", build_lib.INCLUDE, "-o", lib,
                    src], check=True)
    L = ctypes.CDLL(lib)

    def ask(rows, cols, dt):
        """(rows a block takes at once, blocks, turns of a block)"""
        o = (ctypes.c_int * 2)()
        L.ask(rows, cols, int(dt == "f32"), o)
        return o[0], o[1], -(-rows // (o[0] * o[1]))

    return ask


@pytest.mark.parametrize("rows,cols", RAGGED + WHOLE)
def test_sizes_take_many_turns(rule, rows, cols):
    assert all(rule(rows, cols, dt)[2] >= 6 for dt in S.DT)


def test_workspace_holds_every_block(rule):
    build_lib.build()
    for rows, cols in RAGGED + WHOLE + [(1, 1), (3, 16384), (0, 5)]:
        blocks = max(1, *(rule(rows, cols, dt)[1] for dt in S.DT)) if rows else 1
        assert rs.rs_sandwich_norm_bwd_workspace_size(rows, cols) == blocks * 3 * cols * 4


def check_vectors(b, o, dy, dsum, got, chain):
    """dalpha, dpost and dpre as in S.check_backward, with that chain of additions."""
    x, r, z, al = b.operands()
    rho_r, rho_s = o["rstd_r"].double()[:, None], o["rstd_s"].double()[:, None]
    wpost, wpre, dy, d = b.wpost.double(), b.wpre.double(), dy.double(), dsum.double()
    mean = lambda t: t.mean(1, keepdim=True)
    g, eg, _ = S.gate_of(z)
    rh = r * rho_r
    p = g * rh * wpost
    ep = p.abs() * (5 * U + eg)
    sh = (al * x + p) * rho_s
    es = rho_s * (3 * U * (al * x).abs() + ep) + 2 * U * sh.abs()
    t = dy * wpre
    a1, ea = mean(t * sh), mean(t.abs() * es) + 68 * U * mean((t * sh).abs())
    ds = rho_s * (t - sh * a1) + d
    eds = (3 * U * ((rho_s * t).abs() + d.abs()) + rho_s * (sh.abs() * ea + a1.abs() * es + 4 * U * (sh * a1).abs()) +
           U * ds.abs())
    dn = ds * g
    edn = eds * g + dn.abs() * (eg + U)
    for have, v, e in ((got[3], ds * x, eds * x.abs()), (got[4], dn * rh, edn * rh.abs()), (got[5], dy * sh, dy.abs() * es)):
        S.close(have, v.sum(0), e.sum(0) + (chain + 3) * U * v.abs().sum(0) + 1e-37)


def run(rule, rows, cols, dt, kept, gate):
    g = S.gen(rows + cols)
    b = S.Block(g, rows, cols, dt, gate)
    dy, dsum = S.grads_of(g, b)
    o = b.forward(kept)
    if kept:
        S.keep(b, o)
    got = S.check_backward(b, o, dy, dsum)
    at_once, blocks, turns = rule(rows, cols, dt)
    check_vectors(b, o, dy, dsum, got, turns + at_once + -(-blocks // 32) + 5)
    again = S.backward(b, o, dy, dsum)
    assert all(v is None or torch.equal(v, w) for v, w in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", RAGGED)
def test_rows_between_boundaries(rule, rows, cols, dt, kept):
    run(rule, rows, cols, dt, kept, "element")


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", WHOLE)
def test_rows_on_boundaries(rule, rows, cols, dt, kept):
    run(rule, rows, cols, dt, kept, "row" if rows % 3 else "element")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_over_their_upstream_in_many_turns(rule, dt):
    """In place, where rows share words: what one row writes is in no other's copies."""
    rows, cols = 8000, 301
    assert rule(rows, cols, dt)[2] >= 6
    g = S.gen(3)
    b = S.Block(g, rows, cols, dt)
    dy, dsum = S.grads_of(g, b)
    o = b.forward()
    want = S.backward(b, o, dy, dsum)
    for swap in (False, True):
        a, d = dy.clone(), dsum.clone()
        got = S.backward(b, o, a, d, out=(d, a) if swap else (a, d))
        assert all(torch.equal(v, w) for v, w in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [777, 8193])
def test_captured_backward_of_many_turns(cols):
    """Captured before it has ever run eagerly at this size, replayed with other inputs."""
    rows = 500
    g = S.gen(8)
    b = S.Block(g, rows, cols, "f16")
    dy, dsum = S.grads_of(g, b)
    o = b.forward()
    dx, dr = torch.empty_like(dy), torch.empty_like(dy)
    post = torch.empty(cols, device="cuda")
    ws = torch.empty(rs.rs_sandwich_norm_bwd_workspace_size(rows, cols), dtype=torch.uint8, device="cuda")

    def step():
        rs.rs_sandwich_norm_bwd(b.x, b.r, b.wpost, b.wpre, o["rstd_r"], o["rstd_s"], dy, dx, dr, ws, gate=b.gate,
                                residual_scale=b.alpha, dL_dsum=dsum, dL_dpost_weight=post)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in (dx, dr, post):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (dx, dr, post)]
        step()
        assert all(torch.equal(a, c) for a, c in zip(got, (dx, dr, post)))
        dy.copy_(S.rand(g, rows, cols))


@pytest.fixture(scope="module", autouse=True)
def clean():
    yield
    if torch.cuda.is_available():
        assert rs.rs_device_error() == rs.RS_OK
