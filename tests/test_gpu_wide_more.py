"""Gradient clipping, the clipped Adam step and the 128 x 128 forms at sizes and types that real scenes have: blocks that take
several chunks of several tensors, and 16-bit weights.

The norm's tolerance, u = 2^-24: a thread adds 32 values of each of its chunks, ceil(chunks / 1216) of them (a launch has up to
1216 blocks) and one sum a chunk, then 5 exchanges and 8 warps; the up to 1216 partial sums a launch are added 256 apart, ceil(parts / 256) to
a thread, then 5 exchanges and 8 warps.  All terms are positive and added in float32, so the sum is within (length of the longest
chain) u; the square root halves that and rounds once, and squares add one rounding.  Float16 and bfloat16 values are
squared exactly enough (22 and 16 bits)."""
import math

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

from . import test_gpu_wide as W

pytestmark = pytest.mark.gpu
CHUNK, BLOCKS = 8192, 1216


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


def norm_tolerance(sizes, extra=0):
    chunks = sum(-(-k // CHUNK) for k in sizes)
    assert chunks > BLOCKS                                       # some block takes a second chunk
    rounds = -(-chunks // BLOCKS)
    chain = 33 * rounds + 5 + 8 + -(-min(chunks, BLOCKS) // 256) + 5 + 8 + 1 + extra
    return (chain / 2 + 1) * W.U


def coefficient(limit, norm):
    return float(min(np.float32(1), np.float32(limit) / (np.float32(float(norm)) + np.float32(1e-6))))


# one long tensor; tensors whose boundaries lie in a block's later chunks, odd sizes among them
@pytest.mark.parametrize("sizes", [[25_000_000], [600_000] * 40, [9_000_001, 5, 8192, 3_000_017, 1, 12_345_678]])
@pytest.mark.parametrize("limit", [0.25, 4.0])
def test_clip_of_many_chunks(sizes, limit):
    g = W.gen(len(sizes))
    ts = W.tensors(g, sizes)
    want = math.sqrt(sum(float(t.double().pow(2).sum()) for t in ts))
    outs = [torch.full_like(t, 9.0) for t in ts]
    norm, ws = torch.empty(1, device="cuda"), W.clip_ws(len(ts))
    rs.rs_grad_clip([rs.GradTensor(t, out=o) for t, o in zip(ts, outs)], limit * want, norm, ws)
    assert abs(float(norm) / want - 1) < norm_tolerance(sizes)
    c = coefficient(limit * want, norm)
    for t, o in zip(ts, outs):
        assert torch.equal(o, (t.float() * c).to(t.dtype))
    again = torch.empty(1, device="cuda")
    rs.rs_grad_norm([rs.GradTensor(t) for t in ts], again, ws)
    assert torch.equal(norm, again)
    rs.rs_grad_clip([rs.GradTensor(t, out=t) for t in ts], limit * want, norm, ws)
    assert all(torch.equal(t, o) for t, o in zip(ts, outs))


def test_clip_of_unaligned_tensors_of_many_chunks():
    flat = W.rand(W.gen(4), 24_000_010)
    ts = [flat[1:10_000_004], flat[10_000_005:24_000_009]]
    out = torch.full_like(flat, 9.0)
    places = [out[t.storage_offset():t.storage_offset() + t.numel()] for t in ts]
    norm = torch.empty(1, device="cuda")
    rs.rs_grad_clip([rs.GradTensor(t, out=o) for t, o in zip(ts, places)], 1.0, norm, W.clip_ws(2))
    want = math.sqrt(sum(float(t.double().pow(2).sum()) for t in ts))
    assert abs(float(norm) / want - 1) < norm_tolerance([t.numel() for t in ts])
    c = coefficient(1.0, norm)
    assert all(torch.equal(o, t * c) for t, o in zip(ts, places))
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep[1:10_000_004] = keep[10_000_005:24_000_009] = False
    assert bool((out[keep] == 9.0).all())


@pytest.mark.parametrize("sizes", [[12_000_001, 3, 4_000_000], [3 * 400_003, 3 * 400_003, 4 * 400_003, 400_003, 45 * 400_003]])
@pytest.mark.parametrize("counted", [False, True])
def test_adam_step_clipped_of_many_chunks(sizes, counted):
    """More than the 2.5 M values of one pass of the step's blocks."""
    a = W.adam_groups(W.gen(sizes[0]), sizes)
    b = W.copy_groups(a)
    want = math.sqrt(sum(float(W.chained(q).pow(2).sum()) for q in a))
    norm = torch.empty(1, device="cuda")
    step = torch.full((1,), 2, dtype=torch.int32, device="cuda") if counted else 3
    rs.rs_adam_step_clipped(a, step, 0.3 * want, norm, W.clip_ws(len(a)))
    # a sigmoid's derivative: exp, sum, quotient and three products, 2u each at most, counted twice by the square
    assert abs(float(norm) / want - 1) < norm_tolerance(sizes, extra=24)
    c = coefficient(0.3 * want, norm)
    for q in b:
        q.grad = q.grad * c
    rs.rs_adam_step(b, 3)
    assert W.same_groups(a, b)                                   # (at step 3 both ways round the corrections alike)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 257), (300, 77), (77, 301), (512, 256)])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_quantize_blocks_of_16_bits(dt, rows, cols, pad):
    """As for float32: the definition bit for bit, both ways round, whatever the rows' distance."""
    w = W.rand(W.gen(rows), rows, cols + pad).to(W.DT[dt])[:, :cols]
    rb, cb = -(-rows // 128), -(-cols // 128)
    q, qt = rs.fp8_empty(rows, cols)[0], rs.fp8_empty(cols, rows)[0]
    sc, sct = torch.empty(cb, rb, device="cuda"), torch.empty(rb, cb, device="cuda")
    rs.rs_quantize_fp8_blocks(w, q, sc, qt, sct)
    full = torch.zeros(rb * 128, cb * 128)
    full[:rows, :cols] = w.float().cpu()
    top = full.view(rb, 128, cb, 128).abs().amax((1, 3)).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    factors = (f / top).repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = (full * factors).clamp(-448, 448).to(torch.float8_e4m3fn).float()[:rows, :cols]
    assert torch.equal(q.float().cpu(), want) and torch.equal(qt.float().cpu(), want.t())
    assert torch.equal(sc.cpu(), (top / f).t()) and torch.equal(sct.cpu(), top / f)
    for one in (0, 1):                                           # each form alone gives the same
        q1, s1 = (rs.fp8_empty(rows, cols)[0], torch.empty_like(sc)) if one == 0 else (rs.fp8_empty(cols, rows)[0], torch.empty_like(sct))
        rs.rs_quantize_fp8_blocks(w, **(dict(q=q1, scales=s1) if one == 0 else dict(qt=q1, scales_t=s1)))
        assert torch.equal(q1.view(torch.uint8), (q, qt)[one].view(torch.uint8)) and torch.equal(s1, (sc, sct)[one])
