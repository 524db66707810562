"""The clipped Adam step whose number is counted on the device, and the wide network's step captured in a graph.

The corrections are formed from beta^t in double on both sides and rounded to float32, so they differ by one rounding at most: a
relative 2^-23 each, of which the square root halves the second.  With the update's own four roundings a parameter moves by
at most 8 x 2^-24 of the update further, plus half an ulp of itself.  Moments do not depend on them."""
import ctypes
import math

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, pipeline, rs

from . import test_gpu_wide as W

P = ctypes.c_void_p(0x10000)


def test_refusals():
    build_lib.build()
    L = rs.lib()
    need = rs.rs_grad_norm_workspace_size(1)
    seg = (rs.rs_adam_segment * 1)()
    s = seg[0]
    s.d_param = s.d_grad = s.d_m = s.d_v = 0x10000
    s.count, s.lr, s.activation = 10, 0.01, 0
    call = lambda steps=P, b1=0.9, limit=1.0, norm=P, ws=P, bytes=need, n=1: L.rs_adam_step_clipped_counted(
        seg, n, b1, 0.999, 1e-15, steps, limit, norm, ws, bytes, None)
    for c in (dict(steps=None), dict(steps=ctypes.c_void_p(0x10002)), dict(b1=1.0), dict(limit=0.0), dict(norm=None), dict(ws=None),
              dict(n=17)):
        assert call(**c) == rs.RS_ERR_INVALID_ARG, c
    assert call(bytes=need - 1) == rs.RS_ERR_WORKSPACE
    with pytest.raises(TypeError):
        rs.rs_adam_step_clipped([], torch.zeros(1, dtype=torch.int32), 1.0, None, torch.zeros(1, dtype=torch.uint8))


@pytest.fixture(scope="module")
def built():
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


def counter(v=0):
    return torch.full((1,), v, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("taken", [0, 1, 9, 99, 12344, 1000000])
@pytest.mark.parametrize("sizes", [[1], [3 * 1007, 1007, 0, 45 * 1007 - 5], []])
def test_counted_step_is_the_step_of_that_number(built, taken, sizes):
    a = W.adam_groups(W.gen(taken + len(sizes)), sizes)
    b = W.copy_groups(a)
    start = W.copy_groups(a)
    norms, ws, steps = torch.full((2,), -1.0, device="cuda"), W.clip_ws(max(1, len(a))), counter(taken)
    rs.rs_adam_step_clipped(a, steps, 1.0, norms[:1], ws)
    rs.rs_adam_step_clipped(b, taken + 1, 1.0, norms[1:], ws)
    assert int(steps) == taken + 1 and float(norms[0]) == float(norms[1]) >= 0
    for x, y, z in zip(a, b, start):
        assert torch.equal(x.m, y.m) and torch.equal(x.v, y.v)
        moved = (y.param.double() - z.param.double()).abs()
        W.close(x.param, y.param, 8 * W.U * moved + 2 * W.U * y.param.double().abs())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_skipped_steps_do_not_count(built, bad):
    """A first step that is skipped leaves the next one the first."""
    a = W.adam_groups(W.gen(3), [1000, 999])
    b = W.copy_groups(a)
    norm, ws, steps, other = torch.empty(1, device="cuda"), W.clip_ws(2), counter(), counter()
    good = a[1].grad.clone()
    a[1].grad[7] = bad
    rs.rs_adam_step_clipped(a, steps, 1.0, norm, ws)
    assert int(steps) == 0 and not math.isfinite(float(norm)) and torch.equal(a[1].param, b[1].param)
    a[1].grad.copy_(good)
    rs.rs_adam_step_clipped(a, steps, 1.0, norm, ws)
    rs.rs_adam_step_clipped(b, other, 1.0, norm, ws)
    assert int(steps) == int(other) == 1 and W.same_groups(a, b)


def network(seed=5):
    g = torch.Generator("cuda").manual_seed(seed)
    net = pipeline.WideAppearance(torch.randn(500, 128, device="cuda", generator=g), 128, 1, seed=seed)
    return net, torch.randn(3, 500, device="cuda", generator=g)


@pytest.mark.gpu
def test_captured_training_is_eager_training(built):
    """Forward, backward and step captured after one step: replays give what eager steps give, bit for bit."""
    (eager, dcol), (net, _) = network(), network()

    def once(n):
        n.forward()
        n.backward(dcol)
        n.step(1.0, 1e-2)

    for _ in range(6):
        once(eager)
    once(net)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(net)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert int(net.steps) == int(eager.steps) == 6
    assert all(torch.equal(x, y) for (x, _), (y, _) in zip(net.parameters(), eager.parameters()))
    assert all(torch.equal(x, y) for p, q in zip(net.moments, eager.moments) for x, y in zip(p, q))


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_first_step_is_not_captured(built):
    net, dcol = network()
    net.forward()
    net.backward(dcol)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="moments"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            net.step(1.0)
    net.step(1.0)
    assert int(net.steps) == 1


@pytest.mark.gpu
def test_network_does_not_count_skipped_or_refused_steps(built):
    (net, dcol), (fresh, _) = network(), network()
    net.forward()
    net.backward(torch.full_like(dcol, float("nan")))
    net.step(1.0)
    assert int(net.steps) == 0
    many = [rs.AdamGroup(*(torch.zeros(4, device="cuda") for _ in range(4)), 1e-3)] * 16
    with pytest.raises(ValueError):
        net.step(1.0, groups=many)
    assert int(net.steps) == 0
    for n in (net, fresh):
        n.forward()
        n.backward(dcol)
        n.step(1.0)
    assert int(net.steps) == 1 and all(torch.equal(x, y) for (x, _), (y, _) in zip(net.parameters(), fresh.parameters()))
