"""Gradients as small as a loss over an image gives them (1e-7 a value and less) through the wide network's backward.

The whole backward is linear in dL/dcolours, and a power of two passes every one of its steps exactly: float32 sums, e4m3 values
with a scale a block, 16-bit roundings, as long as nothing leaves the normal numbers.  So gradients of dL/dcolours 2^-k
are the gradients of dL/dcolours, times 2^-k, bit for bit; the largest are around 1 and float32 (and bfloat16) reach down to 2^-126."""
import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, pipeline, rs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


def gradients(net, dcol):
    net.backward(dcol)
    return [g.clone() for _, g in net.parameters()]


def network(dtype, n=900):
    g = torch.Generator("cuda").manual_seed(6)
    net = pipeline.WideAppearance(torch.randn(n, 160, device="cuda", generator=g), 192, 2, dtype, seed=6)
    net.forward()
    return net, torch.randn(3, n, device="cuda", generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", [0, 10, 24, 40, -6])
def test_small_gradients_are_scaled_gradients(dtype, k):
    net, dcol = network(dtype)
    base = gradients(net, dcol)
    assert all(bool(torch.isfinite(g).all()) and float(g.abs().max()) > 0 for g in base)
    for a, b in zip(gradients(net, dcol * 2.0 ** -k), base):
        assert torch.equal(a, b * 2.0 ** -k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_no_gradient_and_gradients_that_are_not_finite(dtype):
    net, dcol = network(dtype)
    assert all(float(g.abs().max()) == 0 for g in gradients(net, torch.zeros_like(dcol)))
    for bad in (float("inf"), float("nan")):
        d = dcol.clone()
        d[1, 7] = bad
        net.backward(d)
        net.step(1.0)
        assert int(net.steps) == 0 and not bool(torch.isfinite(net.norm))


def test_no_gaussians():
    net = pipeline.WideAppearance(torch.empty(0, 64, device="cuda"), 64, 1, torch.float16)
    net.forward()
    net.backward(torch.empty(3, 0, device="cuda"))
    assert all(float(g.abs().sum()) == 0 for _, g in net.parameters())


def test_float16_scaled_gradients_in_a_graph():
    net, dcol = network(torch.float16)
    dcol = dcol * 1e-7
    want = gradients(net, dcol)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.backward(dcol)
    for _, g in net.parameters():
        g.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for (_, g), w in zip(net.parameters(), want))
