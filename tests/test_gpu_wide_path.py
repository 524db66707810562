"""The wide appearance network as a user runs it: forward, backward, clipped step, with the renderer around it.

Every stage is checked against float64 from the network's own inputs to that stage, float32 activations (a difference in
the last bit of one value can move it across a tie of e4m3, and from there spread over its row: a chain of stages
has no useful bound).  Tolerances, in the 2-norm: 1e-5 where a stage's inputs are at hand (float32 sums, each error below 1e-6 of
its terms' magnitudes); 1e-3 where they had to be recomputed, as the gradient of the inner sum: a relative difference of 1e-6
crosses a tie (steps of 1/16) with a probability of 3.2e-5 and then changes a value by 1/16, 3.5e-4 of the operand's norm."""
import numpy as np
import pytest
import torch

from gaussian_splatting_tile_gb300 import pipeline, rs, scenes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from gaussian_splatting_tile_gb300 import build_lib
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


def rows8(x):
    """The values of x's 8-bit form by rows (float64 out, the form itself in float32 as defined)."""
    r, c = x.shape
    kb = -(-c // 128)
    xp = torch.nn.functional.pad(x.float(), (0, kb * 128 - c)).view(r, kb, 128)
    top = xp.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    return ((xp * (f / top)).to(torch.float8_e4m3fn).double() * (top / f).double()).view(r, kb * 128)[:, :c]


def cols8(x):
    return rows8(x.t()).t()


def blocks8(w):
    o, i = w.shape
    wp = torch.nn.functional.pad(w, (0, -i % 128, 0, -o % 128))
    t = wp.view(wp.shape[0] // 128, 128, wp.shape[1] // 128, 128)
    top = t.abs().amax((1, 3), keepdim=True).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    return ((t * (f / top)).to(torch.float8_e4m3fn).double() * (top / f).double()).reshape(wp.shape)[:o, :i]


def near(got, want, tol=1e-5):
    assert got.shape == want.shape
    rel = float((got.double() - want).norm() / want.norm())
    assert rel < tol, rel


def norm_bwd(h, w, dy, ds):
    h, w, dy = h.double(), w.double(), dy.double()
    rho = 1 / (h.pow(2).mean(1, keepdim=True) + 1e-6).sqrt()
    xh, t = h * rho, dy * w
    return rho * (t - xh * (t * xh).mean(1, keepdim=True)) + ds, (dy * xh).sum(0)


@pytest.mark.parametrize("n,width,hidden", [(777, 96, 200), (3000, 256, 512), (130, 130, 64)])
def test_stages(n, width, hidden):
    g = torch.Generator("cuda").manual_seed(n)
    net = pipeline.WideAppearance(torch.randn(n, width, device="cuda", generator=g), hidden, 1, torch.float32, seed=3)
    for w in net.norms:
        w.add_(0.2 * torch.randn(width, device="cuda", generator=g))
    dcol = torch.randn(3, n, device="cuda", generator=g)
    net.forward()
    W1, W2, Wo = blocks8(net.up[0].w), blocks8(net.down[0].w), blocks8(net.head.w)
    h0, h1, y0, y1, u = net.h[0], net.h[1], net.y[0], net.y[1], net.u[0]
    assert torch.equal(h0, net.features) and torch.equal(h1, h0 + net.r)
    for h, y, w in ((h0, y0, net.norms[0]), (h1, y1, net.norms[1])):
        near(y, h.double() / (h.double().pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * w.double())
    near(u, torch.relu(rows8(y0) @ W1.t()))
    near(net.r, rows8(u) @ W2.t())
    near(net.z, rows8(y1) @ Wo.t())
    near(net.colors, torch.sigmoid(net.z.double()).t())
    net.backward(dcol)
    dz = (dcol * net.colors * (1 - net.colors)).t().contiguous()
    near(net.head.dw, cols8(dz).t() @ cols8(y1))
    dh1, dg1 = norm_bwd(h1, net.norms[1], rows8(dz) @ Wo, 0)
    near(net.dnorms[1], dg1)
    near(net.down[0].dw, cols8(dh1).t() @ cols8(u), 1e-3)
    near(net.du, rows8(dh1) @ W2, 1e-3)
    du = net.du * (u > 0)
    near(net.up[0].dw, cols8(du).t() @ cols8(y0))
    near(net.dy, rows8(du) @ W1)
    dh0, dg0 = norm_bwd(h0, net.norms[0], net.dy, dh1)
    near(net.dfeatures, dh0)
    near(net.dnorms[0], dg0)


def test_a_block_that_adds_nothing_changes_nothing():
    """Two blocks, the second with W2 = 0, are one block bit for bit: the blocks' chain, forward and backward."""
    F = torch.randn(500, 160, device="cuda")
    one, two = (pipeline.WideAppearance(F.clone(), 192, b, torch.float32, seed=4) for b in (1, 2))
    for a, b in ((one.up[0], two.up[0]), (one.down[0], two.down[0]), (one.head, two.head)):
        b.w.copy_(a.w)
    two.down[1].w.zero_()
    for layer in (*two.up, *two.down, two.head):
        layer.refresh()
    dcol = torch.randn(3, 500, device="cuda")
    for net in (one, two):
        net.forward()
        net.backward(dcol)
    pairs = [(one.colors, two.colors), (one.dfeatures, two.dfeatures), (one.head.dw, two.head.dw), (one.up[0].dw, two.up[0].dw),
             (one.down[0].dw, two.down[0].dw), (one.dnorms[0], two.dnorms[0]), (one.dnorms[1], two.dnorms[2])]
    assert all(torch.equal(a, b) for a, b in pairs)
    assert float(two.up[1].dw.abs().max()) == 0 and float(two.dnorms[1].abs().max()) == 0
    assert float(two.down[1].dw.abs().max()) > 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_16_bit_activations_stay_near_float32(dtype):
    """Roundings to 16 bits (2^-8 at most) move more values across e4m3's ties: at most 2^-8 / (1/16) = 1 in 16, each by
    1/16 of itself: 1/64 of an operand's norm for each of 20 roundings, 7% together, for the colours and the head's gradient (whose
    terms do not cancel between layers)."""
    F = torch.randn(900, 160, device="cuda")
    nets = [pipeline.WideAppearance(F.clone(), 192, 2, d, seed=1) for d in (dtype, torch.float32)]
    dcol = torch.rand(3, 900, device="cuda")
    for net in nets:
        net.forward()
        net.backward(dcol)
    rel = lambda a, b: float((a - b).norm() / b.norm())
    assert rel(nets[0].colors, nets[1].colors) < 0.07 and rel(nets[0].head.dw, nets[1].head.dw) < 0.07


def test_training_with_the_renderer():
    """Colours of a small scene learned through render, L1 loss and both backward passes, geometry in the same
    clipped step; a step never lets the update's gradient norm above the limit."""
    gs, cam = scenes.tiny_scene(seed=1, n=1500)
    dg = rs.DeviceGaussians.from_numpy(gs)
    g = torch.Generator("cuda").manual_seed(0)
    net = pipeline.WideAppearance(torch.randn(gs.n, 128, device="cuda", generator=g), 256)
    R = pipeline.Renderer(cam, gs.n)
    target = R.forward(dg).image.clone()
    gc = rs.DeviceGaussians(dg.means.clone(), dg.scales, dg.quats, dg.opacity, None, -1, net.colors)
    means = rs.AdamGroup(gc.means, torch.empty_like(gc.means), torch.zeros_like(gc.means), torch.zeros_like(gc.means), 1e-5)
    dimg, loss = torch.empty_like(target), torch.zeros(1, device="cuda")
    losses = []
    for _ in range(40):
        net.forward()
        F = R.forward(gc)
        rs.rs_l1_loss_grad(F.image, target, 1.0 / target.numel(), dimg, loss)
        B = R.backward(gc, dimg)
        net.backward(B.dcolor)
        means.grad = B.dmeans
        net.step(max_norm=1e-3, lr=3e-3, groups=[means])
        losses.append(float(loss))
        total = sum(float(x.double().pow(2).sum()) for _, x in net.parameters()) + float(B.dmeans.double().pow(2).sum())
        assert abs(float(net.norm) / total ** 0.5 - 1) < 1e-5
    assert losses[-1] < 0.5 * losses[0], losses


def test_step_skips_what_is_not_finite():
    net = pipeline.WideAppearance(torch.randn(64, 64, device="cuda"), 64, 1)
    net.forward()
    net.backward(torch.full((3, 64), float("nan"), device="cuda"))
    before = [p.clone() for p, _ in net.parameters()]
    net.step(1.0)
    assert all(torch.equal(a, p) for a, (p, _) in zip(before, net.parameters())) and not np.isfinite(float(net.norm))


def test_on_a_stream_and_in_a_graph():
    net = pipeline.WideAppearance(torch.randn(500, 128, device="cuda"), 128, 1, seed=5)
    dcol = torch.randn(3, 500, device="cuda")
    net.forward()
    net.backward(dcol)
    want = [net.colors.clone()] + [x.clone() for _, x in net.parameters()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    net.forward(stream=s)
    net.backward(dcol, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [net.colors] + [x for _, x in net.parameters()]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.forward()
        net.backward(dcol)
    for t in [net.colors] + [x for _, x in net.parameters()]:
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, [net.colors] + [x for _, x in net.parameters()]))
