"""The wide appearance network of sandwich blocks and with 8-bit checkpoints as a user runs it: forward, backward, clipped
step, with the renderer around it.

Every stage is checked against float64 from the network's own inputs to that stage, float32 activations.  Tolerances, in the
2-norm: 1e-5 where a stage's inputs are at hand (float32 sums, each error below 1e-6 of its terms' magnitudes); 1e-3 where they had
to be recomputed or the result is an 8-bit form of a float32 one: a relative difference of 1e-6 crosses a tie (steps of 1/16) with a
probability of 3.2e-5 and then changes a value by 1/16, 3.5e-4 of the operand's norm."""
import numpy as np
import pytest
import torch

from gaussian_splatting_tile_gb300 import pipeline, rs, scenes

pytestmark = pytest.mark.gpu
OPTIONS = [dict(checkpoints=True)] + [dict(sandwich=True, gate=g, checkpoints=c) for g in (None, "row", "element")
                                      for c in (False, True)]
name_of = lambda o: "-".join(f"{k}={v}" for k, v in o.items())


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


def rms(x):
    return 1 / (x.double().pow(2).mean(1, keepdim=True) + 1e-6).sqrt()


def network(n, width, hidden, blocks=1, dtype=torch.float32, seed=3, **options):
    g = torch.Generator("cuda").manual_seed(n)
    net = pipeline.WideAppearance(torch.randn(n, width, device="cuda", generator=g), hidden, blocks, dtype, seed=seed, **options)
    for w in [*net.norms, *(net.posts + net.scales if net.sandwich else [])]:
        w.add_(0.2 * torch.randn(width, device="cuda", generator=g))
    return net, torch.randn(3, n, device="cuda", generator=g)


def norm_bwd(x, rho, w, dy, ds):
    xh, t = x * rho, dy * w.double()
    return rho * (t - xh * (t * xh).mean(1, keepdim=True)) + ds, (dy * xh).sum(0)


@pytest.mark.parametrize("options", OPTIONS, ids=name_of)
@pytest.mark.parametrize("n,width,hidden", [(777, 96, 200), (3000, 256, 512), (130, 130, 64), (50, 33, 40)])
def test_stages(n, width, hidden, options):
    net, dcol = network(n, width, hidden, **options)
    kept8, sandwich = net.checkpoints, net.sandwich
    net.forward()
    value = lambda pair: rs.fp8_dequantize(*pair).double()
    W1, W2, Wo = blocks8(net.up[0].w), blocks8(net.down[0].w), blocks8(net.head.w)
    Wg = blocks8(net.gates[0].w) if net.gates[0] else None
    F = net.features.double()
    h1 = net.h[1].double()
    # an activation as the products read it, and as it is kept
    y = [value(t) for t in net.yq] if kept8 else [rows8(t) for t in net.y]
    u = value(net.uq[0]) if kept8 else rows8(net.u[0])
    tol8 = 1e-3 if kept8 else 1e-5
    y0, y1 = (x * rms(x) * w.double() for x, w in ((F, net.norms[0]), (h1, net.norms[1])))
    near(y[0] if kept8 else net.y[0], rows8(y0) if kept8 else y0, tol8)
    near(y[1] if kept8 else net.y[1], rows8(y1) if kept8 else y1, tol8)
    hidden_out = torch.relu(y[0] @ W1.t())
    near(u if kept8 else net.u[0], rows8(hidden_out) if kept8 else hidden_out, tol8)
    r = net.results[0] if sandwich else net.r
    near(r, u @ W2.t())
    g = 1.0
    if sandwich:
        if Wg is not None:
            near(net.zs[0], y[0] @ Wg.t())
            g = torch.sigmoid(net.zs[0].double())
        al, post = net.scales[0].double(), net.posts[0].double()
        near(h1, al * F + g * (r.double() * rms(r) * post))
        near(net.rstd_r[0], rms(r)[:, 0])
        near(net.rstd[1], rms(h1)[:, 0])
    else:
        near(h1, F + r.double())
    near(net.z, y[1] @ Wo.t())
    near(net.colors, torch.sigmoid(net.z.double()).t())

    net.backward(dcol)
    dz = (dcol * net.colors * (1 - net.colors)).t().contiguous()
    wide_y = y if kept8 else net.y
    wide_u = u if kept8 else net.u[0]
    near(net.head.dw, cols8(dz).t() @ cols8(wide_y[1]))
    dy1 = rows8(dz) @ Wo
    if sandwich:
        X, R = (value(net.kept[0][k]) for k in ("x", "r")) if kept8 else (F, r.double())
        Z = None
        if Wg is not None:
            Z = value(net.kept[0]["gate"]) if "gate" in (net.kept[0] if kept8 else {}) else net.zs[0].double()
            g = torch.sigmoid(Z)
        rh = R * net.rstd_r[0].double()[:, None]
        s = al * X + g * rh * post
        ds, dpre = norm_bwd(s, net.rstd[1].double()[:, None], net.norms[1], dy1, 0)
        dr, dpost = norm_bwd(R, net.rstd_r[0].double()[:, None], net.posts[0], ds * g, 0)
        near(net.dnorms[1], dpre)
        near(net.dposts[0], dpost)
        near(net.dscales[0], (ds * X).sum(0))
        dh = al * ds
        if Z is not None:
            dgate = ds * rh * post * g * torch.sigmoid(-Z)
            near(net.dgate, dgate if dgate.shape == net.dgate.shape and Z.shape[1] > 1 else
                 (ds * rh * post).sum(1, keepdim=True) * g * torch.sigmoid(-Z))
    else:
        dh, dpre = norm_bwd(h1, net.rstd[1].double()[:, None], net.norms[1], dy1, 0)
        dr = dh
        near(net.dnorms[1], dpre)
    near(net.down[0].dw, cols8(dr).t() @ cols8(wide_u), 1e-3)
    near(net.du, rows8(dr) @ W2, 1e-3)
    du = net.du * (wide_u > 0)
    near(net.up[0].dw, cols8(du).t() @ cols8(wide_y[0]))
    dy0 = rows8(du) @ W1
    if Wg is not None:
        near(net.gates[0].dw, cols8(net.dgate).t() @ cols8(wide_y[0]))
        dy0 = dy0 + rows8(net.dgate) @ Wg
    near(net.dy, dy0)
    df, dw = norm_bwd(F, net.rstd[0].double()[:, None], net.norms[0], net.dy.double(), dh)
    near(net.dfeatures, df)
    near(net.dnorms[0], dw)


@pytest.mark.parametrize("options", [dict()] + OPTIONS[1::2], ids=name_of)
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_checkpoints_change_no_colour(options, dtype):
    """In float32 the products read the same 8-bit forms either way; in 16 bits the hidden activations are no longer rounded to
    16 bits before they are to 8: each such rounding (2^-8 at most) moves at most 1 in 16 values across a tie, by 1/16 of itself,
    1/64 of an operand's norm for each of two blocks."""
    nets = [network(900, 160, 192, 2, dtype, checkpoints=c, **{k: v for k, v in options.items() if k != "checkpoints"})[0]
            for c in (False, True)]
    for net in nets:
        net.forward()
    a, b = (net.colors for net in nets)
    if dtype is torch.float32:
        assert torch.equal(a, b)
    else:
        assert float((a - b).norm() / a.norm()) < 0.07
    assert nets[1].kept_bytes() < nets[0].kept_bytes()


@pytest.mark.parametrize("options", OPTIONS, ids=name_of)
def test_two_blocks_keep_their_own(options):
    """The second block's operands are its own: with W2 = 0 in the second block of a sandwich network, and its scale one, the
    first block's gradients are those of a network of one block.

    Of plain blocks bit for bit.  A sandwich block's backward forms mean(ds p) from the parts of ds that it is handed, here all of it
    as dL_dsum, there all of it by dL_dy: sums of the same value in another order, a relative difference of 1e-6 in dr.  Such a
    difference d moves a value of an 8-bit form across a tie with a probability of 32 d and then by 1/16: sqrt(32 d) / 16 of the
    form's norm, 3.5e-4 in dW2, and with that for d once more 6.6e-3 in dW1 and what lies behind it.  The bounds are three times
    that.  (With checkpoints the sums are read back from 8-bit forms of different operands: only the head is compared.)"""
    one, dcol = network(500, 160, 192, 1, **options)
    two, _ = network(500, 160, 192, 2, **options)
    pairs = [(one.up[0], two.up[0]), (one.down[0], two.down[0]), (one.head, two.head)]
    pairs += [(one.gates[0], two.gates[0])] if one.gates[0] else []
    for a, b in pairs:
        b.w.copy_(a.w)
    two.down[1].w.zero_()
    for layer in two._layers():
        layer.refresh()
    two.norms[0].copy_(one.norms[0])
    two.norms[2].copy_(one.norms[1])
    if one.sandwich:
        two.posts[0].copy_(one.posts[0])
        two.scales[0].copy_(one.scales[0])
        two.scales[1].fill_(1)
    for net in (one, two):
        net.forward()
        net.backward(dcol)
    assert torch.equal(one.colors, two.colors)
    assert torch.equal(one.head.dw, two.head.dw)
    if not (one.sandwich and one.checkpoints):
        for a, b, tol in ((one.down[0].dw, two.down[0].dw, 1e-3), (one.up[0].dw, two.up[0].dw, 2e-2),
                          (one.dfeatures, two.dfeatures, 2e-2)):
            if one.sandwich:
                near(a, b.double(), tol)
            else:
                assert torch.equal(a, b)
    assert float(two.down[1].dw.abs().max()) > 0


@pytest.mark.parametrize("options", [OPTIONS[0], OPTIONS[4], OPTIONS[6]], ids=name_of)
def test_training_with_the_renderer(options):
    """Steps on a small scene, geometry in the same clipped step: every parameter moves, all stays finite, and the norm is that of
    all gradients."""
    gs, cam = scenes.tiny_scene(seed=1, n=1500)
    dg = rs.DeviceGaussians.from_numpy(gs)
    g = torch.Generator("cuda").manual_seed(0)
    net = pipeline.WideAppearance(torch.randn(gs.n, 128, device="cuda", generator=g), 256, **options)
    R = pipeline.Renderer(cam, gs.n)
    target = R.forward(dg).image.clone()
    gc = rs.DeviceGaussians(dg.means.clone(), dg.scales, dg.quats, dg.opacity, None, -1, net.colors)
    means = rs.AdamGroup(gc.means, torch.empty_like(gc.means), torch.zeros_like(gc.means), torch.zeros_like(gc.means), 1e-5)
    dimg, loss = torch.empty_like(target), torch.zeros(1, device="cuda")
    before = [p.clone() for p, _ in net.parameters()]
    for _ in range(5):
        net.forward()
        F = R.forward(gc)
        rs.rs_l1_loss_grad(F.image, target, 1.0 / target.numel(), dimg, loss)
        B = R.backward(gc, dimg)
        net.backward(B.dcolor)
        means.grad = B.dmeans
        net.step(max_norm=1e-3, lr=3e-3, groups=[means])
        total = sum(float(x.double().pow(2).sum()) for _, x in net.parameters()) + float(B.dmeans.double().pow(2).sum())
        assert abs(float(net.norm) / total ** 0.5 - 1) < 1e-5 and np.isfinite(float(loss))
    for a, (p, _) in zip(before, net.parameters()):
        assert bool(torch.isfinite(p).all()) and not torch.equal(a, p)


@pytest.mark.parametrize("options", [OPTIONS[0], OPTIONS[3], OPTIONS[6]], ids=name_of)
def test_float16_keeps_small_gradients(options):
    """A loss 2^-24 times as large has gradients exactly 2^-24 times as large, down to what float16 itself cannot hold."""
    net, dcol = network(300, 128, 192, 2, torch.float16, **options)
    got = []
    for f in (1.0, 2.0 ** -24):
        net.forward()
        net.backward(dcol * f)
        got.append([g.clone() for _, g in net.parameters()])
    for a, b in zip(*got):
        assert torch.equal(a, b * 2.0 ** 24) and float(a.abs().max()) > 0


@pytest.mark.parametrize("options", OPTIONS, ids=name_of)
def test_on_a_stream_and_in_a_graph(options):
    net, dcol = network(500, 128, 128, 2, torch.bfloat16, **options)
    results = lambda: [net.colors] + [x for _, x in net.parameters()]
    net.forward()
    net.backward(dcol)
    want = [t.clone() for t in results()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    net.forward(stream=s)
    net.backward(dcol, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    net.step(1.0, lr=0.0)                       # makes the moments; nothing moves
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.forward()
        net.backward(dcol)
        net.step(1.0, lr=0.0)
    for t in results():
        if t is not (net.dvectors if net.sandwich else None):
            t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    assert int(net.steps) == 2


def test_no_blocks_one_gaussian_and_one_feature():
    for options in OPTIONS:
        for n, blocks, width in ((40, 0, 64), (1, 1, 64), (1, 2, 64), (70, 2, 1), (70, 1, 130)):
            net, dcol = network(n, width, 64, blocks, torch.float32, **options)
            net.forward()
            net.backward(dcol)
            assert all(bool(torch.isfinite(g).all()) for _, g in net.parameters())
