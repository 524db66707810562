"""GPU parity of the sandwich norm (norms before and after a block, gate, residual scale) and its backward with float64
formulas, through the C ABI.

Tolerances, with u = 2^-24 (float32's half ulp) and h = the half ulp of the stored type (2^-24, 2^-11, 2^-8):
 - a float32 sum in which no chain of additions is longer than L is within L u of its terms' magnitudes; a row's chains are at
   most 32 values a thread, 5 shuffles and 16 warps: 64 u covers them, 40 u the reciprocal root of such a sum of squares;
 - a gate's e = 2^(-z log2 e): the constant and the product move the exponent by at most 1.5 |z| log2(e) u, so e by 1.5 |z| u,
   and the power of two (PTX: within 2^-22.5) by 3 u; the reciprocal of 1 + e is off by an ulp, 2 u, and the sum's rounding:
   less than (9 + 2.4 |z|) u of g, and of g e = 1 - g, where e counts twice, than (13 + 5 |z|) u;
 - what follows is each formula's operations, one u each, with the errors of what they take.
Functions below carry a value and the bound on its error side by side."""
import math

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_gb300 import rs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}      # half of a subnormal step, or what is flushed
SIZES = [(1, 1), (3, 7), (130, 64), (5, 127), (9, 128), (33, 129), (1, 256), (70, 257), (17, 512), (5, 777), (300, 1000),
         (2, 1025), (9, 2048), (3, 2050), (4, 4096), (3, 4104), (2, 8192), (3, 8193), (2, 16384), (41, 384), (37, 600),
         (37, 601), (700, 768), (9, 1203), (400, 1536), (4, 2601), (300, 3000)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from gaussian_splatting_tile_gb300 import build_lib
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def rand(g, *s):
    return torch.randn(*s, device="cuda", generator=g)


def close(got, want, tol):
    """|got - want| <= tol everywhere (tol a tensor or a number), NaN nowhere."""
    assert got.shape == want.shape
    d = (got.double() - want.double()).abs()
    assert bool((d <= tol).all()), float((d - tol).max())


class Block:
    """A block's operands and how they are handed over."""

    def __init__(self, g, rows, cols, dt, gate="element", scale=True):
        self.rows, self.cols, self.dt = rows, cols, dt
        t = DT[dt]
        self.x, self.r = (3 * rand(g, rows, cols)).to(t), (0.7 * rand(g, rows, cols)).to(t)
        self.gate = None if gate == "none" else (2 * rand(g, rows, 1 if gate == "row" else cols)).to(t)
        self.alpha = 1 + 0.3 * rand(g, cols) if scale else None
        self.wpost, self.wpre = 1 + 0.3 * rand(g, cols), 1 + 0.3 * rand(g, cols)
        self.elements = gate == "element" and cols > 1

    def forward(self, kept=False, eps=1e-6, **extra):
        r, c = self.rows, self.cols
        o = {"sum": torch.empty_like(self.x), "y": torch.empty_like(self.x), "rstd_r": torch.empty(r, device="cuda"),
             "rstd_s": torch.empty(r, device="cuda")}
        q, sc = rs.fp8_empty(r, c)
        keep = {}
        if kept:
            keep = {k: rs.fp8_empty(r, c) for k in ["kept_x", "kept_r"] + ["kept_gate"] * self.elements}
        rs.rs_sandwich_norm_fwd(self.x, self.r, self.wpost, self.wpre, q, sc, gate=self.gate, residual_scale=self.alpha,
                                eps=eps, **(o | keep | extra))
        return o | keep | {"q": q, "scales": sc}

    def operands(self):
        """(x, r, z, alpha) in 64 bits."""
        f = lambda t: rs.fp8_dequantize(*t).double() if isinstance(t, tuple) else t.double()
        one = torch.ones((), dtype=torch.float64, device="cuda")
        return f(self.x), f(self.r), None if self.gate is None else f(self.gate), one if self.alpha is None else self.alpha.double()


def gate_of(z):
    """(g, bound on its relative error, bound on that of 1 - g)."""
    if z is None:
        return 1.0, 0.0, 0.0
    return torch.sigmoid(z), (9 + 2.4 * z.abs()) * U, (13 + 5 * z.abs()) * U


def check_forward(b, kept=False, eps=1e-6):
    o = b.forward(kept, eps)
    x, r, z, al = b.operands()
    h, tiny = HALF_ULP[b.dt], TINY[b.dt]
    rho_r = 1 / (r.pow(2).mean(1, keepdim=True) + eps).sqrt()
    close(o["rstd_r"], rho_r[:, 0], 40 * U * rho_r[:, 0])
    g, eg, _ = gate_of(z)
    n = g * (r * rho_r * b.wpost.double())
    s = al * x + n
    es = U * (al * x).abs() + n.abs() * (46 * U + eg) + U * s.abs()
    close(o["sum"], s, es + h * s.abs() + tiny)
    rho_s = 1 / (s.pow(2).mean(1, keepdim=True) + eps).sqrt()
    erho = 40 * U + es.pow(2).mean(1, keepdim=True).sqrt() * rho_s           # relative
    close(o["rstd_s"], rho_s[:, 0], (erho * rho_s)[:, 0])
    w = b.wpre.double()
    y = s * rho_s * w
    ey = y.abs() * (erho + 4 * U) + es * rho_s * w.abs()
    close(o["y"], y, ey + h * y.abs() + tiny)
    for k in range(-(-b.cols // 128)):
        cut = slice(k * 128, (k + 1) * 128)
        top = y[:, cut].abs().amax(1).clamp_min(2.0 ** -100)
        etop = ey[:, cut].amax(1)
        close(o["scales"][k], top / 448, (etop + 2 * U * top) / 448)
        q = y[:, cut] / (top / 448)[:, None]
        got = o["q"][:, cut].float().double()
        slack = ((ey[:, cut] + q.abs() / 448 * etop[:, None]) / top[:, None] + 4 * U) * 448
        close(got, q, q.abs() / 16 + 2.0 ** -10 + 1.1 * slack)
        assert bool((got.abs().amax(1)[top > 2.0 ** -100] == 448).all())
    if kept:  # bit for bit the forms that rs_quantize_fp8 gives
        for name, t in (("kept_x", b.x), ("kept_r", b.r), ("kept_gate", b.gate)):
            if name in o:
                q, sc = rs.fp8_empty(b.rows, b.cols)
                rs.rs_quantize_fp8(t, q, sc)
                assert torch.equal(q.view(torch.uint8), o[name][0].view(torch.uint8)) and torch.equal(sc, o[name][1])
    return o


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(dt, gate, rows, cols):
    g = gen(rows * 100003 + cols)
    check_forward(Block(g, rows, cols, dt, gate, scale=(rows + cols) % 2 == 0), kept=True)
    check_forward(Block(g, rows, cols, dt, gate, scale=(rows + cols) % 2 == 1), kept=False)


def backward(b, o, dy, dsum, want=("alpha", "post", "pre", "gate"), out=None):
    """(dx, dr, dgate, dalpha, dpost, dpre)"""
    f = lambda: torch.empty(b.cols, device="cuda")
    dx, dr = out or (torch.empty_like(dy), torch.empty_like(dy))
    gate = b.gate[0] if isinstance(b.gate, tuple) else b.gate
    dgate = torch.empty(gate.shape, dtype=dy.dtype, device="cuda") if gate is not None and "gate" in want else None
    da, dpost, dpre = (f() if k in want else None for k in ("alpha", "post", "pre"))
    ws = torch.empty(rs.rs_sandwich_norm_bwd_workspace_size(b.rows, b.cols), dtype=torch.uint8, device="cuda")
    rs.rs_sandwich_norm_bwd(b.x, b.r, b.wpost, b.wpre, o["rstd_r"], o["rstd_s"], dy, dx, dr, ws, gate=b.gate, dL_dgate=dgate,
                            residual_scale=b.alpha, dL_dsum=dsum, dL_dpost_weight=dpost, dL_dpre_weight=dpre,
                            dL_dresidual_scale=da)
    return dx, dr, dgate, da, dpost, dpre


def check_backward(b, o, dy, dsum):
    got = backward(b, o, dy, dsum)
    x, r, z, al = b.operands()
    h, tiny, c, rows = HALF_ULP[b.dt], TINY[b.dt], b.cols, b.rows
    rho_r, rho_s = o["rstd_r"].double()[:, None], o["rstd_s"].double()[:, None]
    wpost, wpre, dy = b.wpost.double(), b.wpre.double(), dy.double()
    d = torch.zeros_like(dy) if dsum is None else dsum.double()
    mean = lambda t: t.mean(1, keepdim=True)
    g, eg, eg1 = gate_of(z)
    rh = r * rho_r                                    # a kept value is a rounded product: 2 u
    n = rh * wpost
    p, ep = g * n, (g * n).abs() * (5 * U + eg)
    sh = (al * x + p) * rho_s
    es = rho_s * (3 * U * (al * x).abs() + ep) + 2 * U * sh.abs()
    t = dy * wpre
    a1, ea = mean(t * sh), mean(t.abs() * es) + 68 * U * mean((t * sh).abs())
    base = (rho_s * t).abs() + d.abs()
    ds = rho_s * (t - sh * a1) + d
    eds = 3 * U * base + rho_s * (sh.abs() * ea + a1.abs() * es + 4 * U * (sh * a1).abs()) + U * ds.abs()
    close(got[0], al * ds, al.abs() * eds + (2 * U + h) * (al * ds).abs() + tiny)
    b1 = mean(ds * p)
    eb = (mean(base * ep) + 71 * U * mean(base * p.abs()) + rho_s * ea * mean((sh * p).abs()) +
          rho_s * a1.abs() * (mean(es * p.abs() + sh.abs() * ep) + 72 * U * mean((sh * p).abs())))
    dn = ds * g
    dr = rho_r * (dn * wpost - rh * b1)
    edn = eds * g + dn.abs() * (eg + U)
    close(got[1], dr, rho_r * (edn * wpost.abs() + U * (dn * wpost).abs() + rh.abs() * eb + 4 * U * (b1 * rh).abs()) +
          (2 * U + h) * dr.abs() + tiny)
    if z is not None:
        g1 = torch.sigmoid(-z)
        if got[2].shape[1] == 1 and c > 1 or not b.elements:
            dz = mean(ds * p) * c * g1
            ez = c * eb * g1 + dz.abs() * (eg1 + 4 * U)
        else:
            dz = ds * p * g1
            ez = eds * (p * g1).abs() + g1 * ds.abs() * ep + dz.abs() * (eg1 + 4 * U)
        close(got[2], dz, ez + h * dz.abs() + tiny)
    # a thread adds its rows one after another, then at most 8 + 32 + 5 partial sums
    total = lambda v, e: (v.sum(0), e.sum(0) + (rows + 66) * U * v.abs().sum(0) + 1e-37)
    for have, v, e in ((got[3], ds * x, eds * x.abs()), (got[4], dn * rh, edn * rh.abs()), (got[5], dy * sh, dy.abs() * es)):
        close(have, *total(v, e + 3 * U * v.abs()))
    return got


def grads_of(g, b):
    return rand(g, b.rows, b.cols).to(DT[b.dt]), rand(g, b.rows, b.cols).to(DT[b.dt])


def keep(b, o):
    b.x, b.r = o["kept_x"], o["kept_r"]
    if "kept_gate" in o:
        b.gate = o["kept_gate"]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", ["none", "row", "element"])
@pytest.mark.parametrize("rows,cols", SIZES + [(4001, 129), (1700, 512), (3000, 1000), (700, 2048), (400, 4096), (200, 16384), (400, 8200), (50, 12288)])
def test_backward(dt, gate, rows, cols):
    g = gen(rows * 7 + cols)
    for kept in (False, True):
        b = Block(g, rows, cols, dt, gate, scale=(rows + cols + kept) % 2 == 0)
        dy, dsum = grads_of(g, b)
        o = b.forward(kept)
        if kept:
            keep(b, o)
        got = check_backward(b, o, dy, dsum if (rows + kept) % 3 else None)
        again = backward(b, o, dy, dsum if (rows + kept) % 3 else None)
        assert all(v is None or torch.equal(v, w) for v, w in zip(got, again))     # sums in a fixed order


def test_backward_against_differences():
    """L = sum(G y) + sum(D s): central differences of the forward's own float32 outputs along random directions, step 1/64.
    The truncation is (1/64)^2 / 6 of the third derivative along the direction (of order |G|, |D| and the weights, with a factor
    of 6 for the products of up to three of its parts), the rounding of y and s 2^-22 of them 64 / 2 times over, both
    summed over 600 values with random signs: 5e-3 sqrt(600) bounds them."""
    g = gen(77)
    rows, cols, h = 3, 200, 1 / 64
    for gate in ("none", "row", "element"):
        b = Block(g, rows, cols, "f32", gate)
        G, D = rand(g, rows, cols), rand(g, rows, cols)
        o = b.forward()
        got = backward(b, o, G, D)

        def loss():
            o = b.forward()
            return float((G.double() * o["y"].double()).sum() + (D.double() * o["sum"].double()).sum())

        for name, d in (("x", got[0]), ("r", got[1]), ("gate", got[2]), ("alpha", got[3]), ("wpost", got[4]), ("wpre", got[5])):
            if d is None:
                continue
            for _ in range(2):
                at, v = getattr(b, name), rand(g, *d.shape)
                setattr(b, name, at + h * v)
                up = loss()
                setattr(b, name, at - h * v)
                fd = (up - loss()) / (2 * h)
                setattr(b, name, at)
                assert abs(fd - float((d.double() * v.double()).sum())) < 5e-3 * math.sqrt(rows * cols), (gate, name)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_offsets_and_in_place(dt):
    g = gen(5)
    rows, cols = 37, 300
    for pad, off in ((8, 8), (3, 1), (5, 0)):
        b = Block(g, rows, cols, dt)
        wide = lambda t: torch.nn.functional.pad(t, (off, pad), value=9.0)[:, off:off + cols]
        b.x, b.r, b.gate = wide(b.x), wide(b.r), wide(b.gate)
        b.wpost = torch.nn.functional.pad(b.wpost, (1, 0))[1:]
        o = check_forward(b, kept=True)
        dy, dsum = (wide(t) for t in grads_of(g, b))
        want = check_backward(b, o, dy, dsum)
        # gradients over their own upstream, both ways round
        for swap in (False, True):
            a, d = wide(dy), wide(dsum)
            got = backward(b, o, a, d, out=(d, a) if swap else (a, d))
            for v, w in zip(got, want):
                assert torch.equal(v, w)
            for t in (a, d):
                whole = t.as_strided((rows - 1, cols + pad + off), (cols + pad + off, 1), t.storage_offset() - off)
                assert bool((whole[:, :off] == 9).all() and (whole[:, off + cols:] == 9).all())
        # the sum over x, and over r
        for name in ("x", "r"):
            t = wide(getattr(b, name))
            c = Block(g, rows, cols, dt)
            c.__dict__.update(b.__dict__)
            setattr(c, name, t)
            got = c.forward(kept=True, sum=t)
            assert torch.equal(t, o["sum"])
            assert all(torch.equal(got[k], o[k]) for k in ("rstd_r", "rstd_s", "y", "scales"))
            assert torch.equal(got["kept_x"][0].view(torch.uint8), o["kept_x"][0].view(torch.uint8))


def test_no_bytes_past_the_columns():
    g = gen(6)
    for cols in (2, 7, 130, 777):
        b = Block(g, 5, cols, "f32")
        raw = [torch.full((5, -(-cols // 16) * 16 + 16), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(4)]
        sc = [rs.fp8_empty(5, cols)[1] for _ in range(4)]
        rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, raw[0][:, :cols], sc[0], gate=b.gate, kept_x=(raw[1][:, :cols], sc[1]),
                                kept_r=(raw[2][:, :cols], sc[2]), kept_gate=(raw[3][:, :cols], sc[3]))
        assert all(bool((t[:, cols:] == 0xAB).all()) for t in raw)


def test_each_output_alone():
    g = gen(16)
    b = Block(g, 9, 300, "bf16")
    o = b.forward(kept=True)
    q, sc = rs.fp8_empty(9, 300)
    rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, q, sc, gate=b.gate, residual_scale=b.alpha)
    assert torch.equal(q.view(torch.uint8), o["q"].view(torch.uint8)) and torch.equal(sc, o["scales"])
    y = torch.empty_like(b.x)
    rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, gate=b.gate, residual_scale=b.alpha, y=y)
    assert torch.equal(y, o["y"])
    for name, t in (("kept_x", b.x), ("kept_r", b.r), ("kept_gate", b.gate)):
        form = rs.fp8_empty(9, 300)
        rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, gate=b.gate, y=y, **{name: form})
        assert torch.equal(form[0].view(torch.uint8), o[name][0].view(torch.uint8)) and torch.equal(form[1], o[name][1])
    dy, dsum = grads_of(g, b)
    want = backward(b, o, dy, dsum)
    for i, k in enumerate(("gate", "alpha", "post", "pre")):
        got = backward(b, o, dy, dsum, want=(k,))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2 + i], want[2 + i])
    got = backward(b, o, dy, dsum, want=())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows():
    w = torch.ones(300, device="cuda")
    e = torch.empty(0, 300, device="cuda")
    rs.rs_sandwich_norm_fwd(e, e, w, w, *rs.fp8_empty(0, 300), gate=e)
    d = [torch.full((300,), 7.0, device="cuda") for _ in range(2)]
    n = torch.empty(0, device="cuda")
    rs.rs_sandwich_norm_bwd(e, e, w, w, n, n, e, e, e, None, dL_dpost_weight=d[0], dL_dresidual_scale=d[1])
    assert all(bool((t == 0).all()) for t in d)


def test_rows_of_zeros_gates_at_the_ends_and_values_that_are_not_finite():
    rows, cols = 8, 300
    g = gen(3)
    for dt in ("f32", "bf16"):
        b = Block(g, rows, cols, dt)
        b.x[0], b.r[0] = 0, 0                                  # nothing
        b.r[1] = 0                                             # a block that gives nothing
        b.gate[2], b.gate[3] = -math.inf, math.inf             # shut, open
        b.gate[4] = torch.finfo(DT[dt]).min                    # shut by the type's lowest value
        b.r[5, 7], b.x[6, 9], b.gate[7, 5] = math.nan, math.inf, math.nan
        o = b.forward(kept=True)
        fine = b.rows - 3
        assert bool((o["sum"][0] == 0).all()) and bool((o["q"][0].float() == 0).all())
        assert abs(float(o["rstd_r"][1]) - 1000.0) < 1e-2
        al = b.alpha.double()
        for i in (1, 2, 4):                                    # sum = alpha x, gates of exp(-80) far below its rounding
            want = al * b.x[i].double()
            close(o["sum"][i], want, (2 * U + HALF_ULP[dt]) * want.abs() + 1e-30)
        n = b.r[3].double() * float(o["rstd_r"][3]) * b.wpost.double()
        close(o["sum"][3], al * b.x[3].double() + n, (50 * U + HALF_ULP[dt]) * ((al * b.x[3].double()).abs() + n.abs()))
        assert bool(torch.isfinite(o["sum"][:fine].float()).all()) and bool(torch.isfinite(o["y"][:fine].float()).all())
        assert bool(torch.isnan(o["sum"][5].float()).all()) and math.isinf(float(o["sum"][6, 9]))
        assert math.isnan(float(o["sum"][7, 5])) and bool(torch.isnan(o["y"][7].float()).all())
        dy, dsum = grads_of(g, b)
        dx, dr, dz = backward(b, o, dy, dsum, want=("gate",))[:3]
        for t in (dx, dr, dz):
            assert bool(torch.isfinite(t[:fine].float()).all())
        assert bool((dz[2:5].float().abs() < 1e-30).all()) and bool((dr[[2, 4]].float().abs() < 1e-28).all())
        assert bool(torch.isnan(dx[5].float()).all() and torch.isnan(dx[7].float()).all())


def test_rows_far_apart():
    """Row offsets past 2^32 bytes, as inputs and as outputs."""
    stride, cols = (1 << 31) + 64, 200
    g = gen(9)
    b = Block(g, 3, cols, "bf16")
    o = b.forward(kept=True)
    dy, dsum = grads_of(g, b)
    want = backward(b, o, dy, dsum)
    flat = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    place = iter(range(0, 4096, 256))

    def far(t):
        v = flat[next(place):].as_strided((3, cols), (stride, 1))
        v.copy_(t)
        return v

    b.x, b.r, b.gate = far(b.x), far(b.r), far(b.gate)
    s, y = far(torch.zeros_like(dy)), far(torch.zeros_like(dy))
    o2 = b.forward(kept=True, sum=s, y=y)
    assert torch.equal(s, o["sum"]) and torch.equal(y, o["y"]) and torch.equal(o2["scales"], o["scales"])
    got = backward(b, o, far(dy), far(dsum), out=(far(torch.zeros_like(dy)), far(torch.zeros_like(dy))))
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    del flat, b, got, s, y
    bytes_ = torch.empty(2 * (1 << 32) + 4096, dtype=torch.uint8, device="cuda")
    b = Block(gen(9), 3, cols, "bf16")
    keep(b, o)
    want = backward(b, o, dy, dsum)
    place = iter(range(0, 4096, 256))

    def far8(pair):
        v = bytes_[next(place):].as_strided((3, cols), (1 << 32, 1))
        v.copy_(pair[0].view(torch.uint8))
        return v, pair[1]

    b.x, b.r, b.gate = far8(b.x), far8(b.r), far8(b.gate)
    assert all(torch.equal(a, c) for a, c in zip(backward(b, o, dy, dsum), want))


def test_streams_and_graphs():
    """Two captured calls that share a workspace, replayed on a stream of their own; inputs changed between replays."""
    g = gen(21)
    b = Block(g, 333, 512, "bf16")
    o = b.forward(kept=True)
    c = Block(g, 333, 512, "bf16")
    c.__dict__.update(b.__dict__)
    keep(c, o)
    dy, dsum = grads_of(g, b)
    q, sc = rs.fp8_empty(333, 512)
    ws = torch.empty(rs.rs_sandwich_norm_bwd_workspace_size(333, 512), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(dy) for _ in range(3)] + [torch.empty(512, device="cuda") for _ in range(3)] for _ in range(2)]

    def step():
        rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, q, sc, gate=b.gate, residual_scale=b.alpha)
        for which, t in zip((b, c), outs):
            rs.rs_sandwich_norm_bwd(which.x, which.r, b.wpost, b.wpre, o["rstd_r"], o["rstd_s"], dy, t[0], t[1], ws, gate=which.gate,
                                    dL_dgate=t[2], residual_scale=b.alpha, dL_dsum=dsum, dL_dpost_weight=t[3],
                                    dL_dpre_weight=t[4], dL_dresidual_scale=t[5])

    step()
    want = [t.clone() for t in (*outs[0], *outs[1], sc)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for value in (7.0, -3.0):
        for t in (*outs[0], *outs[1], sc):
            t.fill_(value)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip((*outs[0], *outs[1], sc), want))
    dy.mul_(2)
    dsum.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1][3], 2 * want[9]) and torch.equal(outs[0][0], (2 * want[0].float()).to(torch.bfloat16))


def test_parameters_and_missing_operands():
    """Tensors of a subclass are tensors; an operand that is missing is refused by the library, not by accident."""
    g = gen(41)
    b = Block(g, 5, 64, "f32")
    o = b.forward()
    want = rs.fp8_empty(5, 64)
    rs.rs_sandwich_norm_fwd(b.x, b.r, b.wpost, b.wpre, *want, gate=b.gate, residual_scale=b.alpha)
    P = lambda t: torch.nn.Parameter(t, requires_grad=False)
    got = rs.fp8_empty(5, 64)
    rs.rs_sandwich_norm_fwd(P(b.x), P(b.r), P(b.wpost), P(b.wpre), *got, gate=P(b.gate), residual_scale=P(b.alpha))
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    for x, r, w in ((b.x, None, b.wpost), (b.x, b.r, None)):
        with pytest.raises(rs.RsError):
            rs.rs_sandwich_norm_fwd(x, r, w, b.wpre, *got)
    dy = torch.ones_like(b.x)
    with pytest.raises(rs.RsError):
        rs.rs_sandwich_norm_bwd(b.x, b.r, b.wpost, b.wpre, o["rstd_r"], None, dy, dy.clone(), dy.clone(), None)
    with pytest.raises(TypeError):    # float32 is no 8-bit matrix
        rs.rs_sandwich_norm_bwd((b.x, None), b.r, b.wpost, b.wpre, o["rstd_r"], o["rstd_s"], dy, dy.clone(), dy.clone(), None)
    with pytest.raises(ValueError):   # nor is one complete without its scales
        rs.rs_sandwich_norm_bwd((got[0], None), b.r, b.wpost, b.wpre, o["rstd_r"], o["rstd_s"], dy, dy.clone(), dy.clone(), None)
