"""GPU parity of the wide appearance network's operators (norm with an 8-bit output, 8-bit matrix product, gradient
clipping) with float64 formulas, through the C ABI.

Tolerances, with u = 2^-24 (float32's half ulp) and h = the half ulp of the stored type (2^-24, 2^-11, 2^-8: 24, 11 and 8 significant bits):
 - a float32 sum of positive terms in which no chain of additions is longer than L is within L u of its value;
   the norm's chains are at most 32 values a thread, 5 shuffles and 16 warps: 64 u, and the square root halves it;
 - e4m3 keeps 4 significant bits: a scaled value moves by at most 1/16 of itself, or 2^-10 below 2^-6;
 - a matrix product adds products of 8 significant bits, which are exact in float32: with a block's 128 products and ceil(k / 128)
   blocks added one after another, each addition losing at most 2u (a truncating adder), the sum of magnitudes bounds
   the error by (128 + k / 128 + 4) 2u."""
import math

import numpy as np
import pytest
import torch

from gaussian_splatting_tile_gb300 import rs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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
    d = (got.double() - want.double()).abs()
    assert bool((d <= tol).all()), float((d - tol).max())


# ------------------------------------------------------------------ norm

def norm_fwd(x, w, residual=None, eps=1e-6, want_sum=True, y=False):
    r, c = x.shape
    q, sc = rs.fp8_empty(r, c)
    s = torch.empty_like(x) if want_sum else None
    yy = torch.empty_like(x) if y else None
    rstd = torch.empty(r, device="cuda")
    rs.rs_rms_norm_fwd(x, w, q, sc, residual=residual, sum=s, y=yy, rstd=rstd, eps=eps)
    return q, sc, s, yy, rstd


def check_norm(x, w, residual, dt, eps=1e-6):
    r, c = x.shape
    q, sc, s, y, rstd = norm_fwd(x, w, residual, eps, True, True)
    xs = x.double() + (residual.double() if residual is not None else 0)
    rho = 1 / (xs.pow(2).mean(1) + eps).sqrt()
    close(rstd, rho, 40 * U * rho)
    close(s, xs, (U + HALF_ULP[dt]) * xs.abs() + 2.0 ** -24)       # f16: subnormal steps
    yy = xs * rho[:, None] * w.double()
    close(y, yy, (48 * U + HALF_ULP[dt]) * yy.abs() + 2.0 ** -24)
    assert sc.shape == (-(-c // 128), r)
    for b in range(sc.shape[0]):
        blk = yy[:, b * 128:(b + 1) * 128]
        top = blk.abs().amax(1).clamp_min(2.0 ** -100)
        close(sc[b], top / 448, 64 * U * top / 448)
        z = blk / (top / 448)[:, None]
        got = q[:, b * 128:(b + 1) * 128].float().double()
        close(got, z, z.abs() / 16 + 2.0 ** -10 + 448 * 64 * U)
        assert bool((got.abs().amax(1)[top > 2.0 ** -100] == 448).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (130, 64), (5, 127), (9, 128), (33, 129), (1, 256), (70, 257),
                                       (17, 512), (5, 777), (300, 1000), (2, 1025), (9, 2048), (3, 2050), (4, 4096),
                                       (3, 4104), (2, 8192), (3, 8193), (2, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(dt, rows, cols, residual):
    g = gen(rows * 100003 + cols)
    x = (3 * rand(g, rows, cols)).to(DT[dt])
    res = rand(g, rows, cols).to(DT[dt]) if residual else None
    check_norm(x, 1 + 0.3 * rand(g, cols), res, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [16, 192, 384, 640, 768, 1024, 1536, 12288])
def test_norm_forward_of_widths_that_threads_fit_exactly_or_nearly(dt, cols):
    g = gen(cols)
    for rows in (1, 5, 67):
        x, res = (3 * rand(g, rows, cols)).to(DT[dt]), rand(g, rows, cols).to(DT[dt])
        check_norm(x, 1 + 0.3 * rand(g, cols), res, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_norm_strides_offsets_and_in_place(dt):
    g = gen(5)
    rows, cols = 37, 300
    for pad, off in ((8, 8), (3, 1), (5, 0)):
        big = (2 * rand(g, rows, cols + pad + off)).to(DT[dt])
        res = rand(g, rows, cols + 5).to(DT[dt])[:, 2:cols + 2]
        x = big[:, off:off + cols]
        w = (1 + rand(g, cols + 1))[1:]
        check_norm(x, w, res, dt)
        want = (x.double() + res.double())
        before = big.clone()
        q, sc = rs.fp8_empty(rows, cols)
        rs.rs_rms_norm_fwd(x, w, q, sc, residual=res, sum=x)
        close(x, want, (U + HALF_ULP[dt]) * want.abs())
        before[:, off:off + cols] = x
        assert torch.equal(before, big)                      # nothing outside the matrix is written


def test_norm_no_bytes_past_the_columns():
    g = gen(6)
    for cols in (1, 7, 130, 777):
        raw = torch.full((5, -(-cols // 16) * 16 + 16), 0xAB, dtype=torch.uint8, device="cuda")
        _, sc = rs.fp8_empty(5, cols)
        rs.rs_rms_norm_fwd(rand(g, 5, cols), torch.ones(cols, device="cuda"), raw[:, :cols], sc)
        assert bool((raw[:, cols:] == 0xAB).all())


def test_norm_zero_rows_empty_rows_and_not_finite_values():
    x = torch.zeros(4, 300, device="cuda")
    x[1] = 1.0
    x[2, 5] = math.inf
    x[3, 7] = math.nan
    w = torch.ones(300, device="cuda")
    q, sc, _, y, rstd = norm_fwd(x, w, y=True)
    assert bool((q[0].float() == 0).all()) and bool((sc[:, 0] == np.float32(2.0 ** -100 / 448)).all())
    assert abs(float(rstd[0]) - 1000.0) < 1e-2
    assert bool((q[1].float() == 448).all())
    d = rs.fp8_dequantize(q, sc)
    assert math.isnan(float(d[2, 5])) and bool(torch.isnan(d[3]).all())
    assert bool(torch.isfinite(d[:2]).all())
    e = torch.empty(0, 300, device="cuda")
    rs.rs_rms_norm_fwd(e, w, *rs.fp8_empty(0, 300))
    dw = torch.full((300,), 7.0, device="cuda")
    rs.rs_rms_norm_bwd(e, w, torch.empty(0, device="cuda"), e, e, dw, torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert bool((dw == 0).all())


def norm_bwd(s, w, rstd, dy, ds):
    dx, dw = torch.empty_like(s), torch.empty(s.shape[1], device="cuda")
    ws = torch.empty(rs.rs_rms_norm_bwd_workspace_size(*s.shape), dtype=torch.uint8, device="cuda")
    rs.rs_rms_norm_bwd(s, w, rstd, dy, dx, dw, ws, dL_dsum=ds)
    return dx, dw


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1000, 64), (5, 127), (9, 128), (4001, 129), (1, 256), (70, 257),
                                       (1700, 512), (5, 777), (3000, 1000), (2, 1025), (900, 2048), (3, 2050),
                                       (400, 4096), (3, 8193), (200, 16384)])
@pytest.mark.parametrize("ds", [False, True])
def test_norm_backward(dt, rows, cols, ds):
    g = gen(rows * 7 + cols)
    s, dy = (2 * rand(g, rows, cols)).to(DT[dt]), rand(g, rows, cols).to(DT[dt])
    dsum = rand(g, rows, cols).to(DT[dt]) if ds else None
    w = 1 + 0.3 * rand(g, cols)
    rstd = (s.double().pow(2).mean(1) + 1e-6).rsqrt().float()
    dx, dw = norm_bwd(s, w, rstd, dy, dsum)
    rho = rstd.double()[:, None]
    xh, t = s.double() * rho, dy.double() * w.double()
    mean = (t * xh).mean(1, keepdim=True)
    want = rho * (t - xh * mean) + (dsum.double() if ds else 0)
    # the mean is a sum with cancellation: its error is relative to the mean of magnitudes
    slack = rho * (4 * U * t.abs() + xh.abs() * (64 * U * (t * xh).abs().mean(1, keepdim=True) + 4 * U * mean.abs()))
    close(dx, want, slack + (2 * U + HALF_ULP[dt]) * want.abs() + 2 * U * (dsum.double().abs() if ds else 0) + 2.0 ** -24)
    # a thread adds its rows one after another, then at most 8 + 32 + 5 partial sums: chains of rows + 64 at most
    mags = (dy.double() * xh).abs()
    close(dw, (dy.double() * xh).sum(0), (rows + 64) * U * mags.sum(0) + U * mags.amax(0))
    dx2, dw2 = norm_bwd(s, w, rstd, dy, dsum)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)     # sums in a fixed order


def test_norm_backward_against_differences():
    """L = sum(G y): central differences of the forward's own float32 y along random directions.  The step 1/64 leaves a
    truncation error of about (1/64)^2 / 6 of the third derivative (of order |G|) and the rounding of y (2^-23 of y)
    64 / 2 times over, both summed over 600 values: 1e-3 of |G| sqrt(600) bounds them."""
    g = gen(77)
    rows, cols, h = 3, 200, 1 / 64
    x, w, G = 1.5 * rand(g, rows, cols), 1 + 0.3 * rand(g, cols), rand(g, rows, cols)
    _, _, _, _, rstd = norm_fwd(x, w, want_sum=False)
    dx, dw = norm_bwd(x, w, rstd, G, None)

    def loss(xx, ww):
        y = torch.empty_like(xx)
        rs.rs_rms_norm_fwd(xx, ww, y=y)
        return float((G.double() * y.double()).sum())

    for k in range(4):
        v, u = rand(g, rows, cols), rand(g, cols)
        fd = (loss(x + h * v, w) - loss(x - h * v, w)) / (2 * h)
        assert abs(fd - float((dx.double() * v.double()).sum())) < 1e-3 * math.sqrt(rows * cols)
        fd = (loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h)
        assert abs(fd - float((dw.double() * u.double()).sum())) < 1e-3 * math.sqrt(rows * cols)


def test_norm_backward_in_place():
    g = gen(8)
    s, dy, ds, w = rand(g, 50, 384), rand(g, 50, 384), rand(g, 50, 384), rand(g, 384)
    rstd = (s.pow(2).mean(1) + 1e-6).rsqrt()
    want, dw = norm_bwd(s, w, rstd, dy, ds)
    ws = torch.empty(rs.rs_rms_norm_bwd_workspace_size(50, 384), dtype=torch.uint8, device="cuda")
    for target in (0, 1):
        a, b = dy.clone(), ds.clone()
        rs.rs_rms_norm_bwd(s, w, rstd, a, (a, b)[target], dw, ws, dL_dsum=b)
        assert torch.equal((a, b)[target], want)


def test_rows_far_apart():
    """Row offsets past 2^32 bytes."""
    stride = (1 << 31) + 64
    flat = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((3, 200), (stride, 1))
    g = gen(9)
    x.copy_(rand(g, 3, 200))
    w = torch.ones(200, device="cuda")
    check_norm(x, w, None, "bf16")
    q, sc = rs.fp8_empty(3, 200)
    q2, sc2 = rs.fp8_empty(3, 200)
    rs.rs_quantize_fp8(x, q, sc)
    rs.rs_quantize_fp8(x.contiguous(), q2, sc2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)
    far = torch.empty(2 * (1 << 32) + 512, dtype=torch.uint8, device="cuda").as_strided((3, 200), (1 << 32, 1))
    far.copy_(q.view(torch.uint8))
    out, out2 = torch.empty(3, 3, device="cuda"), torch.empty(3, 3, device="cuda")
    for o, m in ((out, far), (out2, q)):
        ws = torch.empty(max(1, rs.rs_matmul_fp8_workspace_size(3, 3, 200)), dtype=torch.uint8, device="cuda")
        rs.rs_matmul_fp8(m, sc, m, sc, o, ws)
    assert torch.equal(out, out2)


# ------------------------------------------------------------------ 8-bit forms

def plain_q(x):
    """(bytes, scales) of x [r, c] by the definition, float32 on the CPU (each operation correctly rounded)."""
    r, c = x.shape
    kb = -(-c // 128)
    xp = torch.zeros(r, kb * 128)
    xp[:, :c] = x.float().cpu()
    xp = xp.view(r, kb, 128)
    top = xp.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    q = (xp * (f / top)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(r, kb * 128)[:, :c]
    return q, (top / f).squeeze(2).t().contiguous()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (16, 128), (128, 16), (127, 129), (129, 127),
                                       (128, 128), (1000, 77), (77, 1000), (260, 516)])
@pytest.mark.parametrize("relu", [False, True])
def test_quantize_bit_exact(dt, rows, cols, relu):
    g = gen(rows + 1000 * cols)
    x = (rand(g, rows, cols) * torch.exp(2 * rand(g, rows, 1))).to(DT[dt])
    m = rand(g, rows, cols).to(DT[dt]) if relu else None
    want = torch.where(m > 0, x, torch.zeros_like(x)) if relu else x
    (q, sc), (qt, sct) = rs.fp8_empty(rows, cols), rs.fp8_empty(cols, rows)
    rs.rs_quantize_fp8(x, q, sc, qt, sct, relu=m)
    same = lambda a, b: torch.equal((a.view(torch.uint8) & 0x7f).cpu(), b & 0x7f) and \
        torch.equal(rs.fp8_dequantize(a, torch.ones(-(-a.shape[1] // 128), a.shape[0], device="cuda")).cpu(),
                    b.view(torch.float8_e4m3fn).float())
    for got, s, w in ((q, sc, want), (qt, sct, want.t())):
        pq, ps = plain_q(w)
        assert same(got, pq) and torch.equal(s.cpu(), ps)
    # each form alone gives the same
    (q1, s1), (q2, s2) = rs.fp8_empty(rows, cols), rs.fp8_empty(cols, rows)
    rs.rs_quantize_fp8(x, q1, s1, relu=m)
    rs.rs_quantize_fp8(x, qt=q2, scales_t=s2, relu=m)
    assert torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s1, sc)
    assert torch.equal(q2.view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s2, sct)


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 128), (129, 257), (300, 77), (512, 256)])
def test_quantize_blocks(rows, cols):
    g = gen(rows)
    w = rand(g, rows, cols)
    rb, cb = -(-rows // 128), -(-cols // 128)
    q, qt = rs.fp8_empty(rows, cols)[0], rs.fp8_empty(cols, rows)[0]
    sc, sct = torch.empty(cb, rb, device="cuda"), torch.empty(rb, cb, device="cuda")
    rs.rs_quantize_fp8_blocks(w, q, sc, qt, sct)
    pad = torch.zeros(rb * 128, cb * 128)
    pad[:rows, :cols] = w.cpu()
    top = pad.view(rb, 128, cb, 128).abs().amax((1, 3)).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    full = (f / top).repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = (pad * full).clamp(-448, 448).to(torch.float8_e4m3fn).float()[:rows, :cols]
    assert torch.equal(q.float().cpu(), want) and torch.equal(qt.float().cpu(), want.t())
    assert torch.equal(sc.cpu(), (top / f).t()) and torch.equal(sct.cpu(), top / f)


def test_quantize_values_that_are_not_finite_and_extremes():
    x = torch.zeros(4, 256, device="cuda")
    x[0, 3], x[0, 130] = math.inf, 2.0
    x[1, 3], x[1, 4], x[1, 130] = math.nan, 5.0, -3.0
    x[2, 0] = 3e38
    x[3, 0] = 1e-42
    q, sc = rs.fp8_empty(4, 256)
    rs.rs_quantize_fp8(x, q, sc)
    d = rs.fp8_dequantize(q, sc)
    assert bool(torch.isnan(d[0, :128]).all()) and float(d[0, 130]) == 2.0
    assert math.isnan(float(d[1, 3])) and float(d[1, 4]) == 5.0 and float(d[1, 130]) == -3.0
    assert abs(float(d[2, 0]) / 3e38 - 1) < 1e-6 and abs(float(d[3, 0])) < 2e-30


# ------------------------------------------------------------------ matrix product

def operands(g, m, n, k, blocks):
    """Random e4m3 bytes (every finite value) and scales."""
    q = lambda r: torch.randint(0, 256, (r, k), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    kb = -(-k // 128)

    def mat(r):
        b = q(r)
        b[(b & 0x7f) == 0x7f] = 0x38
        out = rs.fp8_empty(r, k)[0]
        out.view(torch.uint8).copy_(b)
        return out

    sc = lambda r: torch.exp(rand(g, kb, r)) * 1e-3
    return mat(m), sc(m), mat(n), sc(-(-n // 128) if blocks else n)


def product(a, sa, b, sb):
    k, n = a.shape[1], b.shape[0]
    exp = lambda s: s.double().repeat_interleave(128, 0)[:k]
    sbn = sb if sb.shape[1] == n else sb.repeat_interleave(128, 1)[:, :n]
    A, B = a.float().double() * exp(sa).t(), b.float().double() * exp(sbn).t()
    return A @ B.t(), A.abs() @ B.abs().t()


def matmul(a, sa, b, sb, dt="f32", relu=False, out=None):
    m, k = a.shape
    n = b.shape[0]
    out = torch.full((m, n), float("nan"), dtype=DT[dt], device="cuda") if out is None else out
    ws = torch.empty(max(1, rs.rs_matmul_fp8_workspace_size(m, n, k)), dtype=torch.uint8, device="cuda")
    rs.rs_matmul_fp8(a, sa, b, sb, out, ws, relu=relu)
    return out


SIZES = [(1, 1, 1), (1, 3, 128), (1, 512, 512), (1, 1000, 4096), (2, 777, 130), (5, 64, 64), (7, 128, 1000),
         (8, 256, 128), (15, 300, 640), (16, 129, 257), (17, 1001, 777), (31, 512, 2048), (33, 200, 384),
         (63, 96, 160), (64, 640, 1024), (65, 128, 128), (100, 100, 100), (127, 255, 129), (128, 256, 256),
         (129, 257, 385), (256, 512, 1024), (257, 130, 127), (300, 3, 500), (500, 777, 333), (1000, 64, 2000),
         (1024, 1024, 512), (4100, 260, 260), (20000, 128, 96), (128, 128, 20000), (200, 320, 33333), (3, 5, 70000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("blocks", [True, False])
def test_matmul(m, n, k, blocks):
    g = gen(m + n * 3 + k * 5)
    a, sa, b, sb = operands(g, m, n, k, blocks)
    want, mags = product(a, sa, b, sb)
    tol = (128 + k / 128 + 4) * 2 * U * mags
    got = matmul(a, sa, b, sb)
    close(got, want, tol)
    assert torch.equal(got, matmul(a, sa, b, sb))            # sums in a fixed order
    for dt in ("f16", "bf16"):
        small = sb * (1 / max(1.0, float(want.abs().max()))) * 100     # inside float16's range
        w2, m2 = product(a, sa, b, small)
        close(matmul(a, sa, b, small, dt), w2, (128 + k / 128 + 4) * 2 * U * m2 + HALF_ULP[dt] * w2.abs() * 1.01 + 2.0 ** -24)
    close(matmul(a, sa, b, sb, relu=True), want.clamp_min(0), tol)


# long contractions of few tiles are split and joined: 9, 10, 38 and 76 stretches of blocks
@pytest.mark.parametrize("m,n,k", [(300, 140, 10100), (300, 140, 10300), (130, 60, 39000), (70, 50, 80001)])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_matmul_split_sums(m, n, k, dt):
    g = gen(m + n * 3 + k * 5)
    a, sa, b, sb = operands(g, m, n, k, False)
    sb = sb * (1 / max(1.0, float(product(a, sa, b, sb)[0].abs().max()))) * 100     # inside float16's range
    want, mags = product(a, sa, b, sb)
    tol = (128 + k / 128 + 4) * 2 * U * mags
    if dt != "f32":
        tol = tol + HALF_ULP[dt] * want.abs() * 1.01 + 2.0 ** -24
    wide = torch.full((m, n + 3), 7.0, dtype=DT[dt], device="cuda")
    got = matmul(a, sa, b, sb, dt, out=wide[:, 1:1 + n])
    close(got, want, tol)
    assert bool((wide[:, :1] == 7.0).all()) and bool((wide[:, 1 + n:] == 7.0).all())
    assert torch.equal(got, matmul(a, sa, b, sb, dt))
    assert torch.equal(matmul(a, sa, b, sb, dt, relu=True), got.clamp_min(0))


@pytest.mark.parametrize("m,n,k", [(1, 100, 200), (40, 100, 200), (300, 260, 200)])
def test_matmul_strides_and_untouched_memory(m, n, k):
    g = gen(3)
    a, sa, b, sb = operands(g, m, n, k, True)
    wide = torch.zeros(m, 512, dtype=torch.uint8, device="cuda")
    wide[:, 64:64 + k] = a.view(torch.uint8)
    wide[:, 64 + k:] = 0x7f                                  # NaN past the columns must not be read into the sums
    base = matmul(a, sa, b, sb)
    assert torch.equal(matmul(wide[:, 64:64 + k], sa, b, sb), base)
    for off in (0, 1, 8):
        big = torch.full((m + 2, n + 24), 7.0, device="cuda")
        view = big[1:1 + m, off:off + n]
        matmul(a, sa, b, sb, out=view)
        assert torch.equal(view, base)
        keep = torch.ones_like(big, dtype=torch.bool)
        keep[1:1 + m, off:off + n] = False
        assert bool((big[keep] == 7.0).all())


def test_matmul_nan_rows_stay_rows():
    g = gen(4)
    for m in (20, 200):
        a, sa, b, sb = operands(g, m, 300, 256, True)
        base = matmul(a, sa, b, sb)
        a.view(torch.uint8)[7, 100] = 0x7f
        b.view(torch.uint8)[150, 200] = 0x7f
        out = matmul(a, sa, b, sb, relu=True)
        bad = torch.zeros(m, 300, dtype=torch.bool, device="cuda")
        bad[7], bad[:, 150] = True, True
        assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], base.clamp_min(0)[~bad])


def test_matmul_empty_extents():
    z = torch.zeros(0, 16, dtype=torch.uint8, device="cuda")
    e = torch.empty(0, 5, device="cuda")
    one = rs.fp8_empty(5, 16)
    rs.rs_matmul_fp8(z, torch.empty(1, 0, device="cuda"), one[0], one[1], e)
    out = torch.full((3, 5), 7.0, device="cuda")
    rs.rs_matmul_fp8(torch.empty(3, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 3, device="cuda"),
                     torch.empty(5, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 5, device="cuda"), out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("m,n,k", [(40, 96, 64), (1000, 300, 140)])
def test_linear_backward_against_formula_and_differences(m, n, k):
    """Y = A W^T on the 8-bit values A, W.  dA and dW of L = sum(G Y) by the transposed forms; L is linear in A and
    in W, so a difference along any direction V equals <dA, V> up to rounding.  G is made of few-bit values so that its
    8-bit forms are exact, both along rows and along columns (one magnitude per block)."""
    g = gen(m)
    w = rand(g, n, k)
    a = rand(g, m, k)
    G = torch.where(rand(g, m, n) > 0, 0.5, -0.5)
    (qa, sa), (qat, sat) = rs.fp8_empty(m, k), rs.fp8_empty(k, m)
    rs.rs_quantize_fp8(a, qa, sa, qat, sat)
    qw, qwt = rs.fp8_empty(n, k)[0], rs.fp8_empty(k, n)[0]
    nb, kb = -(-n // 128), -(-k // 128)
    sw, swt = torch.empty(kb, nb, device="cuda"), torch.empty(nb, kb, device="cuda")
    rs.rs_quantize_fp8_blocks(w, qw, sw, qwt, swt)
    (gq, gs), (gqt, gst) = rs.fp8_empty(m, n), rs.fp8_empty(n, m)
    rs.rs_quantize_fp8(G, gq, gs, gqt, gst)
    assert torch.equal(rs.fp8_dequantize(gq, gs), G)
    da, dw = matmul(gq, gs, qwt, swt), matmul(gqt, gst, qat, sat)
    W, At = rs.fp8_dequantize(qw, sw).double(), rs.fp8_dequantize(qat, sat).double()
    close(da, G.double() @ W, (132 + n / 128) * 2 * U * (G.abs().double() @ W.abs()))
    close(dw, G.double().t() @ At.t(), (132 + m / 128) * 2 * U * (G.abs().double().t() @ At.abs().t()))
    # difference in A: two 8-bit points A1, A2, L(A1) - L(A2) = <dA, A1 - A2>
    q2, s2 = rs.fp8_empty(m, k)
    rs.rs_quantize_fp8(a + 0.3 * rand(g, m, k), q2, s2)
    A1, A2 = rs.fp8_dequantize(qa, sa).double(), rs.fp8_dequantize(q2, s2).double()
    L = lambda q, s: float((G.double() * matmul(q, s, qw, sw).double()).sum())
    fd, an = L(qa, sa) - L(q2, s2), float((da.double() * (A1 - A2)).sum())
    mags = float((G.abs().double() * ((A1.abs() + A2.abs()) @ W.abs().t())).sum())
    assert abs(fd - an) <= (264 + (k + n) / 128) * 2 * U * mags


# ------------------------------------------------------------------ gradient norm and clipping

def tensors(g, sizes, kinds=("f32", "bf16", "f16"), scale=1.0):
    return [(scale * rand(g, k)).to(DT[kinds[i % len(kinds)]]) for i, k in enumerate(sizes)]


def clip_ws(n):
    return torch.empty(rs.rs_grad_norm_workspace_size(n), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [8191, 8192, 8193], [1000003], [7] * 401, [100 + 13 * i for i in range(900)],
                                   [3_000_001, 17, 64, 0, 250_000]])
@pytest.mark.parametrize("limit", [0.25, 4.0])
def test_clip(sizes, limit):
    g = gen(len(sizes) + sizes[0])
    ts = tensors(g, sizes)
    want = math.sqrt(sum(float(t.double().pow(2).sum()) for t in ts))
    outs = [torch.full_like(t, 9.0) for t in ts]
    norm, ws = torch.empty(1, device="cuda"), clip_ws(len(ts))
    keep = [t.clone() for t in ts]
    rs.rs_grad_clip([rs.GradTensor(t, out=o) for t, o in zip(ts, outs)], limit * want, norm, ws)
    # chains: 32 values a chunk and at most 2 chunks, 5 shuffles, 8 warps, then float64
    assert abs(float(norm) / want - 1) < 80 * U
    c = min(np.float32(1), np.float32(limit * want) / (np.float32(float(norm)) + np.float32(1e-6)))
    for t, o, k in zip(ts, outs, keep):
        assert torch.equal(t, k)
        assert torch.equal(o, (t.float() * float(c)).to(t.dtype))
    rs.rs_grad_clip([rs.GradTensor(t, out=t) for t in ts], limit * want, norm, ws)
    for t, o in zip(ts, outs):
        assert torch.equal(t, o)                              # in place
    n2 = torch.empty(1, device="cuda")
    rs.rs_grad_norm([rs.GradTensor(t) for t in keep], n2, ws)
    rs.rs_grad_norm(rs.GradTable([rs.GradTensor(t) for t in keep]), norm, ws)
    assert torch.equal(n2, norm) and abs(float(n2) / want - 1) < 80 * U


def test_clip_of_nothing_and_of_unaligned_tensors():
    norm, ws = torch.full((1,), 5.0, device="cuda"), clip_ws(3)
    rs.rs_grad_clip([], 1.0, norm, ws)
    assert float(norm) == 0
    rs.rs_grad_norm([rs.GradTensor(torch.empty(0, device="cuda"))], norm, ws)
    assert float(norm) == 0
    g = gen(11)
    flat = rand(g, 30000)
    ts = [flat[1:9000], flat[9001:9003], flat[9003:25000]]
    out = torch.full((30000,), 9.0, device="cuda")
    rs.rs_grad_clip([rs.GradTensor(t, out=out[t.storage_offset():t.storage_offset() + t.numel()]) for t in ts], 1.0, norm, ws)
    want = math.sqrt(sum(float(t.double().pow(2).sum()) for t in ts))
    assert abs(float(norm) / want - 1) < 80 * U
    mask = torch.ones(30000, dtype=torch.bool, device="cuda")
    mask[1:9000] = mask[9001:25000] = False
    assert bool((out[mask] == 9.0).all()) and bool((out[~mask] != 9.0).all())


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_clip_values_that_are_not_finite(bad):
    t = torch.ones(1000, device="cuda")
    t[5] = bad
    o, norm = torch.empty_like(t), torch.empty(1, device="cuda")
    rs.rs_grad_clip([rs.GradTensor(t, out=o)], 1.0, norm, clip_ws(1))
    c = 1.0 / (float(norm) + 1e-6)
    assert math.isnan(float(norm)) if math.isnan(bad) else math.isinf(float(norm))
    assert math.isnan(float(o[5])) and (math.isnan(float(o[0])) if math.isnan(bad) else float(o[0]) == c == 0.0)


ACTS = (rs.RS_ACT_IDENTITY, rs.RS_ACT_EXP, rs.RS_ACT_SIGMOID)


def adam_groups(g, sizes):
    out = []
    for i, k in enumerate(sizes):
        act = ACTS[i % 3]
        p = 0.5 * rand(g, k) - (3.0 if act == rs.RS_ACT_EXP else 0.0)
        out.append(rs.AdamGroup(p, rand(g, k), 0.1 * rand(g, k), 0.01 * rand(g, k).square(), 10.0 ** -(2 + i % 3), act,
                                torch.full((k,), 3.0, device="cuda") if act else None))
    return out


def copy_groups(gs):
    c = lambda t: None if t is None else t.clone()
    return [rs.AdamGroup(c(q.param), c(q.grad), c(q.m), c(q.v), q.lr, q.activation, c(q.activated)) for q in gs]


def same_groups(a, b):
    eq = lambda x, y: (x is None and y is None) or torch.equal(x, y)
    return all(eq(x.param, y.param) and eq(x.m, y.m) and eq(x.v, y.v) and eq(x.activated, y.activated) for x, y in zip(a, b))


def chained(q):
    p, gr = q.param.double(), q.grad.double()
    if q.activation == rs.RS_ACT_EXP:
        return gr * p.exp()
    return gr * p.sigmoid() * (1 - p.sigmoid()) if q.activation == rs.RS_ACT_SIGMOID else gr


@pytest.mark.parametrize("sizes", [[1], [3 * 1007, 3 * 1007, 1007, 45 * 1007 - 5, 0], [40000] * 16])
@pytest.mark.parametrize("limit", [0.1, 10.0])
def test_adam_step_clipped(sizes, limit):
    g = gen(sizes[0])
    a = adam_groups(g, sizes)
    b = copy_groups(a)
    want = math.sqrt(sum(float(chained(q).pow(2).sum()) for q in a))
    norm = torch.empty(1, device="cuda")
    rs.rs_adam_step_clipped(a, 3, limit * want, norm, clip_ws(len(a)))
    assert abs(float(norm) / want - 1) < 96 * U              # the activations' derivatives add a few roundings
    c = min(np.float32(1), np.float32(limit * want) / (np.float32(float(norm)) + np.float32(1e-6)))
    for q, r in zip(b, a):
        assert torch.equal(q.grad, r.grad)
        q.grad = q.grad * float(c)
    rs.rs_adam_step(b, 3)
    assert same_groups(a, b)                                 # the unclipped step on scaled gradients, bit for bit


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_adam_step_clipped_skips_what_is_not_finite(bad):
    a = adam_groups(gen(2), [1000, 999])
    a[1].grad[7] = bad
    b = copy_groups(a)
    norm = torch.empty(1, device="cuda")
    rs.rs_adam_step_clipped(a, 1, 1.0, norm, clip_ws(2))
    assert same_groups(a, b) and not math.isfinite(float(norm))


def test_calls_on_another_stream():
    """Everything runs on the stream given, after what is on it."""
    s = torch.cuda.Stream()
    g = gen(12)
    x, w = rand(g, 5000, 512), torch.ones(512, device="cuda")
    q0, sc0, *_ = norm_fwd(x, w)
    torch.cuda.synchronize()
    later = torch.zeros_like(x)
    q, sc = rs.fp8_empty(5000, 512)
    out, norm, ws = torch.empty(5000, 5000, device="cuda"), torch.empty(1, device="cuda"), clip_ws(1)
    mws = torch.empty(max(1, rs.rs_matmul_fp8_workspace_size(5000, 5000, 512)), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        later.copy_(x)
    rs.rs_rms_norm_fwd(later, w, q, sc, stream=s)
    rs.rs_matmul_fp8(q, sc, q, sc, out, mws, stream=s)
    rs.rs_grad_norm([rs.GradTensor(out)], norm, ws, stream=s)
    s.synchronize()
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(sc, sc0)
    want = product(q0, sc0, q0, sc0)[0]
    assert abs(float(norm) / float(want.norm()) - 1) < 1e-5
