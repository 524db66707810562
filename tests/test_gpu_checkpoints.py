"""8-bit activation checkpoints on the GPU: the product whose result leaves in 8 bits, the checkpoint's transposed form, and
a gradient through a relu kept in 8 bits.  The forms are compared bit for bit with their definition in float32 (every
operation of it is correctly rounded), the product's sums with float64."""
import math

import pytest
import torch

from gaussian_splatting_tile_gb300 import rs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def plain_q(x):
    """(bytes, scales) of x [r, c] by the definition, float32 on the CPU (each operation correctly rounded)."""
    r, c = x.shape
    kb = -(-c // 128)
    xp = torch.zeros(r, kb * 128)
    xp[:, :c] = x.float().cpu()
    xp = xp.view(r, kb, 128)
    top = xp.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    f = torch.full_like(top, 448.0)
    q = (xp * (f / top)).clamp(-448, 448).to(torch.float8_e4m3fn).view(r, kb * 128)[:, :c]
    return q.float(), (top / f).squeeze(2).t().contiguous()


def same(pair, want):
    """The form's values and scales; a zero's sign does not count."""
    return torch.equal(pair[0].view(torch.float8_e4m3fn).float().cpu(), want[0]) and torch.equal(pair[1].cpu(), want[1])


def equal(a, b):
    return torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def kept(x):
    form = rs.fp8_empty(*x.shape)
    rs.rs_quantize_fp8(x, *form)
    return form


# ------------------------------------------------------------------ the transposed form

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (16, 128), (128, 16), (127, 129), (129, 127), (128, 128),
                                       (256, 256), (1000, 77), (77, 1000), (260, 516), (3, 4096), (4100, 17)])
def test_transpose_bit_exact(rows, cols):
    g = gen(rows + 1000 * cols)
    q, sc = kept(rand(g, rows, cols) * torch.exp(2 * rand(g, rows, 1)))
    form = rs.fp8_empty(cols, rows)
    rs.rs_transpose_fp8(q, sc, *form)
    assert same(form, plain_q(rs.fp8_dequantize(q, sc).t()))


def test_transpose_of_every_byte_and_scales_of_any_size():
    """All 256 bytes in every row, scales from 2^-109 to 2^100, and a row whose scale is infinite (its values are NaN where they
    are zero): the blocks' largest magnitudes leave NaN out, as everywhere."""
    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(300, 1)
    q = torch.stack([row.roll(i) for i, row in enumerate(q)]).contiguous()
    q[(q & 0x7f) == 0x7f] = 0x38
    sc = torch.exp2(torch.linspace(-109, 100, 600, device="cuda")).view(2, 300).contiguous()
    form = rs.fp8_empty(256, 300)
    rs.rs_transpose_fp8(q, sc, *form)
    assert same(form, plain_q(rs.fp8_dequantize(q, sc).t()))
    q[5, 7], sc[0, 9] = 0x7f, math.inf
    rs.rs_transpose_fp8(q, sc, *form)
    d = rs.fp8_dequantize(*form)
    v = rs.fp8_dequantize(q, sc).t()
    # the NaN stays one value; the infinities take their blocks (rows 0 to 127 of the first 128 columns)
    assert math.isnan(float(d[7, 5])) and bool(torch.isnan(d[:128, 9]).all())
    clean = torch.isfinite(v[:, 128:]).all(1)
    assert bool(torch.isfinite(d[:, 128:][clean]).all()) and bool(torch.isfinite(d[128:]).all())


def test_transpose_strides_and_bytes_past_the_rows():
    g = gen(4)
    for rows, cols in ((5, 7), (130, 33), (17, 300)):
        q, sc = kept(rand(g, rows, cols))
        wide = torch.full((rows, -(-cols // 16) * 16 + 32), 0x7f, dtype=torch.uint8, device="cuda")
        wide[:, :cols] = q.view(torch.uint8)
        raw = torch.full((cols, -(-rows // 16) * 16 + 16), 0xAB, dtype=torch.uint8, device="cuda")
        sct = torch.empty(-(-rows // 128), cols, device="cuda")
        rs.rs_transpose_fp8(wide[:, :cols], sc, raw[:, :rows], sct)
        assert same((raw[:, :rows].contiguous(), sct), plain_q(rs.fp8_dequantize(q, sc).t()))
        assert bool((raw[:, rows:] == 0xAB).all())
    rs.rs_transpose_fp8(*rs.fp8_empty(0, 8), *rs.fp8_empty(8, 0))
    rs.rs_transpose_fp8(*rs.fp8_empty(8, 0), *rs.fp8_empty(0, 8))


def test_rows_far_apart():
    """Row offsets past 2^32 bytes, read and written."""
    g = gen(9)
    q, sc = kept(rand(g, 3, 200))
    want = rs.fp8_empty(200, 3)
    rs.rs_transpose_fp8(q, sc, *want)
    flat = torch.empty(2 * (1 << 32) + 8192, dtype=torch.uint8, device="cuda")
    far = flat.as_strided((3, 200), (1 << 32, 1))
    far.copy_(q.view(torch.uint8))
    got = rs.fp8_empty(200, 3)
    rs.rs_transpose_fp8(far, sc, *got)
    assert equal(got, want)
    back = rs.fp8_empty(3, 200)
    rs.rs_transpose_fp8(*want, *back)
    out = flat[4096:].as_strided((3, 200), (1 << 32, 1))
    rs.rs_transpose_fp8(*want, out, back[1].clone())
    assert torch.equal(out, back[0].view(torch.uint8))
    dx = rand(g, 3, 200)
    forms = [rs.fp8_empty(3, 200) for _ in range(2)]
    for u, f in ((far, forms[0]), (q, forms[1])):
        rs.rs_quantize_fp8_relu8(dx, u, *f)
    assert equal(*forms)
    # the product's rows of 8 bits
    a, b = kept(rand(g, 70, 64)), rand(g, 200, 64)
    bq = rs.fp8_empty(200, 64)[0]
    bs = torch.empty(1, 2, device="cuda")
    rs.rs_quantize_fp8_blocks(b, bq, bs)
    r = rs.fp8_empty(70, 200)
    rs.rs_matmul_fp8_q(*a, bq, bs, *r)
    flat = flat[:1]
    del far, out
    flat = torch.empty(69 * (1 << 27) + 8192, dtype=torch.uint8, device="cuda")
    far = flat.as_strided((70, 200), (1 << 27, 1))
    sc = torch.empty_like(r[1])
    rs.rs_matmul_fp8_q(*a, bq, bs, far, sc)
    assert torch.equal(far, r[0].view(torch.uint8)) and torch.equal(sc, r[1])


# ------------------------------------------------------------------ through a relu

@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (300, 1), (16, 128), (127, 129), (128, 128), (1000, 77), (77, 1000),
                                       (260, 516)])
def test_relu8_bit_exact(dt, rows, cols):
    g = gen(rows + 1000 * cols)
    x = (rand(g, rows, cols) * torch.exp(2 * rand(g, rows, 1))).to(DT[dt])
    u, _ = kept(rand(g, rows, cols))                                  # of both signs
    forms = rs.fp8_empty(rows, cols), rs.fp8_empty(cols, rows)
    rs.rs_quantize_fp8_relu8(x, u, *forms[0], *forms[1])
    want = torch.where(u.float() > 0, x, torch.zeros_like(x))
    assert same(forms[0], plain_q(want)) and same(forms[1], plain_q(want.t()))
    alone = rs.fp8_empty(rows, cols), rs.fp8_empty(cols, rows)
    rs.rs_quantize_fp8_relu8(x, u, *alone[0])
    rs.rs_quantize_fp8_relu8(x, u, qt=alone[1][0], scales_t=alone[1][1])
    assert equal(alone[0], forms[0]) and equal(alone[1], forms[1])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_relu8_of_every_byte(dt):
    """Zeros of both signs and negative values let nothing through, positive values and NaN do; rows off 16-byte boundaries
    take another path."""
    u = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(3, 1)
    v = u.view(torch.float8_e4m3fn).float()
    for x in (torch.ones(3, 256, device="cuda", dtype=DT[dt]), torch.ones(3, 259, device="cuda", dtype=DT[dt])[:, 2:258]):
        q, sc = rs.fp8_empty(3, 256)
        rs.rs_quantize_fp8_relu8(x, u, q, sc)
        assert torch.equal(rs.fp8_dequantize(q, sc) == 1, ~(v <= 0))


# ------------------------------------------------------------------ the product

def weights(g, n, k):
    q = rs.fp8_empty(n, k)[0]
    sc = torch.empty(-(-k // 128), -(-n // 128), device="cuda")
    rs.rs_quantize_fp8_blocks(rand(g, n, k) / k ** 0.5, q, sc)
    return q, sc


def wide(m):
    q, sc = m
    s = sc if sc.shape[1] == q.shape[0] else sc.repeat_interleave(128, 1)[:, :q.shape[0]]
    return q.float().double() * s.double().repeat_interleave(128, 0)[:q.shape[1]].t()


def product_q(a, b, relu=False):
    m, n, k = a[0].shape[0], b[0].shape[0], a[0].shape[1]
    form = rs.fp8_empty(m, n)
    ws = torch.empty(max(1, rs.rs_matmul_fp8_q_workspace_size(m, n, k)), dtype=torch.uint8, device="cuda")
    rs.rs_matmul_fp8_q(*a, *b, *form, ws, relu=relu)
    return form


def product(a, b, relu=False):
    m, n, k = a[0].shape[0], b[0].shape[0], a[0].shape[1]
    out = torch.empty(m, n, device="cuda")
    ws = torch.empty(max(1, rs.rs_matmul_fp8_workspace_size(m, n, k)), dtype=torch.uint8, device="cuda")
    rs.rs_matmul_fp8(*a, *b, out, ws, relu=relu)
    return out


def check_product(a, b, relu):
    form = product_q(a, b, relu)
    y, mags, k = wide(a) @ wide(b).t(), wide(a).abs() @ wide(b).abs().t(), a[0].shape[1]
    # 8 significant bits a product: exact; additions of at most 2u each (a truncating adder), one after another
    ey = (128 + k / 128 + 4) * 2 * U * mags
    y = torch.relu(y) if relu else y
    for i in range(-(-y.shape[1] // 128)):
        cut = slice(i * 128, (i + 1) * 128)
        top = y[:, cut].abs().amax(1).clamp_min(2.0 ** -100)
        etop = ey[:, cut].amax(1)
        assert bool(((form[1][i].double() - top / 448).abs() <= (etop + 2 * U * top) / 448).all())
        z = y[:, cut] / (top / 448)[:, None]
        got = form[0][:, cut].float().double()
        # where the largest magnitude is itself uncertain the bound says nothing
        sure = (etop < 0.01 * top)[:, None]
        slack = 1.1 * ((ey[:, cut] + z.abs() / 448 * etop[:, None]) / top[:, None] + 4 * U) * 448
        assert bool(((got - z).abs() <= z.abs() / 16 + 2.0 ** -10 + slack)[sure.expand_as(z)].all())
    return form


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 4096, 512), (37, 1001, 777), (64, 256, 128), (65, 256, 128), (65, 1, 64),
                                   (130, 129, 200), (256, 256, 256), (257, 255, 129), (300, 512, 1000), (777, 77, 96),
                                   (2000, 300, 260), (4100, 640, 384), (20000, 513, 100), (512, 256, 9300),
                                   (64, 200, 1024), (64, 200, 1025), (3, 517, 2000), (300, 256, 2048), (300, 250, 2100)])
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("per_row", [False, True])
def test_product(m, n, k, relu, per_row):
    g = gen(m + n + k)
    a = kept(rand(g, m, k) * torch.exp(rand(g, m, 1)))
    b = kept(rand(g, n, k) / k ** 0.5) if per_row else weights(g, n, k)
    form = check_product(a, b, relu)
    assert equal(form, product_q(a, b, relu))
    # The form of the float32 product, bit for bit, where that takes the same sums in the same order.  (A float32 product of up
    # to 64 rows multiplies a block's sum by one scale and then by the other, the tiles by the scales' product, and one that is
    # split joins its stretches' sums: other roundings of the same sum, both within the bound above.)
    if rs.rs_matmul_fp8_q_workspace_size(m, n, k) > 0 or (m > 64 and rs.rs_matmul_fp8_workspace_size(m, n, k) == 0):
        want = rs.fp8_empty(m, n)
        rs.rs_quantize_fp8(product(a, b, relu), *want)
        assert equal(form, want)


def test_product_without_a_contraction_and_of_nothing():
    for m, n in ((70, 300), (3, 5)):
        form = product_q(rs.fp8_empty(m, 0), (rs.fp8_empty(n, 0)[0], torch.empty(0, n, device="cuda")))
        zeros = kept(torch.zeros(m, n, device="cuda"))
        assert equal(form, zeros)
    product_q(rs.fp8_empty(0, 64), weights(gen(1), 8, 64))
    product_q(rs.fp8_empty(8, 64), (rs.fp8_empty(0, 64)[0], torch.empty(1, 0, device="cuda")))


def test_product_bytes_past_the_columns():
    g = gen(8)
    for m, n, k in ((100, 300, 200), (70, 5, 200), (300, 513, 200), (20, 33, 200), (20, 33, 1300), (7, 130, 1300)):
        a, b = kept(rand(g, m, k)), weights(g, n, k)
        want = product_q(a, b)
        raw = torch.full((m, -(-n // 16) * 16 + 32), 0xAB, dtype=torch.uint8, device="cuda")
        sc = torch.empty_like(want[1])
        ws = torch.empty(max(1, rs.rs_matmul_fp8_q_workspace_size(m, n, k)), dtype=torch.uint8, device="cuda")
        rs.rs_matmul_fp8_q(*a, *b, raw[:, :n], sc, ws)
        assert torch.equal(raw[:, :n], want[0].view(torch.uint8)) and torch.equal(sc, want[1])
        assert bool((raw[:, n:] == 0xAB).all())


def test_product_of_scales_whose_product_is_no_normal_number():
    """a's scales near 2^-109 and 2^100 against b's the other way round and alike: the result goes by one scale after the other."""
    g = gen(13)
    for m, k in ((300, 256), (40, 1300)):
        check_scales_apart(g, m, 300, k)


def check_scales_apart(g, m, n, k):
    a, b = kept(rand(g, m, k)), weights(g, n, k)
    a[1][:, ::3] *= 2.0 ** -70
    a[1][:, 1::3] *= 2.0 ** 70
    for f in (2.0 ** -70, 2.0 ** 40, 1.0):
        form = product_q((a[0], a[1]), (b[0], b[1] * f))
        want = rs.fp8_empty(m, n)
        rs.rs_quantize_fp8(product(a, (b[0], b[1] * f)), *want)
        assert equal(form, want)


def test_product_of_values_that_are_not_finite():
    g = gen(14)
    for m, k in ((40, 256), (40, 1300), (300, 256)):
        a, b = kept(rand(g, m, k)), weights(g, 300, k)
        a[0].view(torch.uint8)[7, 3] = 0x7f
        a[1][1, 9] = math.inf
        d = rs.fp8_dequantize(*product_q(a, b, relu=True))
        assert bool(torch.isnan(d[7]).all()) and bool(torch.isnan(d[9]).all())
        d[7], d[9] = 0, 0
        assert bool(torch.isfinite(d).all())


def test_two_streams_and_graphs():
    """Products on two streams at once, and captured calls replayed, with the checkpoints' other uses behind them."""
    g = gen(31)
    a, b = kept(rand(g, 3000, 256)), weights(g, 512, 256)
    dx = rand(g, 3000, 512).bfloat16()
    want = product_q(a, b, True)
    want_t = rs.fp8_empty(512, 3000)
    rs.rs_transpose_fp8(*want, *want_t)
    want_g = rs.fp8_empty(512, 3000)
    rs.rs_quantize_fp8_relu8(dx, want[0], qt=want_g[0], scales_t=want_g[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[rs.fp8_empty(3000, 512), rs.fp8_empty(512, 3000), rs.fp8_empty(512, 3000)] for _ in streams]

    def step(o):
        rs.rs_matmul_fp8_q(*a, *b, *o[0], relu=True)
        rs.rs_transpose_fp8(*o[0], *o[1])
        rs.rs_quantize_fp8_relu8(dx, o[0][0], qt=o[2][0], scales_t=o[2][1])

    for _ in range(3):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                step(o)
    torch.cuda.synchronize()
    good = lambda o: equal(o[0], want) and equal(o[1], want_t) and equal(o[2], want_g)
    assert all(good(o) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs[0])
    for q, sc in outs[0]:
        q.view(torch.uint8).zero_()
        sc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert good(outs[0])
