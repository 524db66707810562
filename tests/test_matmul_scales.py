"""The 8-bit matrix product with scales whose product is no normal float32 although the results are: below 2^-126 it would be
rounded to a few bits or zero, above 2^128 it would be infinite and make NaN of a sum of zero.  Every kernel and both scale forms are held to
the tolerance of ordinary scales, (128 + k / 128 + 4) 2u of the sum of magnitudes (2u = 2^-23): scaling by one factor after the
other rounds once more, within the 4."""
import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

from . import test_gpu_wide as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()
    yield
    assert rs.rs_device_error() == rs.RS_OK


# the kernels of up to 16, 32 and 64 rows, tiles of 128 and 256 columns, split sums
SIZES = [(7, 300, 500), (30, 300, 500), (64, 300, 500), (65, 300, 500), (300, 140, 10100), (9800, 300, 200), (2000, 700, 10000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("blocks", [True, False])
def test_small_scales(m, n, k, blocks):
    """Scales of about 2^-80 and 2^-60; sums mostly above 2^15, so that nearly all results are normal numbers.  A product
    of the scales formed first is a multiple of 2^-149: 2^-10 of it lost, 2^6 times the tolerance.  Where even the magnitudes add
    up to less than 2^-126, an addition loses at most 2^-149, which is 2u of 2^-126."""
    a, sa, b, sb = W.operands(W.gen(m), m, n, k, blocks)
    sa, sb = sa.clamp(5e-4, 2e-3) * (1000 * 2.0 ** -80), sb.clamp(5e-4, 2e-3) * (1370 * 2.0 ** -60)
    want, mags = W.product(a, sa, b, sb)
    assert float((mags > 2.0 ** -126).double().mean()) > 0.99
    W.close(W.matmul(a, sa, b, sb), want, (128 + k / 128 + 4) * 2 * W.U * mags.clamp_min(2.0 ** -126))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("blocks", [True, False])
def test_large_scales(m, n, k, blocks):
    """Scales of about 2^70 and 2^60, values of 2^-9 (sums of 2^-11 at most), and rows of zeros, which stay zero."""
    g = W.gen(m)
    a, sa, b, sb = W.operands(g, m, n, k, blocks)
    for q in (a, b):
        q.view(torch.uint8)[:] = torch.randint(0, 2, q.shape, device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
        q.view(torch.uint8)[::5] = 0
    sa, sb = sa.clamp(5e-4, 2e-3) * (1000 * 2.0 ** 70), sb.clamp(5e-4, 2e-3) * (1370 * 2.0 ** 60)
    want, mags = W.product(a, sa, b, sb)
    assert float(mags.max()) < 2.0 ** 127
    got = W.matmul(a, sa, b, sb)
    W.close(got, want, (128 + k / 128 + 4) * 2 * W.U * mags)
    assert bool((got[::5] == 0).all()) and bool((got[:, ::5] == 0).all())


@pytest.mark.parametrize("m", [64, 65, 9800])
@pytest.mark.parametrize("blocks", [True, False])
def test_ordinary_and_extreme_blocks_side_by_side(m, blocks):
    """One block of four has extreme scales, and in one row and column alone: the others' sums are as they are without."""
    n, k = 300, 512
    a, sa, b, sb = W.operands(W.gen(m), m, n, k, blocks)
    sa, sb = sa.clamp(5e-4, 2e-3), sb.clamp(5e-4, 2e-3)
    base = W.matmul(a, sa, b, sb)
    sa2, sb2 = sa.clone(), sb.clone()
    sa2[2, 5], sb2[2, 0] = 2.0 ** -80, 1.37 * 2.0 ** -60
    want, mags = W.product(a, sa2, b, sb2)
    got = W.matmul(a, sa2, b, sb2)
    W.close(got, want, (128 + k / 128 + 4) * 2 * W.U * mags)
    cols = slice(128, None) if blocks else slice(1, None)
    rows = torch.arange(m, device="cuda") != 5
    assert torch.equal(got[rows][:, cols], base[rows][:, cols])


@pytest.mark.parametrize("m", [64, 65, 2000])
def test_rows_of_zeros_against_small_weights(m):
    """As the quantiser leaves them: a block of zeros has a scale of 2^-109, whose product with small weights' is subnormal.  The
    rows' other blocks count as ever."""
    g = W.gen(m)
    x, w = W.rand(g, m, 700), 1e-6 * W.rand(g, 300, 700)
    x[::3, 128:384] = 0
    x[1] = 0
    x[2, 256:] *= 2.0 ** -95                                     # nonzero, and below the smallest scale's block
    (a, sa), b = rs.fp8_empty(m, 700), rs.fp8_empty(300, 700)[0]
    sb, sbt = torch.empty(6, 3, device="cuda"), torch.empty(3, 6, device="cuda")
    rs.rs_quantize_fp8(x, a, sa)
    rs.rs_quantize_fp8_blocks(w, b, sb, rs.fp8_empty(700, 300)[0], sbt)
    want, mags = W.product(a, sa, b, sb)
    got = W.matmul(a, sa, b, sb)
    W.close(got, want, (128 + 700 / 128 + 4) * 2 * W.U * mags.clamp_min(2.0 ** -126))
    assert bool((got[1] == 0).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off,pad", [(0, 4), (1, 2)])
def test_rows_formed_anew_leave_like_others(dt, off, pad):
    """Through a relu, into 16 bits, into rows on and off 16-byte boundaries with nothing written beside them."""
    m, n, k = 400, 300, 500
    a, sa, b, sb = W.operands(W.gen(8), m, n, k, True)
    sa, sb = sa.clamp(5e-4, 2e-3), sb.clamp(5e-4, 2e-3) * 2.0 ** -60
    sa[:, ::7] *= 2.0 ** -70
    want, mags = W.product(a, sa, b, sb)
    tol = (128 + k / 128 + 4) * 2 * W.U * mags.clamp_min(2.0 ** -126) + (W.HALF_ULP[dt] * 1.01 * want.abs() if dt != "f32" else 0)
    tol = tol + (2.0 ** -133 if dt != "f32" else 0)              # bf16's subnormal step
    big = torch.full((m + 2, n + off + pad), 7.0, dtype=W.DT[dt], device="cuda")
    view = big[1:1 + m, off:off + n]
    W.matmul(a, sa, b, sb, dt, relu=True, out=view)
    W.close(view, want.clamp_min(0), tol)
    view.fill_(7.0)
    assert bool((big == 7.0).all())
