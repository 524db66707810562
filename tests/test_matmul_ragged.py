"""The 8-bit matrix product's output rows: whatever their width, offset and distance, nothing beside them is written."""
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


# rows: the few-rows kernel, 128-column tiles, 256-column tiles; a split product
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,k", [(20, 200), (300, 200), (9800, 96), (300, 10100)])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 24), (1, 3), (3, 5), (8, 16)])
def test_rows_alone_are_written(dt, m, k, off, pad):
    """Rows on 16-byte boundaries whose width is no multiple of 16 bytes among them, from widths below 16 bytes on."""
    for n in (1, 3, 4, 7, 8, 9, 31, 100, 127, 131, 257, 300, 303):
        if m > 5000 and n < 257:
            continue
        a, sa, b, sb = W.operands(W.gen(31 + n), m, n, k, True)
        sb = sb * 1e-3                                           # inside float16's range
        base = W.matmul(a, sa, b, sb, dt)
        want, mags = W.product(a, sa, b, sb)
        W.close(base, want, (128 + k / 128 + 4) * 2 * W.U * mags + W.HALF_ULP[dt] * 1.01 * want.abs() + 2.0 ** -24)
        for total in {n + off + pad, -(-(n + off + pad) // 8) * 8}:
            big = torch.full((m + 2, total), 7.0, dtype=W.DT[dt], device="cuda")
            view = big[1:1 + m, off:off + n]
            W.matmul(a, sa, b, sb, dt, out=view)
            assert torch.equal(view, base), n
            view.fill_(7.0)
            assert bool((big == 7.0).all()), (n, total)


# the few-rows kernel, 128- and 256-column tiles
@pytest.mark.parametrize("m,n", [(20, 300), (300, 140), (9800, 300)])
@pytest.mark.parametrize("blocks", [True, False])
def test_bytes_past_the_columns_do_not_count(m, n, blocks):
    """NaN in every byte between a row's last column and the next row, for widths of every remainder by 16."""
    for k in [*range(1, 18), 129, 131, 134, 140, 143, 255, 257, 383]:
        a, sa, b, sb = W.operands(W.gen(k), m, n, k, blocks)
        clean = []
        for q in (a, b):
            wide = torch.full((q.shape[0], -(-k // 16) * 16 + 16), 0x7f, dtype=torch.uint8, device="cuda")
            wide[:, :k] = q.view(torch.uint8)
            clean.append(wide[:, :k])
        want, mags = W.product(a, sa, b, sb)
        got = W.matmul(clean[0], sa, clean[1], sb)
        W.close(got, want, (128 + k / 128 + 4) * 2 * W.U * mags)
