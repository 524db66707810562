"""Who waits for whom in the 8-bit matrix product.  Tensor memory is asked for with a wait that nothing bounds, so no CTA may
hold it while it waits for one that may still be asking: products on several streams share SMs, and two clusters
could each hold what the other's members wait for."""
import os
import re

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs


def kernel_body(name):
    """The statements of a kernel of matmul.cu, comments taken out."""
    with open(os.path.join(build_lib.CSRC, "matmul.cu")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    m = re.search(r"__global__[^;{]*?\b" + name + r"\s*\(", src, re.S)
    at = src.index("{", m.end())
    depth, end = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(src[end], 0)
        end += 1
        if depth == 0:
            return src[at:end]


def test_few_rows_free_tensor_memory_before_they_wait_for_their_cluster():
    body = kernel_body("k_matmul_rows")
    alloc, dealloc, first = (body.index(s) for s in ("tcgen05.alloc", "tcgen05.dealloc", "cluster_sync()"))
    assert body.count("tcgen05.alloc") == body.count("tcgen05.dealloc") == 1
    assert alloc < dealloc < first


def test_tiles_share_no_sm():
    """A pair of the tile kernel does wait for its other half with tensor memory in hand: two such CTAs must not fit an SM
    (228 KB of shared memory)."""
    with open(os.path.join(build_lib.CSRC, "matmul.cu")) as f:
        assert re.search(r"static_assert\(2 \* sizeof\(TileSmem<128>\) > kSmemSm && 2 \* sizeof\(TileSmem<256>\) > kSmemSm",
                         f.read())


@pytest.mark.gpu
def test_products_of_few_rows_on_several_streams():
    """Each stream's products give what they give alone, bit for bit."""
    build_lib.build()
    g = torch.Generator("cuda").manual_seed(21)

    def mat(r, c):
        q, s = rs.fp8_empty(r, c)
        rs.rs_quantize_fp8(torch.randn(r, c, device="cuda", generator=g), q, s)
        return q, s

    jobs = []
    for m, n, k in ((5, 1200, 2048), (16, 4096, 1024), (9, 2500, 4096), (16, 640, 2048), (40, 1200, 2048), (64, 300, 8192)):
        a, b, out = mat(m, k), mat(n, k), torch.empty(m, n, device="cuda")
        rs.rs_matmul_fp8(*a, *b, out)
        jobs.append((a, b, out, out.clone(), torch.cuda.Stream()))
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for a, b, out, _, stream in jobs:
            rs.rs_matmul_fp8(*a, *b, out, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(out, alone) for _, _, out, alone, _ in jobs)
    assert rs.rs_device_error() == rs.RS_OK
