"""What the wide network's blocks keep for the backward: each its own, and nothing that nobody reads."""
import pytest
import torch

from gaussian_splatting_tile_gb300 import rs

from . import test_gpu_sandwich_path as P

pytestmark = pytest.mark.gpu
built = P.built


@pytest.mark.parametrize("gate", [None, "row", "element"])
@pytest.mark.parametrize("checkpoints", [False, True])
def test_sandwich_networks_hold_no_matrix_for_plain_blocks(gate, checkpoints):
    """The matrices [n, width] of the activations' type that such a network holds: per block its stream, result and element gate
    (with checkpoints one of each that the blocks share), one more norm's input, the norms' outputs where they are not
    kept in 8 bits, and four gradients (dh, dy, dr, and an element gate's)."""
    n, width, blocks = 1000, 96, 2
    net, _ = P.network(n, width, 64, blocks, torch.bfloat16, sandwich=True, gate=gate, checkpoints=checkpoints)
    seen = {}

    def look(v):
        if isinstance(v, torch.Tensor):
            if v.dtype is torch.bfloat16 and v.shape == (n, width):
                seen[v.data_ptr()] = v
        elif isinstance(v, (list, tuple)):
            for x in v:
                look(x)
        elif isinstance(v, dict):
            look(list(v.values()))

    look(list(vars(net).values()))
    element = int(gate == "element")
    gradients = 3 + element
    kept = 2 + element if checkpoints else (blocks + 1) + blocks + blocks * element + (blocks + 1)
    assert len(seen) == gradients + kept


def dequantised(pair):
    return rs.fp8_dequantize(*pair)


@pytest.mark.parametrize("options", [dict()] + [dict(sandwich=True, gate=g) for g in (None, "row", "element")], ids=P.name_of)
@pytest.mark.parametrize("n,width,hidden", [(500, 160, 192), (777, 256, 130)])
def test_every_block_keeps_its_own(n, width, hidden, options):
    """Three blocks in float32.  Each block's checkpoints are, bit for bit, the 8-bit forms of what the network without
    checkpoints holds there (the float32 forwards are the same).  And the backward from them is, bit for bit, that of the other
    network from the values that they stand for: q times scale in float32 is what both read, in the same order of operations."""
    full, dcol = P.network(n, width, hidden, 3, **options)
    kept, _ = P.network(n, width, hidden, 3, checkpoints=True, **options)
    full.forward()
    assert torch.equal(full.colors, kept.forward())

    def form(t):
        q = rs.fp8_empty(*t.shape)
        rs.rs_quantize_fp8(t, *q)
        return q

    def same(pair, t):
        want = form(t)
        assert torch.equal(pair[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(pair[1], want[1])

    for b in range(4):
        same(kept.yq[b], full.y[b])
    for b in range(3):
        same(kept.uq[b], full.u[b])
        if full.sandwich:
            same(kept.kept[b]["x"], full.h[b])
            same(kept.kept[b]["r"], full.results[b])
            if options["gate"] == "element":
                same(kept.kept[b]["gate"], full.zs[b])
    first = full.h[0].clone()
    for b in range(4):
        full.y[b].copy_(dequantised(kept.yq[b]))
    for b in range(3):
        full.u[b].copy_(dequantised(kept.uq[b]))
        if full.sandwich:
            full.h[b].copy_(dequantised(kept.kept[b]["x"]))
            full.results[b].copy_(dequantised(kept.kept[b]["r"]))
            if options["gate"] == "element":
                full.zs[b].copy_(dequantised(kept.kept[b]["gate"]))
    norm_backward = full._norm_backward
    full._norm_backward = lambda b, x, *rest: norm_backward(b, first if b == 0 else x, *rest)
    full.backward(dcol)
    kept.backward(dcol)
    for (_, a), (_, b) in zip(full.parameters(), kept.parameters()):
        assert torch.equal(a, b) and float(a.abs().max()) > 0


@pytest.mark.parametrize("options", P.OPTIONS, ids=P.name_of)
@pytest.mark.parametrize("n,width,hidden", [(1, 64, 64), (70, 130, 64), (2, 129, 257)])
def test_stages_of_few_gaussians(n, width, hidden, options):
    P.test_stages(n, width, hidden, options)
