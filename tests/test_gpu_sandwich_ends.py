"""The sandwich norm where its operands come to an end: no rows, gates that are shut or wide open, kept in 8 bits.
Tolerances are those of test_gpu_sandwich."""
import math

import pytest
import torch

from gaussian_splatting_tile_gb300 import pipeline, rs

from . import test_gpu_sandwich as S

pytestmark = pytest.mark.gpu
built = S.built


@pytest.mark.parametrize("gate", ["none", "row", "element"])
def test_no_rows_of_checkpoints(gate):
    """Nothing to do, but the vectors' gradients become zero."""
    c = 300
    w, none = torch.ones(c, device="cuda"), torch.empty(0, device="cuda")
    e = torch.empty(0, c, dtype=torch.bfloat16, device="cuda")
    kept = [rs.fp8_empty(0, c) for _ in range(3)]
    z = {"none": None, "row": e[:, :1], "element": e}[gate]
    rs.rs_sandwich_norm_fwd(e, e, w, w, *rs.fp8_empty(0, c), gate=z, kept_x=kept[0], kept_r=kept[1],
                            kept_gate=kept[2] if gate == "element" else None)
    d = [torch.full((c,), 7.0, device="cuda") for _ in range(3)]
    rs.rs_sandwich_norm_bwd(kept[0], kept[1], w, w, none, none, e, e, e, None, gate=kept[2] if gate == "element" else z,
                            dL_dgate=None if z is None else torch.empty_like(z), dL_dpost_weight=d[0], dL_dpre_weight=d[1],
                            dL_dresidual_scale=d[2])
    assert all(bool((t == 0).all()) for t in d)
    x = torch.empty(2, c, dtype=torch.bfloat16, device="cuda")  # with rows, scales that are missing still are
    with pytest.raises(ValueError):
        rs.rs_sandwich_norm_bwd((rs.fp8_empty(2, c)[0], None), rs.fp8_empty(2, c), w, w, w, w, x, x, x.clone(), None)


@pytest.mark.parametrize("options", [dict()] + [dict(sandwich=s, checkpoints=k, gate=g) for s in (False, True) for k in (False, True)
                                                for g in (None, "row", "element") if s or (k and g is None)], ids=str)
def test_networks_of_no_gaussians(options):
    net = pipeline.WideAppearance(torch.empty(0, 96, device="cuda"), 64, 2, **options)
    net.forward()
    net.backward(torch.empty(3, 0, device="cuda"))
    net.step(max_norm=1.0)
    for p, g in net.parameters():
        assert bool((g == 0).all()) and bool(torch.isfinite(p).all())
    assert float(net.norm) == 0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [300, 301, 512, 4200])
def test_gates_at_the_ends_from_checkpoints(dt, cols):
    """A gate beyond 80 either way is as good as shut or open and is kept as 80, so that neither an infinity nor a type's lowest
    value takes the other gates of its block of 128 along."""
    g = S.gen(cols)
    b = S.Block(g, 12, cols, dt)
    low, high = torch.finfo(S.DT[dt]).min, torch.finfo(S.DT[dt]).max
    b.gate[1], b.gate[2], b.gate[3] = -math.inf, math.inf, low
    b.gate[4, 7], b.gate[5, 130], b.gate[6, 299] = -math.inf, math.inf, low
    b.gate[7, ::2], b.gate[8, 5], b.gate[9, 5], b.gate[9, 6] = high, 79.5, 80, -80.5
    b.gate[10, 3], b.gate[10, 4] = 1000, -1000
    o = b.forward(kept=True)
    held = b.gate.clamp(-80, 80)
    want = rs.fp8_empty(b.rows, cols)
    rs.rs_quantize_fp8(held, *want)
    assert torch.equal(o["kept_gate"][0].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(o["kept_gate"][1], want[1])
    z = b.gate
    S.keep(b, o)
    back = rs.fp8_dequantize(*b.gate)
    # a block's largest gate comes back to two roundings of its scale, the others to half an e4m3 step
    assert bool(((back - held.float()).abs() <= held.float().abs() / 16 * (1 + 2 ** -20) + 80 / 448 * 2.0 ** -10).all())
    dy, dsum = S.grads_of(g, b)
    got = S.check_backward(b, o, dy, dsum)
    assert all(bool(torch.isfinite(t.float()).all()) for t in got)
    shut = (z < -80).float()
    assert bool((got[2].float() * shut).abs().max() < 1e-28)


def test_a_gate_that_is_no_number_stays_one():
    g = S.gen(11)
    b = S.Block(g, 3, 300, "bf16")
    b.gate[1, 5] = math.nan
    o = b.forward(kept=True)
    z = rs.fp8_dequantize(*o["kept_gate"])
    assert int(torch.isnan(z).sum()) == 1 and math.isnan(float(z[1, 5]))
