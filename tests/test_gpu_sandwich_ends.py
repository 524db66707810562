"""The sandwich norm where its operands come to an end: no rows."""
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
