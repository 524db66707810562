"""The wide network's options that the constructor refuses (CPU only)."""
import pytest
import torch

from gaussian_splatting_tile_gb300 import pipeline


@pytest.mark.parametrize("options", [dict(gate="row"), dict(gate="element", checkpoints=True), dict(sandwich=True, gate="column"),
                                     dict(blocks=5, sandwich=True), dict(blocks=5, checkpoints=True)])
def test_refused(options):
    with pytest.raises(ValueError):
        pipeline.WideAppearance(torch.zeros(4, 8), 8, **options)
