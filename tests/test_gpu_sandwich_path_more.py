"""What the wide network's blocks keep: nothing that nobody reads."""
import pytest
import torch

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
