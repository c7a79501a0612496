"""GPU tests of the single operators' kernels one by one, at what each has of its own: its tiles' borders, the
strides and the aliases that its epilogue allows, its activations."""
import pytest
import torch

from gpu_util import device, log
from mlp_neural_shading_amd import ops

pytestmark = pytest.mark.gpu


def test_the_last_slots_of_2_to_the_31():
    """As many slots as there can be, for the kernel with the largest tiles: the last one ends at 2^31 - 1."""
    n, t = 2 ** 31 - 1, torch.float16
    log("2^31 - 1 slots")
    x = torch.empty(n, 1, dtype=t, device=device())
    for i in range(0, n, 1 << 28):
        x[i:i + (1 << 28), 0] = (torch.arange(min(1 << 28, n - i), device=device()) % 61).to(t)
    w = torch.tensor([3.0, 5.0], dtype=t, device=device()).view(2, 1, 1)
    last = 1000
    offsets = torch.tensor([0, n - last, n], dtype=torch.int32, device=device())
    unused = torch.empty(n, dtype=torch.int32, device=device())  # slots and places: x is by slot, nothing is combined
    y = torch.full((n, 1), -1.0, dtype=t, device=device())
    ops.expert_linear(x, w, ops.Dispatch(offsets, unused, unused), k=1, rows="slots", out=y)
    for i in range(0, n, 1 << 28):
        part = slice(i, min(i + (1 << 28), n - last))
        assert torch.equal(y[part], x[part] * 3)
    assert torch.equal(y[-last:], x[-last:] * 5)
