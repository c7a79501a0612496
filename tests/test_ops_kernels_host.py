"""Host-side checks of what the single operators' kernels compute about sizes (no GPU needed)."""
import pytest
import torch
import torch.autograd.forward_ad as fa

import ops_kernels as K
from mlp_neural_shading_amd import binding as B
from mlp_neural_shading_amd import ops

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("begin,end", [(0, 1), (0, 512), (0, 513), (7, 1031), (MOST - 1, MOST), (MOST - 512, MOST), (MOST - 513, MOST),
                                       (MOST - 2000, MOST - 3), (5, MOST), (0, MOST)])
@pytest.mark.parametrize("size", [16, 64, 128, 256, 512])
def test_tiles_cover_an_experts_slots_once(begin, end, size):
    """Up to the last slot there can be: row0 + size passes 2^31 in the last tiles."""
    tiles = (end - begin + size - 1) // size
    shown = range(tiles) if tiles < 100 else (0, 1, tiles // 2, tiles - 2, tiles - 1)
    for t in shown:
        assert B.mlp_testing_expert_tile(begin, end, size, t) == (begin + t * size, min(begin + (t + 1) * size, end))
    for t in (-1, tiles):
        with pytest.raises(B.MlpError, match="tile"):
            B.mlp_testing_expert_tile(begin, end, size, t)


# The kernels of the products and a size of each; tests/test_gpu_ops_kernels.py runs these.
LINEAR = {"few": (70, 100, 60, False), "few wide": (300, 72, 700, False), "small": (601, 136, 699, False),
          "mid": (1501, 200, 1303, False), "big": (5001, 200, 1801, False), "tile": (9001, 72, 63, False),
          "narrow": (524301, 24, 20, False)}
GATED = {"few wide": (100, 72, 40, True), "small": (600, 136, 351, True), "mid": (1301, 200, 1099, True),
         "big": (2601, 264, 1700, True), "tile": (8200, 72, 32, True), "narrow": (524289, 33, 15, True)}
EXPERTS = {"few": (37, 3, 5, 200, 130, False), "small": (900, 2, 5, 136, 700, False), "mid": (3000, 2, 4, 72, 1201, False),
           "big": (3000, 2, 4, 72, 1200, True), "tile": (700, 2, 6, 33, 300, False), "narrow": (530000, 1, 5, 40, 12, False),
           "few wide": (200, 2, 6, 64, 200, True)}


@pytest.mark.parametrize("gated", [False, True])
def test_layers_that_take_each_kernel(gated):
    for name, size in (GATED if gated else LINEAR).items():
        assert K.linear_kernel(*size) == name, size
    assert not gated or set(GATED) | {"few"} == set(LINEAR)


def test_experts_that_take_each_kernel():
    assert set(EXPERTS) == set(LINEAR)
    for name, size in EXPERTS.items():
        assert K.expert_kernel(*size) == name, size


def test_kernels_for_rows_at_odd_elements():
    """Only `tile` and the few-row and narrow kernels take rows that are not 4-byte aligned."""
    size = LINEAR["big"]
    for over in (dict(ldx=201), dict(ldw=203), dict(x=K.FAR + 2), dict(w=2 * K.FAR + 2)):
        assert K.linear_kernel(*size, **over) == "tile", over
    assert K.linear_kernel(*size, ldx=206, ldw=202, x=K.FAR + 4, w=2 * K.FAR + 12) == "big"
    assert K.expert_kernel(*EXPERTS["mid"], w_stride=72 * 1201 + 1) == "tile"


def test_router_layouts():
    """By experts and k; with groups, by the lanes that each takes: a power of two."""
    for experts, k, name in ((1, 1, "lanes 16x4"), (64, 15, "lanes 16x4"), (64, 16, "lanes 64x8"), (65, 8, "lanes 16x8"),
                             (128, 15, "lanes 16x8"), (129, 8, "lanes 16x16"), (256, 15, "lanes 16x16"), (256, 16, "lanes 64x8"),
                             (257, 1, "lanes 64x8"), (512, 32, "lanes 64x8"), (513, 1, "wave"), (1024, 32, "wave")):
        assert K.route_kernel(experts, k) == name, (experts, k)
    for experts, groups, name in ((64, 8, "lanes 16x4"), (256, 8, "lanes 16x16"), (160, 8, "lanes 16x16"), (512, 16, "lanes 64x8"),
                                  (96, 96, "wave"), (640, 8, "wave"), (12, 6, "lanes 16x4")):
        assert K.route_kernel(experts, 2, groups, groups // 2) == name, (experts, groups)


def test_kernel_names_are_checked_calls():
    assert K.linear_kernel(0, 8, 8) == "none"
    assert K.expert_kernel(0, 2, 4, 8, 8) == "none"
    for call in (lambda: K.linear_kernel(4, 0, 8), lambda: K.linear_kernel(4, 8, 8, ldx=7), lambda: K.expert_kernel(4, 2, 0, 8, 8),
                 lambda: K.route_kernel(8, 9)):
        with pytest.raises(B.MlpError):
            call()


def test_forward_mode_duals_are_refused():
    """A dual tensor does not require a gradient, and its tangent would be lost."""
    x, t = torch.ones(4, 8, dtype=torch.float16), torch.ones(4, 8, dtype=torch.float16)
    with fa.dual_level():
        dual = fa.make_dual(x, t)
        for call in (lambda v: ops.linear(v, v), lambda v: ops.route(v, 2), lambda v: ops.expert_linear(v, v[None], None, k=2)):
            with pytest.raises(ValueError, match="tangent"):
                call(dual)
            with pytest.raises(ValueError, match="on the GPU"):
                call(x)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                call(dual)


def test_counts_are_whole_numbers():
    """2.5 experts per token are not 2."""
    x, index = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 2, dtype=torch.int32)
    for bad in (2.5, 2.0, "2", None, torch.tensor([1, 2])):
        for call in (lambda: ops.route(x, bad), lambda: ops.dispatch(index, bad), lambda: ops.expert_linear(x, x[None], None, k=bad)):
            with pytest.raises(ValueError, match="whole number"):
                call()
    for good in (2, torch.tensor(2), True):
        with pytest.raises(ValueError, match="on the GPU"):
            ops.route(x, good)


def test_one_experts_stride_means_nothing():
    """It decides no kernel: an odd one does not make the rows odd."""
    for w_stride in (0, 7, -1, 2 ** 40 + 1):
        assert K.expert_kernel(3000, 2, 1, 72, 1200, w_stride=w_stride) == "mid"
