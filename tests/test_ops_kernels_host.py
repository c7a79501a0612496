"""Host-side checks of what the single operators' kernels compute about sizes (no GPU needed)."""
import pytest

from mlp_neural_shading_amd import binding as B

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
