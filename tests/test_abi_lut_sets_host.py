"""Workspace and path of the checkpoint's LUT gradient with many LUT sets (no GPU
needed: sizes only)."""
import pytest

pytest.importorskip("torch")

from compressive_fine_tuning_b200 import sk  # noqa: E402

PART = 512 << 20                  # room of the partial bins


def _size(n, d, bits, gpr, T, sets):
    return sk.workspace_bytes(sk.SK_OP_BWD_LUT_CKPT8, n, d, bits, gpr, T, sets)


@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("n,d,gpr", [(11008, 4096, 8), (11008, 4096, 1), (4096, 11008, 4), (8192, 5120, 5),
                                     (8192, 28672, 128), (64, 96, 3)])
@pytest.mark.parametrize("T", [300, 8192])
def test_workspace_is_bounded_whatever_the_sets(n, d, gpr, bits, T):
    for sets in (1, 2, 8, 64, 200, 256):
        tiles = (d + 255) // 256
        slots = min(255 // (d // gpr) + 2, gpr)
        one = tiles * n * slots * (1 << bits) * 4
        rows = T + (sets * 63 if sets > 1 else 0)
        routed = rows * 4 + sets * 8 + rows * n * 2 if sets > 1 else 0
        # X as bf16, a part of one round's tiles (74 of 256 rows), and each array's padding
        most = rows * d * 2 + routed + max(PART, one) + 74 * 256 * slots * (1 << bits) * 4 + 8 * 256
        assert rows * d * 2 <= _size(n, d, bits, gpr, T, sets) <= most, sets


@pytest.mark.parametrize("sets", [2, 3, 8, 10])
def test_few_sets_keep_the_tensor_cores(sets):
    for T in (5 + sets, 6 + sets):                      # a call without task ids is one for one set
        one = _size(4096, 4096, 4, 128, T, 1)
        size = _size(4096, 4096, 4, 128, T, sets)
        assert size > one if T >= 6 + sets else size == one


@pytest.mark.parametrize("n,d,gpr", [(11008, 4096, 8), (4096, 4096, 1)])
@pytest.mark.parametrize("sets", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 16, 19])
def test_few_tokens_of_many_sets_need_no_room_for_the_sets(n, d, gpr, sets, T):
    """Every set costs the tensor cores n d bins, the CUDA cores only the named ones."""
    assert _size(n, d, 4, gpr, T, sets) == _size(n, d, 4, gpr, T, 1)
    assert _size(n, d, 4, gpr, 2 * sets, sets) > _size(n, d, 4, gpr, 2 * sets, 1) > 0
