"""What the 8-bit cache's Python entry points refuse, on the host: each check comes before the library is called."""
import pytest
import torch

import token_level_dynamic_seq_b200 as logo


def step(n, gate, selected=None, B=2):
    c = logo.cache8(B, 2, 200, 64, "cpu")
    q = torch.zeros(B, 2, n, 64, dtype=torch.bfloat16)
    return logo.decode8(q, c, torch.zeros(B, dtype=torch.int32), gate, torch.zeros(1), 16, selected=selected)


@pytest.mark.parametrize("n,shape", [(1, (2, 4)), (1, (4,)), (1, (8,)), (1, (1, 2)), (3, (3, 2)), (3, (6,)), (3, (2, 4)),
                                     (3, (2,)), (2, (2, 1)), (2, (2, 2, 1)), (1, ())])
def test_gates_and_flags_of_another_shape(n, shape):
    """A buffer of four gates a sequence with a step of one token, gates the other way round."""
    with pytest.raises(ValueError, match="gate"):
        step(n, torch.zeros(shape))
    with pytest.raises(ValueError, match="selected"):
        step(n, torch.zeros(2, n), torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("n,shape", [(1, (2, 1)), (1, (2,)), (3, (2, 3))])
def test_gates_of_the_right_shape_get_past(n, shape):
    with pytest.raises(ValueError, match="CUDA"):     # the cache lies on the host
        step(n, torch.zeros(shape), torch.zeros(shape, dtype=torch.int32))


def test_more_blocks_than_a_grid_takes():
    """2^20 pairs of a sequence and a head times 2^11 blocks and more: refused as unsupported, nothing is launched."""
    import ctypes

    lib = logo.load_library()
    at = ctypes.c_void_p(1 << 20)
    for block, longest in ((64, 1 << 16), (128, 1 << 17), (128, 1 << 20)):
        c = logo.Cache8Desc(1 << 14, 1 << 6, 1 << 20, 64, block, 1, *[1 << 20] * 6)
        rows = logo.Shape(1, 64, 64, 1 << 20, 64, 0x1000, 1 << 14, longest)
        assert lib.logo_cache8_append(ctypes.byref(c), at, at, rows, at, None, at, 256, None) == 2
        assert "blocks" in lib.logo_last_error().decode()
        assert lib.logo_cache8_read(ctypes.byref(c), at, rows, at, at, at, 256, None) == 2


def test_workspace_of_a_cache_that_is_not_on_the_current_device(monkeypatch):
    """The workspace is cleared on the current device's stream: for a cache elsewhere that would be in no order with the
    calls that use it."""
    with pytest.raises(ValueError, match="CUDA"):
        logo.decode8_workspace(logo.cache8(2, 2, 200, 64, "cpu"), 2)
    other = logo.cache8(2, 2, 200, 64, "cpu")
    other.index = 7                                    # as a cache on another device says
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        logo.decode8_workspace(other, 2)


@pytest.mark.parametrize("shape", [(2,), (0,), (2, 1)])
def test_more_than_one_threshold(shape):
    """One threshold serves the batch: of several the first would be taken for all."""
    c = logo.cache8(2, 2, 200, 64, "cpu")
    with pytest.raises(ValueError, match="tau"):
        logo.decode8(torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16), c, torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1),
                     torch.zeros(shape), 16)
