"""Sizes at the edge of what the model's calls count, without a GPU."""
import pytest

from autograd_arena_allocated_gb300 import api
from autograd_arena_allocated_gb300 import build as native_build


@pytest.mark.parametrize("B", [1 << 21, 1 << 22, 2 ** 31 - 1])
def test_no_plan_for_more_positions_than_an_int_counts(B):
    """B T of 2^31, of 2^32 (0 in 32 bits) and beyond."""
    native_build.build()
    cfg = api.make_config(1, 64, 4, 65, 1024, "fp32")
    assert api.arena_bytes(cfg, B, 1024) == 0
    assert api.arena_bytes(cfg, 2, 1024) > 0
