"""Host-side checks of the list operators' C ABI, without a GPU: NULL and
missing contexts, and the beam search's exact arena plan."""
import ctypes as C

import pytest

from autograd_arena_allocated_gb300 import _native, api
from autograd_arena_allocated_gb300 import build as native_build


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return _native.lib()


def test_null_context_is_refused(lib):
    assert lib.tt_op_top_logits(None, 0, None, None, None, None, 1, 1, 1, 1, 1.0) == -2
    assert lib.tt_op_distill(None, 0, None, None, None, None, None, None, None, None, 1, 1, 1, 1, 1.0, 1.0, 1.0) == -2
    assert lib.tt_op_beam_select(None, 0, None, None, None, None, None, None, None, 1, 1, 1, 1, 1, -1) == -2
    assert lib.tt_op_beam_reorder(None, None, None, 1, 1, 1, 1, 0, 1) == -2
    assert lib.tt_gpt2_step_distill(None, None, None, None, None, None, None, None, 1, 1.0, 1.0, 1, 1, 0, None, None) == -2
    assert lib.tt_gpt2_top_logits(None, None, None, 1, 1, 1, 1.0, None, None, None) == -2
    assert lib.tt_gpt2_generate_beam(None, None, None, 1, 1, 1, 1, -1, None, None) == -2


def test_beam_arena_plan(lib):
    cfg = api.make_config(12, 768, 12, 50257, 1024, "bf16")
    plans = [api.generate_beam_arena_bytes(cfg, 2, 64, 32, K) for K in (1, 4, 8)]
    assert 0 < plans[0] < plans[1] < plans[2]
    # eight beams hold eight caches
    assert plans[2] > 8 * 2 * 12 * 1024 * 2 * 768 * 2
    for bad in [(0, 64, 32, 4), (2, 0, 32, 4), (2, 64, -1, 4), (2, 64, 961, 4), (2, 64, 32, 0), (2, 64, 32, 33),
                (1 << 30, 64, 32, 4), (2, 2 ** 31 - 1, 2 ** 31 - 1, 4)]:
        assert api.generate_beam_arena_bytes(cfg, *bad) == 0, bad
    half = api.make_config(12, 768, 12, 50257, 1024, "fp16")
    assert api.generate_beam_arena_bytes(half, 2, 64, 32, 4) == 0
    small = api.make_config(2, 64, 4, 7, 32, "fp32")
    assert api.generate_beam_arena_bytes(small, 1, 4, 4, 7) > 0
    assert api.generate_beam_arena_bytes(small, 1, 4, 4, 8) == 0  # more beams than tokens
    assert lib.tt_gpt2_generate_beam_arena_bytes(C.byref(cfg), 1, 1, 0, 1) > 0
