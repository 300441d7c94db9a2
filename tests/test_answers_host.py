"""Host-side checks of the calls on answers, without a GPU: NULL and missing
contexts, and the arena plan."""
import pytest

from autograd_arena_allocated_gb300 import _native, api
from autograd_arena_allocated_gb300 import build as native_build


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return _native.lib()


def test_null_context_is_refused(lib):
    n = None
    assert lib.tt_op_logprobs(n, 0, n, n, n, n, 1, 1, 1, 1.0) == -2
    assert lib.tt_op_policy(n, 0, n, n, n, n, n, n, n, n, n, n, 1, 1, 1, 0.2, 0.2, 0.0, 1.0, 1.0) == -2
    assert lib.tt_op_preference(n, 0, n, n, n, n, n, n, n, n, 1, 1, 1, 1, 0.1, 0.0, 0.0, 0, 1.0, 1.0) == -2
    assert lib.tt_op_group_attention_fwd(n, 0, n, n, n, n, 1, 1, 64, 1, 1) == -2
    assert lib.tt_op_group_attention_bwd(n, 0, n, n, n, n, n, n, 1, 1, 64, 1, 1) == -2
    assert lib.tt_gpt2_logprobs(n, n, n, n, n, 0, 1, 1, 1.0, n, n) == -2
    assert lib.tt_gpt2_step_policy(n, n, n, n, n, n, n, n, n, 0.2, 0.2, 0.0, 1.0, n, 0, 1, 1, 0, n, n, n) == -2
    assert lib.tt_gpt2_step_preference(n, n, n, n, n, n, n, 1, 0.1, 0.0, 0.0, 0, 1.0, n, 0, 1, 1, 0, n, n, n) == -2


def test_answers_arena_plan(lib):
    cfg = api.make_config(12, 768, 12, 50257, 1024, "bf16")
    plain = api.arena_bytes(cfg, 8, 1024)
    assert plain < api.answers_arena_bytes(cfg, 8, 1024) <= plain + 20 * 8 * 1024 + 1024
    # groups may be longer than the position table: 8 groups of 2048 are 16 sequences' work
    assert api.arena_bytes(cfg, 8, 2048) == 0 and api.answers_arena_bytes(cfg, 8, 2048) == 0
    grouped = api.answers_arena_bytes(cfg, 8, 2048, 4)
    assert 0.9 * api.arena_bytes(cfg, 16, 1024) < grouped < 1.1 * api.arena_bytes(cfg, 16, 1024)
    for bad in [(0, 64, 2), (2, 0, 2), (2, 64, -1), (1 << 20, 1 << 12, 2), (1, 65535 * 64 + 1, 1)]:
        assert api.answers_arena_bytes(cfg, *bad) == 0, bad
