"""Training on answers where values that are no result could reach one:
padding, a neighbouring sequence, labels behind a group's end, rows at the end
of the range of counts; and the reference term near 0.  Bounds as in
test_gpu_answers.py, or beside the test."""
import math

import pytest
import torch

from autograd_arena_allocated_gb300 import api
from test_gpu_answers import group_case, run_group_bwd, run_group_fwd
from test_gpu_head import DEV, TYPES, ctx, gen, make_logits  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,C,H", [("bf16", 128, 2), ("fp16", 128, 2), ("bf16", 64, 2), ("fp16", 64, 4), ("fp32", 128, 2)])
def test_padding_moves_no_bit_of_a_group(ctx, dtype, C, H):
    """Padded queries with scores far above every other, in the rows behind an answer's end and in the next
    sequence's: a softmax that takes a new reference for them would round the positions beside them otherwise."""
    T, starts = 260, [[150, 170, 200], [140, 140, 205], [200, 230, 259]]
    qkv, st = group_case(dtype, starts, T, C, 7, pad=0.0)
    dy = torch.randn(len(starts) * T, C, generator=gen(8), device=DEV).to(TYPES[dtype])
    y, lse = run_group_fwd(ctx, dtype, qkv, st, T, C, H)
    d = run_group_bwd(ctx, dtype, qkv, st, y, lse, dy, T, C, H)
    for b, s in enumerate(starts):
        rows = qkv.view(len(starts), T, 3 * C)[b, s[-1]:]
        rows.copy_(30.0 * torch.randn(rows.shape, generator=gen(9 + b), device=DEV))
    y2, lse2 = run_group_fwd(ctx, dtype, qkv, st, T, C, H)
    assert torch.equal(y2, y) and torch.equal(lse2, lse)
    assert torch.equal(run_group_bwd(ctx, dtype, qkv, st, y2, lse2, dy, T, C, H), d)


@pytest.mark.parametrize("T", [70, 200, 300])
def test_the_next_sequence_moves_no_bit_of_causal_attention(ctx, T):
    """A tile that runs past its sequence's end loads the next one's queries."""
    B, C, H = 2, 128, 2
    qkv = torch.randn(B, T, 3 * C, generator=gen(17), device=DEV).bfloat16()
    qkv[1] *= 30.0
    dy = torch.randn(B, T, C, generator=gen(18), device=DEV).bfloat16()
    out = []
    for n in (1, 2):
        y = torch.empty(n * T, C, device=DEV, dtype=torch.bfloat16)
        lse, d = torch.empty(n, H, T, device=DEV), torch.empty(n * T, 3 * C, device=DEV, dtype=torch.bfloat16)
        ctx.reset()
        ctx.attention_fwd("bf16", qkv[:n].contiguous(), y, lse, n, T, C, H)
        ctx.attention_bwd("bf16", qkv[:n].contiguous(), y, lse, dy[:n].contiguous(), d, n, T, C, H)
        ctx.sync()
        out.append((y[:T], lse[0], d[:T]))
    for alone, beside in zip(*out):
        assert torch.equal(alone, beside)
