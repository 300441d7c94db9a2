"""Training on answers where values that are no result could reach one:
padding, a neighbouring sequence, labels behind a group's end, rows at the end
of the range of counts; and the reference term near 0.  Bounds as in
test_gpu_answers.py, or beside the test."""
import math

import pytest
import torch

from autograd_arena_allocated_gb300 import api, synth
from test_gpu_answers import group_case, run_group_bwd, run_group_fwd
from test_gpu_head import DEV, TYPES, U, ctx, gen, make_logits  # noqa: F401 (ctx: a fixture)

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


@pytest.mark.parametrize("dtype,C,H", [("bf16", 128, 2), ("fp16", 64, 2), ("bf16", 64, 4), ("fp32", 64, 1)])
def test_the_next_group_moves_no_bit(ctx, dtype, C, H):
    """A group without padding, alone and in front of one whose queries its last tile loads."""
    T, starts = 200, [[140, 160, 200], [20, 100, 200]]
    qkv, st = group_case(dtype, starts, T, C, 27)
    qkv[T:] *= 30.0
    dy = torch.randn(2 * T, C, generator=gen(28), device=DEV).to(TYPES[dtype])
    out = []
    for n in (1, 2):
        y, lse = run_group_fwd(ctx, dtype, qkv[:n * T], st[:n].contiguous(), T, C, H)
        d = run_group_bwd(ctx, dtype, qkv[:n * T], st[:n].contiguous(), y, lse, dy[:n * T], T, C, H)
        out.append((y[:T], lse[0], d[:T]))
    for alone, beside in zip(*out):
        assert torch.equal(alone, beside)


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


def test_pairs_at_the_last_rows(ctx):
    """2^31 - 1 rows: answers that begin and end at the last of them, empty ones among them.  With two columns of
    equal logits every log probability is -ln 2, the gradient +-k / 2."""
    M, V = 2 ** 31 - 1, 2
    z = torch.zeros(M, V, dtype=torch.bfloat16, device=DEV)
    t = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    t[:5] = 0
    t[-300:] = 1
    spans = torch.tensor([[M - 300, M - 100], [M - 100, M], [0, 5], [M, M], [M, M], [M, M]], dtype=torch.int32, device=DEV)
    seq, pair, mean = torch.empty(6, device=DEV), torch.empty(3, device=DEV), torch.empty(1, device=DEV)
    big = api.Context(20 * M + (1 << 20))
    big.preference("bf16", z, t, None, spans, z, seq, pair, mean, M, V, V, 3, 0.01, 0.0, 0.0, False, 1.0, 1.0)
    big.sync()
    big.close()
    ln2 = math.log(2.0)
    want = -ln2 * torch.tensor([200.0, 100.0, 5.0, 0.0, 0.0, 0.0])
    assert torch.allclose(seq.cpu(), want, rtol=1e-5, atol=0.0)  # sums of 200 at most, each term off by 4 u
    v = 0.01 * (want[0::2] - want[1::2])
    loss = torch.nn.functional.softplus(-v)
    assert torch.allclose(pair.cpu(), loss, rtol=1e-5) and abs(float(mean) - float(loss.mean())) < 1e-5
    k = 0.01 * torch.sigmoid(-v)  # -d loss / d S of the preferred answer
    half = lambda x: torch.tensor([0.5 * x, -0.5 * x]).bfloat16().double()  # noqa: E731
    for rows, sign, hot in ((slice(M - 300, M - 100), -k[0], 1), (slice(M - 100, M), k[0], 1), (slice(0, 5), -k[1], 0)):
        g = z[rows].cpu().double()
        w = half(float(sign)) if hot == 0 else half(float(sign)).flip(0)
        assert bool(((g - w).abs() <= 2 ** -7 * w.abs()).all())  # a step of bf16
    assert not z[5:M - 300].any()
    del z, t
    torch.cuda.empty_cache()


@pytest.mark.parametrize("V", [65, 3000])
def test_reference_term_near_zero(ctx, V):
    """beta (e^x - x - 1) alone (no advantage, beta 1), x = ref - lp from a unit in lp's last place to 3.  x is the
    same fp32 difference here and there, and the product with beta adds to 0, so what is left is the term's own
    error.  Up to |x| = 1/2 a series: its sum 2 u (later terms are below a third of the first), the square and the
    product u each, what is left out below u / 10, the last rounding u; 8 u with room.  Beyond: e^x - 1 off by a unit in
    the last place, 2 u |e^x - 1|, and two roundings of the term."""
    M = 4000
    z = make_logits("fp32", M, V, V, 61)
    t = torch.randint(0, V, (M,), generator=gen(62), device=DEV).int()
    zero, row = torch.zeros(M, device=DEV), torch.empty(M, device=DEV)

    def go(ref):
        lp = torch.empty(M, device=DEV)
        ctx.reset()
        ctx.policy("fp32", z, t, None, ref, zero, None, None, lp, row, None, M, V, V, 0.2, 0.2, 1.0, 1.0, 1.0)
        ctx.sync()
        return lp

    lp = go(zero)
    size = 10.0 ** (-6.5 + 7.0 * torch.rand(M, generator=gen(63), device=DEV))
    ref = lp + torch.where(torch.rand(M, generator=gen(64), device=DEV) < 0.5, size, -size)
    assert torch.equal(go(ref), lp)
    x = (ref - lp).double()
    assert int((x.abs() < 1e-5).sum()) > 300
    # in 64 bits e^x - 1 - x is off by 2^-53 |x|, below 2^-31 of the term from |x| = 2e-7 on
    want = torch.where(x.abs() < 1e-3, x * x * (0.5 + x * (1 / 6 + x * (1 / 24 + x / 120))), torch.expm1(x) - x)
    bound = torch.where(x.abs() <= 0.5, 8 * U * want, 2 * U * torch.expm1(x).abs() + 4 * U * want)
    got = row.double()
    assert bool((got >= 0).all())
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / want)[x != 0].max())


@pytest.mark.parametrize("name,dtype", [("tiny_fp32", "fp32"), ("char_bf16", "bf16"), ("tiny_fp32", "fp16")])
def test_labels_behind_a_groups_end_are_reported(name, dtype):
    """Padding has no embedding and no gradient: a label there would be a wrong loss."""
    sh = synth.WORKLOADS[name].shape
    p = synth.init_params(sh)
    B, T = 2, 32
    tok = torch.zeros(B, T, dtype=torch.int32, device=DEV)
    f = torch.ones(B * T, device=DEV)
    st = torch.tensor([[4, 12, 20], [0, 16, T]], dtype=torch.int32, device=DEV)
    spans = torch.tensor([[4, 12], [12, 20]], dtype=torch.int32, device=DEV)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, dtype)
    with api.Context(api.answers_arena_bytes(cfg, B, T, 2)) as c:
        c.set_model(cfg)
        ws = torch.from_numpy(p).to(DEV).to(TYPES[dtype])
        g, out = torch.empty(p.size, device=DEV), torch.empty(B * T, device=DEV)
        calls = [lambda tgt, s: c.step_policy(ws, g, tok, tgt, None, None, f, None, 0.2, 0.2, 0.0, B=B, T=T, starts=s, K=2),
                 lambda tgt, s: c.step_preference(ws, g, tok, tgt, None, spans, 1, 0.1, B=B, T=T, starts=s, K=2),
                 lambda tgt, s: (c.logprobs_of(ws, tok, tgt, B, T, out, starts=s, K=2), c.sync())]
        tgt = torch.full((B, T), -1, dtype=torch.int32)
        tgt[0, 4:20] = 1
        tgt[1, T - 1] = 2
        for call in calls:
            for host in (True, False):
                x = tgt if host else tgt.to(DEV)
                c.reset()
                call(x, st)  # the last position of a group without padding may have one
                for at in (20, T - 1):
                    bad = tgt.clone()
                    bad[0, at] = 0
                    c.reset()
                    with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                        call(bad if host else bad.to(DEV), st)
                    c.reset()
                    call(bad if host else bad.to(DEV), None)  # without groups it is a label like others


def test_profile_counts_no_products_of_groups(ctx):
    """How many pairs of positions a group has is in device memory: its calls count bytes only."""
    T, C, H = 100, 64, 1
    qkv, st = group_case("bf16", [[20, 60, 100]], T, C, 71)
    y, lse = run_group_fwd(ctx, "bf16", qkv, st, T, C, H)
    d = torch.empty_like(qkv)
    ctx.set_profiling(True)
    try:
        ctx.group_attention_fwd("bf16", qkv, st, y, lse, 1, T, C, H, 2)
        ctx.group_attention_bwd("bf16", qkv, st, y, lse, y, d, 1, T, C, H, 2)
        rows = ctx.profile()
        assert set(rows) == {"attn_fwd", "attn_bwd"}  # with the statistics, 4 bytes a row and head
        assert all(r["flops"] == 0.0 and r["calls"] == 1 for r in rows.values())
        assert rows["attn_fwd"]["bytes"] == 4 * T * C * 2 + 4 * T and rows["attn_bwd"]["bytes"] == 8 * T * C * 2 + 4 * T
        ctx.attention_fwd("bf16", qkv, y, lse, 1, T, C, H)
        assert ctx.profile()["attn_fwd"]["flops"] > 0.0
    finally:
        ctx.set_profiling(False)
