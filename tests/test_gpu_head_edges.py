"""The list operators at the edges of their arithmetic: rows that mix two kinds
of mask, mass off the list that is tiny beside it, long sums, many rows.

The references are the definitions in 64 bits and in logarithms, so that no
term is lost to underflow, and every comparison asks for `error <= bound`: a
NaN on either side fails.

Tolerances of distillation, with u = 2^-24 (half a step of fp32):
 - p_j = exp(t_j / tau - base): the quotient, the difference and the product
   with log2 e are each off by half a step of at most |t_j| / tau + |base|, the
   exponential by two steps: (4 (|t_j| / tau + |base|) + 8) u relative;
 - p_r is 1 less their sum: off by the sum of their errors and 12 additions;
 - a student's probability is exp((z - R) / tau) over a sum: (3 |ln q| + depth +
   64) u relative, the numerator's argument, the sum (as in test_gpu_head.py)
   and the reference's rounding;
 - the gradient adds these and half a step of its storage type; the loss
   multiplies them by the logarithms that it weighs, which are themselves off
   by their own size in u and by the sum's relative error."""
import math

import pytest
import torch

import test_gpu_head as base
from autograd_arena_allocated_gb300 import api, synth
from test_gpu_head import DEPTH, DEV, INF, TYPES, U, ctx, gen, make_lists, make_logits  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.gpu
OFF_MIN = -700.0  # ln q_r below this counts as no mass off the list


def exact_distill(z, V, lists, targets, alpha, tau, rest):
    """Losses, d loss / d z and the bounds of their errors, in 64 bits."""
    vals, idx, lse = lists
    M = z.shape[0]
    x = z[:, :V].double()
    used = idx >= 0
    at = torch.where(used, idx, V).long()
    logq = torch.log_softmax(x / tau, 1)
    wide = torch.cat([logq, torch.zeros(M, 1, dtype=torch.float64, device=z.device)], 1)
    lq = wide.gather(1, at)
    t = torch.where(used, vals.double() / tau, -INF)
    norm = lse.double()[:, None] if rest else torch.logsumexp(t, 1, keepdim=True)
    some = used.any(1, keepdim=True)
    lp = torch.where(used, t - norm, -INF)
    p = torch.where(some, lp.exp(), 0.0)
    on = p > 0
    lp0, lq0 = torch.where(on, lp, 0.0), torch.where(on, lq, 0.0)
    arg = torch.where(on, t.abs() + norm.abs(), 0.0)
    dp = p * (4 * arg + 8) * U
    total = p.sum(1, keepdim=True)
    dpr = dp.sum(1, keepdim=True) + 12 * U * total.clamp(min=1.0)
    kl = (p * (lp0 - lq0)).sum(1)
    size = (dp * (lp0.abs() + lq0.abs() + 1) + p * (2 * arg + 4 * lq0.abs() + DEPTH + 64) * U).sum(1)
    listed = torch.zeros(M, V + 1, dtype=torch.bool, device=z.device).scatter_(1, at, True)[:, :V]
    off = torch.zeros_like(logq)
    pr = torch.zeros_like(total)
    if rest:
        lqr = torch.logsumexp(torch.where(listed, -INF, logq), 1, keepdim=True)
        pr = torch.where(some & (lqr >= OFF_MIN), (1 - total).clamp(min=0), 0.0)
        have = pr > 0
        lr = torch.where(have, lqr, 0.0)
        lpr = torch.where(have, pr, 1.0).log()
        kl = kl + (pr * (lpr - lr))[:, 0]
        ask = some & (lqr >= OFF_MIN)
        size = size + torch.where(ask, dpr * (torch.where(have, lpr.abs(), 17.0) + torch.where(ask, lqr, 0.0).abs() + 1)
                                  + pr * (2 * DEPTH + 64 + 4 * lr.abs()) * U, 0.0)[:, 0]
        off = torch.where(ask & ~listed, (logq - torch.where(ask, lqr, 0.0)).exp(), 0.0)
    q = logq.exp()
    W = total + pr
    spread = lambda v: torch.zeros(M, V + 1, dtype=torch.float64, device=z.device).scatter_add_(1, at, v)[:, :V]
    soft = torch.where(some, 1.0, 0.0) * alpha * tau
    rel = (2 * DEPTH + 64 + 3 * logq.abs().clamp(max=800.0)) * U
    grad = soft * (W * q - spread(p) - pr * off)
    bound = soft * (W * q * rel + dpr * q + spread(dp) + (dpr + pr * rel) * off)
    loss = torch.where(some[:, 0], alpha * tau * tau * kl, 0.0)
    lb = torch.where(some[:, 0], alpha * tau * tau * size, 0.0)
    if targets is not None and alpha < 1:
        y = targets.long()
        hard = (y >= 0)[:, None]
        ls = torch.log_softmax(x, 1)
        s = ls.exp()
        hot = torch.zeros_like(s).scatter_(1, y.clamp(min=0)[:, None], 1.0)
        ce = -ls.gather(1, y.clamp(min=0)[:, None])[:, 0]
        grad = grad + torch.where(hard, (1 - alpha) * (s - hot), 0.0)
        bound = bound + torch.where(hard, (1 - alpha) * (s * (2 * DEPTH + 64 + 3 * ls.abs().clamp(max=800.0)) + 2 * hot) * U, 0.0)
        loss = loss + torch.where(hard[:, 0], (1 - alpha) * ce, 0.0)
        lb = lb + torch.where(hard[:, 0], (1 - alpha) * (DEPTH + 64 + 4 * (ce.abs() + 30)) * U, 0.0)
    return loss, lb + 4 * U * loss.abs(), grad, bound


def within(got, want, bound, what):
    ok = (got - want).abs() <= bound
    assert bool(torch.isfinite(want).all()) and bool(torch.isfinite(got).all()), what
    assert bool(ok.all()), (what, int((~ok).sum()), ok.shape, float(((got - want).abs() / bound)[~ok].max()))


def check_strict(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=None):
    dscale = 1.0 / z.shape[0] if dscale is None else dscale
    row, mean, d = base.run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=dscale)
    loss, lb, grad, gb = exact_distill(z, V, lists, targets, alpha, tau, rest)
    within(row.double(), loss, lb, "loss")
    f = torch.finfo(TYPES[dtype])
    within(d[:, :V].double(), grad * dscale,
           f.eps / 2 * 1.001 * (grad * dscale).abs() + gb * abs(dscale) + f.smallest_normal * f.eps / 2 + 1e-37, "gradient")
    assert bool((d[:, V:] == 0).all())
    in_place = base.run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=dscale, in_place=True)
    assert torch.equal(in_place[0], row) and torch.equal(in_place[2], d)
    only = base.run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=dscale, grad=False)
    assert torch.equal(only[0], row)
    return row, mean, d


# ---------------------------------------------------------------- two kinds of mask
def mixed_masks(dtype, V, ld, extra=0):
    """Eight rows whose columns are -inf here and the type's lowest value (or
    half of it) there, with a few real logits or none; -> z, the real columns
    (the rows that have none: columns of their largest value)."""
    low = torch.finfo(TYPES[dtype]).min
    cut = min(V // 2, 6000)
    z = make_logits(dtype, 8, V, ld, 33 + V, extra, pad=math.nan)
    z[:, :cut] = -INF
    z[:, cut:V] = low
    at = [torch.linspace(cut + 3, V - 2, 6).long().tolist() for _ in range(8)]
    z[1, at[1][:3]] = torch.tensor([-100.0, -101.0, -100.5], device=DEV).to(z.dtype)
    z[2, :V] = low
    z[2, cut:V] = -INF
    at[2] = torch.linspace(1, cut - 2, 6).long().tolist()
    z[2, at[2][:3]] = torch.tensor([-200.0, -201.0, -200.5], device=DEV).to(z.dtype)
    z[3, :V] = -INF
    z[3, V - 40:V] = low
    z[3, V - 7] = -1000.0
    at[3] = [V - 7]
    blocks = (torch.arange(V, device=DEV) // 64) % 2 == 0
    z[4, :V] = torch.where(blocks, -INF, low).to(z.dtype)
    z[4, V // 3] = 5.0
    at[4] = [V // 3]
    z[5, cut:V] = low / 2
    z[5, cut:cut + 5] = low
    at[5] = [c for c in at[5] if c >= cut + 5]
    z[6, :V] = -INF
    z[6, V - 9:V] = low
    at[6] = [V - 9, V - 1]
    z[7, V // 2:V] = -INF
    z[7, cut:V // 2 + 1] = low
    at[7] = [cut] if V // 2 == cut else [cut, V // 2]
    return z, at


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(100, 1), (700, 1), (6000, 1), (6000, 600), (50257, 1), (50257, 500)])
def test_top_logits_of_two_kinds_of_mask(ctx, dtype, V, copies):
    """A grammar's -inf and a library's lowest value in one row."""
    z, _ = mixed_masks(dtype, V, V + 3)
    z = z.repeat(copies, 1)
    for tau in (1.0, 2.5):
        base.check_top(ctx, dtype, z, V, 12, tau=tau)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [700, 6000, 50257])
def test_beam_select_of_two_kinds_of_mask(ctx, dtype, V):
    z, _ = mixed_masks(dtype, V, V)
    scores = torch.tensor([[-2.0, -1.0, -3.0, -4.0], [-2.5, -1.5, -0.5, -3.5]], device=DEV)
    base.check_select(ctx, dtype, z, scores, None, 4, V, 4, -1)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(100, 1), (700, 1), (6000, 1), (6000, 50), (50257, 1), (50257, 40), (60001, 20)])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_of_two_kinds_of_mask(ctx, dtype, V, copies, rest):
    z, at = mixed_masks(dtype, V, V + 1)
    k = 4
    vals, idx, lse = make_lists(8, V, k, 7, unused=False)
    y = torch.empty(8, dtype=torch.int32, device=DEV)
    for r in range(8):
        c = at[r]
        idx[r] = torch.tensor((c[:2] + [-1] * k)[:k])
        y[r] = c[-1] if r in (0, 5, 6, 7) else c[0] if r % 2 else c[:3][-1]
    lists = tuple(x.repeat(copies, *([1] * (x.dim() - 1))) for x in (vals, idx, lse))
    for alpha in (0.5, 1.0):
        check_strict(ctx, dtype, z.repeat(copies, 1), V, lists, y.repeat(copies), alpha, 2.0, rest)


# ---------------------------------------------------------------- little mass off the list
GAPS = [0.0, 40.0, 60.0, 80.0, 86.0, 90.0, 120.0, 200.0, 300.0, 640.0, 760.0]


def little_off_the_list(dtype, V, ld, k, tau, seed):
    """A row for each of GAPS, whose listed logits are that many tau above the
    others, and a teacher with 0.3 of its mass off the list."""
    M = len(GAPS)
    z = make_logits(dtype, M, V, ld, seed, pad=math.nan)
    vals, idx, _ = make_lists(M, V, k, seed + 1)
    up = torch.tensor(GAPS, device=DEV)[:, None] * tau
    for r in range(M):
        c = idx[r][idx[r] >= 0].long()
        z[r, c] = (z[r, c].float() + up[r]).to(z.dtype)
    lse = torch.logsumexp(torch.where(idx >= 0, vals.double() / tau, -INF), 1) - math.log(0.7)
    return z, (vals, idx, lse.float())


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(100, 1), (500, 1), (900, 4), (6000, 1), (6000, 40), (50257, 1), (50257, 14),
                                      (60001, 14)])
@pytest.mark.parametrize("tau", [0.5, 1.0, 1.7, 2.0, 3.0])
def test_distill_with_little_mass_off_the_list(ctx, dtype, V, copies, tau):
    """The remaining mass's term and its gradient count however small q_r is,
    at coefficients as large as a loss scale makes them on a small batch."""
    M, k = len(GAPS), 5
    z, lists = little_off_the_list(dtype, V, V + 2, k, tau, 40 + V)
    y = torch.randint(0, V, (M,), generator=gen(3), device=DEV, dtype=torch.int32)
    y[::2] = lists[1][::2, 1]
    y[4] = -1
    many = z.repeat(copies, 1)
    lists = tuple(x.repeat(copies, *([1] * (x.dim() - 1))) for x in lists)
    for alpha in (1.0, 0.6):
        check_strict(ctx, dtype, many, V, lists, y.repeat(copies) if alpha < 1 else None, alpha, tau, True,
                     dscale=32768.0 / 16)


# ---------------------------------------------------------------- the mean of many rows
@pytest.mark.parametrize("M", [1000, 40000, (1 << 25) + 7])
def test_mean_loss_of_many_rows(ctx, M):
    """The mean of losses that no power of two divides: compensated sums (two
    half steps a thread) and a tree of ten additions, then one division."""
    z = torch.zeros(M, 2, dtype=torch.float16, device=DEV)
    z[:, 1] = torch.rand(M, generator=gen(2), device=DEV) * 0.01 - 2.0
    vals, idx = torch.zeros(M, 1, device=DEV), torch.zeros(M, 1, dtype=torch.int32, device=DEV)
    row, mean = torch.empty(M, device=DEV), torch.empty(1, device=DEV)
    ctx.reset()
    ctx.distill("fp16", z, vals, idx, None, None, None, row, mean, M, 2, 2, 1, 1.0, 1.0, 1.0)
    ctx.sync()
    want = float(row.double().mean())
    assert 0.12 < want < 0.13
    assert abs(float(mean) - want) <= 14 * U * want
    row[:] = 7.0
    z[M // 2, 0] = -INF  # the listed column ruled out: this row's loss is +inf, and so is the mean
    ctx.distill("fp16", z, vals, idx, None, None, None, row, mean, M, 2, 2, 1, 1.0, 1.0, 1.0)
    with pytest.raises(api.TTError, match="TT_ERR_NONFINITE"):
        ctx.sync()
    assert float(row[M // 2]) == INF and float(mean) == INF


# ---------------------------------------------------------------- refusals
def test_pointers_off_a_word_are_refused(ctx):
    """Every 32-bit argument of the four operators and of the model's calls, one
    at a time two bytes off: an error, and nothing is launched."""
    M, V, k = 4, 50, 5
    z = make_logits("fp32", M, V, V, 1)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)
    f32 = lambda *n: torch.zeros(*n, device=DEV)
    off = lambda t: t.data_ptr() + 2

    def refused(call, args, names):
        ctx.reset()
        call(**args)
        ctx.sync()
        ctx.reset()
        n0 = ctx.launches
        for name in names:
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                call(**{**args, name: off(args[name])})
        assert ctx.launches == n0
        ctx.sync()

    vals, idx, lse = make_lists(M, V, k, 2)
    lists = lambda: dict(vals=f32(M, k), idx=i32(M, k), lse=f32(M))
    refused(lambda **a: ctx.top_logits("fp32", **a), dict(logits=z, M=M, V=V, ld=V, k=k, **lists()), ["vals", "idx", "lse"])
    refused(lambda **a: ctx.distill("fp32", **a),
            dict(logits=z, t_vals=vals, t_idx=idx, t_lse=lse, targets=i32(M), dlogits=None, row_loss=f32(M), mean_loss=f32(1),
                 M=M, V=V, ld=V, k=k, alpha=0.5, tau=1.0, dscale=1.0),
            ["t_vals", "t_idx", "t_lse", "targets", "row_loss", "mean_loss"])
    refused(lambda **a: ctx.beam_select("fp32", **a),
            dict(logits=z, scores=f32(2, 2), done=i32(2, 2), parent=i32(2, 2), token=i32(2, 2), out_scores=f32(2, 2),
                 out_done=i32(2, 2), B=2, K=2, V=V, ld=V, n=2, eos=3),
            ["scores", "done", "parent", "token", "out_scores", "out_done"])
    refused(ctx.beam_reorder, dict(state=z.clone(), parents=i32(2, 2), N=1, B=2, K=2, row_bytes=200, first=0, count=200),
            ["parents"])
    sh = synth.WORKLOADS["tiny_fp32"].shape
    p = synth.init_params(sh)
    _, w = base.device_params(ctx, sh, p, "fp32")
    B, T = 2, 8
    tok, _ = synth.token_stream(B, T, sh.V, "uniform")
    vals, idx, lse = make_lists(B * T, sh.V, k, 1)
    refused(ctx.step_distill,
            dict(params=w, grads=f32(p.size), tokens=tok, targets=i32(B * T), t_vals=vals, t_idx=idx, t_lse=lse, k=k,
                 alpha=0.5, tau=1.0, B=B, T=T), ["targets", "t_vals", "t_idx", "t_lse"])
    refused(ctx.top_logits_of,
            dict(params=w, tokens=tok, B=B, T=T, k=k, vals=f32(B * T, k), idx=i32(B * T, k), lse=f32(B * T)),
            ["vals", "idx", "lse"])


def test_more_positions_than_an_int_counts_are_refused(ctx):
    cfg = api.make_config(1, 64, 4, 65, 1024, "fp32")
    ctx.set_model(cfg)
    w = torch.zeros(1 << 17, device=DEV)
    f, i = torch.zeros(8, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV)
    ctx.reset()
    n0 = ctx.launches
    for B in (1 << 22, 1 << 21, 2 ** 31 - 1):
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.top_logits_of(w, i, B, 1024, 1, f, i, None)
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.step_distill(w, w, i, i, f, i, None, 1, 0.5, 1.0, B, 1024)
    assert ctx.launches == n0


# ---------------------------------------------------------------- long sums
def long_row(dtype, V, head, masked=0):
    """A row whose sum has a few terms of 1 and then terms so small that an
    addition to what has gathered by then loses each of them; before them
    `masked` columns of the type's lowest value."""
    z = torch.full((1, V), -14.0, device=DEV, dtype=TYPES[dtype])
    z[0, :masked] = torch.finfo(TYPES[dtype]).min
    z[0, masked:masked + head] = 0.0
    return z


@pytest.mark.parametrize("dtype,V,M", [("bf16", 50257, 2000), ("fp32", 50257, 2000), ("bf16", 50257, 3), ("fp16", 300001, 1900),
                                       ("bf16", 800000, 1900), ("fp32", 400000, 1900), ("fp32", 400000, 1)])
@pytest.mark.parametrize("head", [1024, 4096])
@pytest.mark.parametrize("masked", [0, 4096])
def test_top_logits_of_long_sums(ctx, dtype, V, M, head, masked):
    """The bound of a sum of n exponentials holds for chains of any length that
    a row can have."""
    one = long_row(dtype, V, head, masked)
    want = torch.logsumexp(one.double(), 1)
    z = one.expand(M, V).contiguous()
    vals, idx, lse = torch.empty(M, 1, device=DEV), torch.empty(M, 1, dtype=torch.int32, device=DEV), torch.empty(M, device=DEV)
    ctx.reset()
    ctx.top_logits(dtype, z, vals, idx, lse, M, V, V, 1, 1.0)
    ctx.sync()
    assert bool((idx == masked).all()) and bool((vals == 0).all())
    assert bool(((lse.double() - want).abs() <= base.lse_tol(want, 30.0)).all()), float((lse.double() - want).abs().max())


@pytest.mark.parametrize("dtype,V,M", [("bf16", 900, 8), ("bf16", 50257, 160), ("fp32", 25000, 160), ("bf16", 3000, 400),
                                       ("bf16", 50257, 1), ("bf16", 800000, 1), ("bf16", 800000, 60), ("fp32", 400000, 60)])
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("masked", [False, True])
def test_distill_of_long_sums(ctx, dtype, V, M, rest, masked):
    """The same in every kernel of distillation: the cross entropy of a label
    whose logit is 0 is the row's log-sum-exp."""
    head = min(V // 4, 4096)
    one = long_row(dtype, V, head, head if masked else 0)
    want = torch.logsumexp(one.double(), 1)
    z = one.expand(M, V).contiguous()
    lists = make_lists(M, V, 4, 5)
    row, _, _ = base.run_distill(ctx, dtype, z, V, lists, torch.full((M,), head, dtype=torch.int32, device=DEV) - (0 if masked else 1),
                                0.0, 1.0, rest)
    assert bool(((row.double() - want).abs() <= base.lse_tol(want, 30.0)).all()), float((row.double() - want).abs().max())


# ---------------------------------------------------------------- logits far from 0
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(100, 1), (900, 1), (6000, 1), (6000, 100), (50257, 1), (50257, 40), (60001, 40)])
@pytest.mark.parametrize("rest", [True, False])
def test_cross_entropy_far_from_zero(ctx, dtype, V, copies, rest):
    """The cross entropy is a matter of differences: z_y and the log-sum-exp
    may be thousands, or the type's lowest value, and the loss is as exact."""
    z = make_logits(dtype, 4, V, V, 3 + V)
    z[0] = (z[0].float() + 3000.0).to(z.dtype)
    z[1] = torch.finfo(TYPES[dtype]).min
    z[2] = (z[2].float() - 20000.0).to(z.dtype)
    y = torch.randint(0, V, (4,), generator=gen(8), device=DEV, dtype=torch.int32)
    want = -torch.log_softmax(z.double(), 1).gather(1, y.long()[:, None])[:, 0]
    lists = make_lists(4 * copies, V, 3, 9)
    row, _, _ = base.run_distill(ctx, dtype, z.repeat(copies, 1), V, lists, y.repeat(copies), 0.0, 1.0, rest)
    err = (row.double() - want.repeat(copies)).abs()
    assert bool((err <= (DEPTH + 34) * U + 4 * U * want.repeat(copies)).all()), float(err.max())


def test_temperatures_whose_arithmetic_overflows_are_refused(ctx):
    M, V, k = 3, 300, 4
    z = make_logits("fp32", M, V, V, 1)
    vals, idx, lse = make_lists(M, V, k, 2)
    row = torch.empty(M, device=DEV)
    ctx.reset()
    n0 = ctx.launches
    for tau in (4e-39, 1e-40):  # 1 / tau is finite for the first, log2(e) / tau is not
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.top_logits("fp32", z, vals.clone(), idx.clone(), None, M, V, V, k, tau)
    for tau in (4e-39, 2e19, 1e38):
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.distill("fp32", z, vals, idx, lse, None, None, row, None, M, V, V, k, 1.0, tau, 1.0)
    assert ctx.launches == n0
    ctx.distill("fp32", z, vals, idx, None, None, None, row, None, M, V, V, k, 1.0, 1e18, 1.0)
    ctx.top_logits("fp32", z, vals.clone(), idx.clone(), row, M, V, V, k, 1e38)
    ctx.sync()
    assert bool(((row.double() - math.log(V)).abs() <= base.lse_tol(row.double(), 30.0)).all())


# ---------------------------------------------------------------- the model's paths at larger vocabularies
def wide(monkeypatch, V, C, H, maxT=32):
    sh = synth.GPT2Shape(2, C, H, V, maxT)
    monkeypatch.setitem(synth.WORKLOADS, "wide", synth.Workload("wide", sh, 1, 8, "fp32", "uniform"))
    return sh


@pytest.mark.parametrize("V,B,T", [(3000, 2, 17), (3000, 20, 20), (50257, 2, 17), (50257, 10, 20), (60001, 8, 20)])
@pytest.mark.parametrize("dtype,tol", [("fp32", 1e-4), ("bf16", 2e-2), ("fp16", 2.5e-3)])
@pytest.mark.parametrize("rest,alpha", [(True, 0.5), (False, 1.0)])
def test_teacher_and_student_step_of_a_larger_vocabulary(oracle, monkeypatch, V, B, T, dtype, tol, rest, alpha):
    """The lists from a forward whose rows are cut into parts, then the step in
    the kernels that hold a row on chip, in a cluster, or stream it; in half
    with a device loss scale.  Bounds as at the small vocabularies."""
    wide(monkeypatch, V, 64, 1)
    base.test_teacher_and_student_step(oracle, "wide", B, T, dtype, tol, rest, alpha)


@pytest.mark.parametrize("V,B,T", [(100, 2, 9), (3000, 2, 17), (3000, 20, 20), (50257, 2, 17), (50257, 10, 20), (60001, 8, 20)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_step_distill_loss_scale(ctx, monkeypatch, V, B, T, dtype):
    """A device loss scale of 2^8 multiplies every gradient by it (a power of
    two: no other rounding; the sums' order is the step's own)."""
    sh = wide(monkeypatch, V, 64, 1)
    p = synth.init_params(sh, jitter=0.05)
    tok, tgt = synth.token_stream(B, T, V, "uniform", seed=3)
    k = 9
    lists = make_lists(B * T, V, k, 4)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, dtype)
    with api.Context(api.arena_bytes(cfg, B, T)) as c:
        _, w = base.device_params(c, sh, p, dtype)
        out = []
        for scale in (None, torch.tensor([256.0], device=DEV)):
            grads = torch.full((p.size,), math.nan, device=DEV)
            c.reset()
            loss = c.step_distill(w, grads, tok, tgt, *lists, k, 0.5, 2.0, B, T, loss_scale=scale)
            out.append((loss, grads.double()))
    assert out[0][0] == out[1][0]
    assert bool(torch.isfinite(out[0][1]).all()) and float(out[0][1].norm()) > 0
    assert float((out[1][1] - 256 * out[0][1]).norm()) <= 1e-6 * 256 * float(out[0][1].norm())


@pytest.mark.parametrize("B,K,n_new,seed", [(1, 4, 6, 13), (1, 4, 6, 16), (1, 12, 5, 14), (5, 4, 5, 11)])
def test_generate_beam_of_a_whole_vocabulary(oracle, monkeypatch, B, K, n_new, seed):
    """Rows of 50257 logits are cut into parts, whose lists the recorded step
    joins; few rows and more than the few-row linear layers take."""
    wide(monkeypatch, 50257, 64, 4)
    base.test_generate_beam_matches_a_plain_search(oracle, "wide", B, 5, n_new, K, False, seed)


# ---------------------------------------------------------------- masks, strictly
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,copies", [(65, 1), (700, 1), (3000, 1), (3000, 40), (50257, 1), (50257, 20), (60001, 20)])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_masks_strictly(ctx, dtype, V, copies, rest):
    """Empty lists, rows without a label, masked logits, entries of probability
    0, one entry that has all the mass or a list that has next to none: every
    gradient is finite and within its bound, at every weight of the two losses."""
    M, k = 10, 20
    low = torch.finfo(TYPES[dtype]).min
    z = make_logits(dtype, M, V, V + 5, 21, pad=math.nan)
    vals, idx, lse = make_lists(M, V, k, 22)
    y = torch.randint(0, V, (M,), generator=gen(6), device=DEV, dtype=torch.int32)
    idx[0] = -1
    y[1] = -1
    free = torch.ones(V, dtype=torch.bool, device=DEV)
    free[idx[2].long().clamp(min=0)] = False
    free[y[2].long()] = False
    z[2, :V][free] = -INF
    vals[3, 3:7] = -INF
    z[4, :V] = 0.5
    z[5, :V] += 300.0
    z[6, :V] = low / 4
    z[6, idx[6, 0].long()] = 1.0
    vals[6, 1:] = -INF
    z[6, y[6].long()] = 0.5
    idx[7, 1:] = -1
    lse[7] = vals[7, 0] / 2.0
    lse[8] = 200.0
    z[9, :V] = low
    lists = tuple(t.repeat(copies, *([1] * (t.dim() - 1))) for t in (vals, idx, lse))
    for alpha in (0.0, 0.5, 1.0):
        check_strict(ctx, dtype, z.repeat(copies, 1), V, lists, y.repeat(copies), alpha, 2.0, rest)
