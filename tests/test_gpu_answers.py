"""The operators of training on answers against plain implementations in 64
bits: log probabilities of given tokens, the clipped policy loss, the loss of
pairs of answers, attention over groups, at the sizes, alignments and masks
where they can go wrong.

Tolerances, with u = 2^-24 (half a step of fp32) and h half a step of the
storage type relative to the value (bf16 2^-8, half 2^-11):
 - the log-sum-exp l of u_v = z_v / tau: the sum of exponentials is off by at
   most (DEPTH + 4 + 30) u relative (as in test_gpu_head.py: DEPTH bounds the
   additions in a row on the way of one term, exponentials below e^-30 of the
   largest do not count), 1 / tau and log2(e) / tau are rounded once, which
   moves every u_v by 3 u |u_v| at most; ln pi = u_y - l inherits both, plus
   its own rounding: lp_tol below.
 - policy: with d = ln pi - old off by that and u |d|, r = e^d is off by (d's
   error + 8 u) relative, the term beta (e^x - x - 1) by |e^x - 1| times x's
   error and 4 u of what it subtracts, and the coefficient alike.
 - preference: v is a sum of log probabilities times beta, in 64 bits; the loss
   and coefficient have slopes of at most 1 and 1/4 in v.
 - a gradient element c ([i = y] - s_i) / tau: c's error, s_i off by (2 DEPTH +
   64 + 3 |ln s_i|) u relative, and half a step of storage.
 - attention: a dot product of D terms is off by (D + 6) u times the sum of the
   terms' sizes; a probability inherits that of its score (and of the
   log-sum-exp) plus 8 u; a sum over n positions adds (n + 80) u of the terms'
   sizes; in 16 bits P and dS are rounded once (h) before the second product
   and the result once (h); what is below the type's normal range is then off
   by half a step there (h2: 2^-25 in half) instead.  group_refs writes these
   out per element."""
import math

import pytest
import torch

from autograd_arena_allocated_gb300 import api
from test_gpu_head import DEPTH, DEV, INF, TYPES, U, ctx, gen, make_logits  # noqa: F401 (ctx: a fixture)

pytestmark = pytest.mark.gpu


def within(got, want, bound, what):
    """error <= bound everywhere; a NaN on either side fails."""
    got = got.double()
    assert bool(torch.isfinite(want).all()) and bool(torch.isfinite(got).all()), what
    ok = (got - want).abs() <= bound
    assert bool(ok.all()), (what, int((~ok).sum()), tuple(ok.shape), float(((got - want).abs() / bound)[~ok].max()))


def same_place(z):
    """A copy at the same place of a 16-byte line: sums are cut at those lines, so only it has the same bits."""
    n, es = z.numel(), z.element_size()
    at = z.data_ptr() % 16 // es
    buf = torch.empty(n + 16, dtype=z.dtype, device=z.device)
    return buf[at:at + n].view(z.shape).copy_(z)


def stored(want, dtype):
    """half a step of the storage type"""
    f = torch.finfo(TYPES[dtype])
    return f.eps / 2 * 1.001 * want.abs() + f.smallest_normal * f.eps / 2 + 1e-37


def make_targets(M, V, seed, missing=0.3):
    g = gen(seed)
    y = torch.randint(0, V, (M,), generator=g, device=DEV)
    return torch.where(torch.rand(M, generator=g, device=DEV) < missing, -1, y).int()


class Rows:
    """ln pi of the labels, the softmax and their bounds, in 64 bits."""

    def __init__(self, z, targets, V, tau):
        x = z[:, :V].double() / tau
        self.on = targets >= 0
        self.y = targets.clamp(min=0).long()[:, None]
        self.lse = torch.logsumexp(x, 1)
        xy = x.gather(1, self.y)[:, 0]
        self.lp = xy - self.lse
        self.ls = x - self.lse[:, None]
        big = torch.maximum(x.abs().amax(1), xy.abs())
        self.lse_tol = (DEPTH + 34) * U + 4 * U * big + U * self.lse.abs()
        self.lp_tol = self.lse_tol + 3 * U * big + U * self.lp.abs()
        self.zero = torch.zeros_like(self.lp)
        self.tau, self.big = tau, big

    def mask(self, v):
        return torch.where(self.on, v, self.zero)

    def gradient(self, c, c_tol, dscale):
        """of coefficients by ln pi -> value and bound (without storage)"""
        s = torch.where(self.on[:, None], self.ls.exp(), 0.0)
        hot = torch.zeros_like(s).scatter_(1, self.y, 1.0) * self.on[:, None]
        c, c_tol = self.mask(c)[:, None], self.mask(c_tol)[:, None]
        k = dscale / self.tau
        rel = (2 * DEPTH + 64 + 3 * self.ls.abs().clamp(max=800.0) + 8 * self.big[:, None]) * U
        return c * (hot - s) * k, (c_tol * (hot - s).abs() + c.abs() * (s * rel + 4 * U * hot)) * abs(k)


# ---------------------------------------------------------------- log probabilities
ROWS = [  # M, V, ld, offset: shorter and longer rows, few and many, odd places
    (1, 1, 1, 0), (3, 2, 5, 1), (70, 7, 8, 0), (40, 65, 128, 0), (200, 100, 100, 3), (9, 255, 256, 1), (33, 513, 513, 5),
    (20, 1000, 1003, 2), (5, 2041, 2048, 0), (6, 2060, 2060, 7), (3, 4097, 4100, 2), (500, 3001, 3001, 0),
    (2, 50257, 50304, 0), (170, 50257, 50257, 1), (2, 151936, 151936, 0), (1, 300001, 300001, 7),
]


def run_logprobs(ctx, dtype, z, targets, V, tau, lse=True):
    M, ld = z.shape
    lp, l = torch.full((M,), 123.0, device=DEV), torch.full((M,), 123.0, device=DEV)
    ctx.reset()
    ctx.logprobs(dtype, z, targets, lp, l if lse else None, M, V, ld, tau)
    return lp, l


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,offset", ROWS)
def test_logprobs(ctx, dtype, M, V, ld, offset):
    z = make_logits(dtype, M, V, ld, 3 + V, offset, pad=math.nan)
    t = make_targets(M, V, 4 + M)
    t[-1] = V - 1
    z[t < 0] = math.nan  # not read
    for tau in (1.0, 0.7, 3.0):
        r = Rows(torch.where(t[:, None] < 0, 0.0, z.float()), t, V, tau)
        lp, l = run_logprobs(ctx, dtype, z, t, V, tau)
        ctx.sync()
        within(lp, r.mask(r.lp), r.mask(r.lp_tol), "logp")
        within(l, r.mask(r.lse), r.mask(r.lse_tol), "lse")
        only, _ = run_logprobs(ctx, dtype, z, t, V, tau, lse=False)
        assert torch.equal(only, lp)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V", [65, 3000, 50257])
def test_logprobs_of_masked_rows(ctx, dtype, V):
    """Masks of -inf and of the type's lowest value, alone and together, far
    logits, a masked label, infinities and NaN."""
    low = torch.finfo(TYPES[dtype]).min
    z = make_logits(dtype, 10, V, V + 3, 5, pad=math.nan)
    t = torch.full((10,), 3, dtype=torch.int32, device=DEV)
    z[0, :V] = -INF
    z[0, 3], z[0, 5] = 1.0, 2.0
    z[1, :V] = low
    z[1, 3], z[1, 5] = 1.0, 2.0
    z[2, :V // 2] = -INF
    z[2, V // 2:V] = low
    z[2, 3], z[2, V - 1] = -100.0, -101.0
    z[3, :V] = low  # all equal: -ln V
    z[4, :V] += 3000.0
    z[5, :V] = -INF
    z[5, 3] = low  # the only one
    r = Rows(z[:6], t[:6], V, 1.0)
    want, tol = r.lp.clone(), r.lp_tol.clone()
    want[3], want[5] = -math.log(V), 0.0
    tol[3], tol[5] = (DEPTH + 34) * U + 2 * U * math.log(V), U
    # differences of masks of the lowest value are exact or far below e^-30, so the size of the masked logits does not count
    tol[1:3] = (DEPTH + 34) * U + 8 * U * 110
    tol[0] = (DEPTH + 34) * U + 8 * U * 2
    z[6, 3] = -INF  # the label: impossible
    z[7, 4] = math.nan
    z[8, 4] = INF
    z[9, :V] = -INF
    lp, l = run_logprobs(ctx, dtype, z, t, V, 1.0)
    ctx.sync()
    within(lp[:6], want, tol, "logp")
    assert lp[6] == -INF and math.isnan(lp[7]) and lp[8] == -INF and l[8] == INF and l[9] == -INF
    assert math.isfinite(l[6]) and math.isnan(l[7]) and math.isnan(lp[9])


def test_rows_without_labels_and_bad_labels(ctx):
    for V in (300, 5000):
        z = make_logits("bf16", 5, V, V, 9)
        t = torch.full((5,), -1, dtype=torch.int32, device=DEV)
        lp, l = run_logprobs(ctx, "bf16", z, t, V, 1.0)
        ctx.sync()
        assert not lp.any() and not l.any()
        for bad in (-2, V, 2 ** 31 - 1, -2 ** 31):
            t[:] = 1
            t[3] = bad
            lp, _ = run_logprobs(ctx, "bf16", z, t, V, 1.0)
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                ctx.sync()
            assert lp[3] == 0.0 and lp[2] < 0.0
    ctx.reset()


# ---------------------------------------------------------------- policy
def make_policy(r, seed, ref=True, weight=True, lo=0.2, hi=0.3):
    """old, ref, adv and weight of a policy near the given log probabilities; no ratio next to a bound"""
    g = gen(seed)
    M = r.lp.shape[0]
    n = lambda sd: sd * torch.randn(M, generator=g, device=DEV)  # noqa: E731
    d = n(0.3)
    for edge in (math.log1p(-lo), math.log1p(hi)):
        d = torch.where((d - edge).abs() < 2e-3, d + 5e-3, d)
    old = (r.lp.float() - d)
    adv = n(1.0)
    adv[::5] = 0.0
    return (old, (r.lp.float() + n(0.4)) if ref else None, adv, (0.5 + torch.rand(M, generator=g, device=DEV)) if weight else None)


def exact_policy(r, p, lo, hi, beta):
    """losses, coefficients and their bounds"""
    old, ref, adv, w = p
    A = adv.double()
    w = torch.ones_like(A) if w is None else w.double()
    d = torch.zeros_like(r.lp) if old is None else r.lp - old.double()
    d_tol = torch.zeros_like(d) if old is None else r.lp_tol + U * d.abs()
    ratio = d.exp()
    inside = torch.where(A >= 0, ratio <= 1 + hi, ratio >= 1 - lo)
    if old is None:
        inside[:] = True
    loss = -torch.minimum(ratio * A, ratio.clamp(1 - lo, 1 + hi) * A)
    ra = torch.where(inside, ratio * A, 0.0)
    coef, tol = -ra, ra.abs() * (d_tol + 8 * U) + 4 * U * loss.abs()
    c_tol = ra.abs() * (d_tol + 8 * U)
    if beta > 0:
        x = ref.double() - r.lp
        x_tol = r.lp_tol + U * x.abs()
        e = torch.expm1(x)
        loss = loss + beta * (e - x)
        coef = coef - beta * e
        tol = tol + beta * (e.abs() * x_tol + 6 * U * (e.abs() + x.abs()))
        c_tol = c_tol + beta * (x.exp() * x_tol + 6 * U * e.abs())
    return w * loss, w * (tol + 4 * U * loss.abs()), w * coef, w * (c_tol + 4 * U * coef.abs())


def run_policy(ctx, dtype, z, t, p, V, lo, hi, beta, tau, dscale, grad=True, in_place=False, sync=True):
    M, ld = z.shape
    z = same_place(z) if in_place else z
    d = z if in_place else torch.full_like(z, 7.0) if grad else None
    lp, row, mean = (torch.full((n,), 123.0, device=DEV) for n in (M, M, 1))
    ctx.reset()
    ctx.policy(dtype, z, t, p[0], p[1], p[2], p[3], d, lp, row, mean, M, V, ld, lo, hi, beta, tau, dscale)
    if sync:
        ctx.sync()
    return lp, row, mean, d


def check_policy(ctx, dtype, z, t, p, V, lo=0.2, hi=0.3, beta=0.1, tau=1.0, dscale=None):
    M, ld = z.shape
    dscale = 1.0 / M if dscale is None else dscale
    clean = torch.where(t[:, None] < 0, 0.0, z.float())
    r = Rows(clean, t, V, tau)
    loss, tol, coef, c_tol = exact_policy(r, p, lo, hi, beta)
    lp, row, mean, d = run_policy(ctx, dtype, z, t, p, V, lo, hi, beta, tau, dscale)
    within(lp, r.mask(r.lp), r.mask(r.lp_tol), "logp")
    within(row, r.mask(loss), r.mask(tol), "row_loss")
    total = r.mask(loss)
    within(mean[0], total.mean(), r.mask(tol).mean() + 8 * U * total.abs().mean() + U * total.mean().abs(), "mean_loss")
    grad, bound = r.gradient(coef, c_tol, dscale)
    within(d[:, :V], grad, bound + stored(grad, dtype), "dlogits")
    assert not d[:, V:].any() and not d[t < 0].any()
    again = run_policy(ctx, dtype, z, t, p, V, lo, hi, beta, tau, dscale, in_place=True)
    assert torch.equal(again[1], row) and torch.equal(again[3], d)
    only = run_policy(ctx, dtype, z, t, p, V, lo, hi, beta, tau, dscale, grad=False)
    assert torch.equal(only[1], row) and torch.equal(only[2], mean)
    return lp, row, mean, d


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,offset", ROWS)
def test_policy(ctx, dtype, M, V, ld, offset):
    z = make_logits(dtype, M, V, ld, 13 + V, offset, pad=math.nan)
    t = make_targets(M, V, 14 + M)
    t[-1] = V - 1
    z[t < 0] = math.nan
    clean = torch.where(t[:, None] < 0, 0.0, z.float())
    dscale = 64.0 if dtype == "fp16" else None
    check_policy(ctx, dtype, z, t, make_policy(Rows(clean, t, V, 1.0), 15), V, dscale=dscale)
    check_policy(ctx, dtype, z, t, make_policy(Rows(clean, t, V, 0.8), 16, ref=False, weight=False, hi=0.2), V, hi=0.2,
                 beta=0.0, tau=0.8, dscale=dscale)
    p = make_policy(Rows(clean, t, V, 1.5), 17)
    check_policy(ctx, dtype, z, t, (None,) + p[1:], V, lo=0.0, hi=0.0, tau=1.5, dscale=dscale)  # no old policy: a ratio of 1


@pytest.mark.parametrize("dtype,V", [("bf16", 65), ("fp32", 700), ("fp16", 5001), ("bf16", 30000)])
def test_policy_gradient_of_another_alignment(ctx, dtype, V):
    """logits and dlogits at different places of a 16-byte line"""
    M, ld = 6, V + 5
    t = make_targets(M, V, 20, 0.2)
    z = make_logits(dtype, M, V, ld, 21, 1)
    p = make_policy(Rows(z, t, V, 1.0), 22)
    _, row, _, d = run_policy(ctx, dtype, z, t, p, V, 0.2, 0.3, 0.1, 1.0, 1.0)
    buf = torch.full((M * ld + 9,), 7.0, dtype=TYPES[dtype], device=DEV)
    for off in (0, 2, 3):
        d2 = buf[off:off + M * ld].view(M, ld)
        row2 = torch.empty(M, device=DEV)
        ctx.reset()
        buf.fill_(7.0)
        ctx.policy(dtype, z, t, p[0], p[1], p[2], p[3], d2, None, row2, None, M, V, ld, 0.2, 0.3, 0.1, 1.0, 1.0)
        ctx.sync()
        assert torch.equal(row2, row) and torch.equal(d2, d)
        assert bool((buf[:off] == 7.0).all()) and bool((buf[off + M * ld:] == 7.0).all())


@pytest.mark.parametrize("dtype,V", [("fp32", 65), ("bf16", 65), ("bf16", 50257), ("fp32", 3000)])
def test_policy_of_masked_and_far_logits(ctx, dtype, V):
    """Vocabularies masked by -inf and by the type's lowest value; logits far from zero."""
    low = torch.finfo(TYPES[dtype]).min
    z = make_logits(dtype, 8, V, V, 31)
    t = torch.full((8,), 3, dtype=torch.int32, device=DEV)
    z[0, 6:] = -INF
    z[1, 6:] = low
    z[2, 6:V // 2] = -INF
    z[2, V // 2:] = low
    z[3] += 500.0
    z[4, :3] = -INF
    z[5, 10:] = -INF
    M = z.shape[0]
    clean = torch.where(z.double() < -1e30, -INF, z.double())
    x = clean[:, :V]
    r = Rows(torch.where(torch.isinf(x), -60000.0, x), t, V, 1.0)  # -60000: nothing beside the rest, but finite
    r.big = torch.where(torch.isinf(x), 0.0, x.abs()).amax(1)
    r.lse_tol = (DEPTH + 34) * U + 4 * U * r.big + U * r.lse.abs()
    r.lp_tol = r.lse_tol + 3 * U * r.big + U * r.lp.abs()
    p = make_policy(r, 32)
    loss, tol, coef, c_tol = exact_policy(r, p, 0.2, 0.3, 0.1)
    lp, row, _, d = run_policy(ctx, dtype, z, t, p, V, 0.2, 0.3, 0.1, 1.0, 1.0)
    within(lp, r.lp, r.lp_tol, "logp")
    within(row, loss, tol, "row_loss")
    grad, bound = r.gradient(coef, c_tol, 1.0)
    within(d, grad, bound + stored(grad, dtype), "dlogits")
    assert not d[torch.isinf(x)].any() and M == 8


def test_policy_ratios_at_and_beyond_the_bounds(ctx):
    """Either sign of the advantage, the ratio inside, on and outside the bounds, and so far off that it overflows."""
    V = 65
    d = torch.tensor([0.0, 0.1, 0.5, -0.5, 200.0, -200.0, 0.0, 0.1, 0.5, -0.5, -200.0], device=DEV)
    M = d.numel()
    z = make_logits("fp32", M, V, V, 41)
    t = torch.full((M,), 7, dtype=torch.int32, device=DEV)
    adv = torch.tensor([2.0] * 6 + [-2.0] * 5, device=DEV)
    lp, _ = run_logprobs(ctx, "fp32", z, t, V, 1.0)
    ctx.sync()
    p = (lp - d, None, adv, None)
    _, row, _, g = run_policy(ctx, "fp32", z, t, p, V, 0.2, 0.3, 0.0, 1.0, 1.0)
    e = math.exp
    want = torch.tensor([-2.0, -2 * e(0.1), -2.6, -2 * e(-0.5), -2.6, -2 * e(-200.0), 2.0, 2 * e(0.1), 2 * e(0.5), 1.6, 1.6])
    assert torch.allclose(row.cpu(), want, rtol=1e-5, atol=1e-30)
    live = (g.abs().sum(1) > 0).cpu()
    # the coefficient of a ratio of e^-200 is below fp32
    assert live.tolist() == [True, True, False, True, False, False, True, True, True, False, False]
    # a ratio that overflows where it is not bounded is reported
    run_policy(ctx, "fp32", z[:1], t[:1], (lp[:1] - 200.0, None, -adv[:1], None), V, 0.2, 0.3, 0.0, 1.0, 1.0, sync=False)
    with pytest.raises(api.TTError, match="TT_ERR_NONFINITE"):
        ctx.sync()
    # no advantage: no loss and no gradient whatever the ratio is
    for dd in (0.0, 200.0, -200.0):
        _, row, _, g = run_policy(ctx, "fp32", z[:1], t[:1], (lp[:1] - dd, None, 0 * adv[:1], None), V, 0.2, 0.3, 0.0, 1.0, 1.0)
        assert not row.any() and not g.any()
    # NaN anywhere shows
    for i in (0, 1, 2, 3):
        p = [lp[:1] - 0.1, lp[:1] + 0.1, adv[:1].clone(), torch.ones(1, device=DEV)]
        p[i] = torch.full((1,), math.nan, device=DEV)
        _, row, _, g = run_policy(ctx, "fp32", z[:1], t[:1], p, V, 0.2, 0.3, 0.1, 1.0, 1.0, sync=False)
        with pytest.raises(api.TTError, match="TT_ERR_NONFINITE"):
            ctx.sync()
        assert math.isnan(row[0]) and bool(torch.isnan(g).all())


@pytest.mark.parametrize("V", [40, 3000])
def test_policy_against_differences(ctx, V):
    """d loss / d z by central differences of the 64-bit loss at a step of 1e-5:
    its error is below 1e-9 of the third derivative's size."""
    M = 3
    z = make_logits("fp32", M, V, V, 51, spread=1.5)
    t = torch.tensor([1, V - 1, -1], dtype=torch.int32, device=DEV)
    p = make_policy(Rows(z, t, V, 1.2), 52)
    _, _, _, d = run_policy(ctx, "fp32", z, t, p, V, 0.2, 0.3, 0.2, 1.2, 1.0)

    def total(x):
        r = Rows(x, t, V, 1.2)
        return r.mask(exact_policy(r, p, 0.2, 0.3, 0.2)[0]).sum()

    r = Rows(z, t, V, 1.2)
    _, _, coef, c_tol = exact_policy(r, p, 0.2, 0.3, 0.2)
    _, bound = r.gradient(coef, c_tol, 1.0)
    for row, col in [(0, 1), (0, 0), (1, V - 1), (1, 5), (2, 3)]:
        x = z.double()
        x[row, col] += 1e-5
        up = total(x)
        x[row, col] -= 2e-5
        fd = (up - total(x)) / 2e-5
        assert abs(float(d[row, col]) - float(fd)) <= float(bound[row, col]) + 1e-8


# ---------------------------------------------------------------- pairs
def run_preference(ctx, dtype, z, t, ref, spans, V, beta, gamma, smooth, mean, tau, dscale, grad=True, in_place=False,
                   sync=True):
    M, ld = z.shape
    P = spans.shape[0] // 2
    z = same_place(z) if in_place else z
    d = z if in_place else torch.full_like(z, 7.0) if grad else None
    seq, loss, m = (torch.full((n,), 123.0, device=DEV) for n in (2 * P, P, 1))
    ctx.reset()
    ctx.preference(dtype, z, t, ref, spans, d, seq, loss, m, M, V, ld, P, beta, gamma, smooth, mean, tau, dscale)
    if sync:
        ctx.sync()
    return seq, loss, m, d


def exact_preference(r, ref, spans, beta, gamma, smooth, mean):
    """sums, losses, coefficients and their bounds"""
    M = r.lp.shape[0]
    total, tt, score, st, n = [], [], [], [], []
    for a, b in spans.tolist():
        on = r.on[a:b]
        lp = r.lp[a:b][on]
        tol = r.lp_tol[a:b][on].sum()
        total.append(lp.sum())
        tt.append(tol + U * lp.sum().abs())
        k = max(int(on.sum()), 1) if mean else 1
        s = (lp - ref[a:b][on].double()).sum() if ref is not None else lp.sum()
        score.append(s / k)
        st.append(tol / k)
        n.append(k)
    total, tt, score, st = (torch.stack(x) for x in (total, tt, score, st))
    v = beta * (score[0::2] - score[1::2]) - gamma
    v_tol = beta * (st[0::2] + st[1::2])
    zero = torch.zeros_like(v)
    loss = (1 - smooth) * torch.logaddexp(zero, -v) + smooth * torch.logaddexp(zero, v)
    dv = smooth * torch.sigmoid(v) - (1 - smooth) * torch.sigmoid(-v)
    coef, c_tol = torch.zeros(M, dtype=torch.float64, device=DEV), torch.zeros(M, dtype=torch.float64, device=DEV)
    for i, (a, b) in enumerate(spans.tolist()):
        coef[a:b] = (1 if i % 2 == 0 else -1) * beta * dv[i // 2] / n[i]
        c_tol[a:b] = beta * (v_tol[i // 2] * dv[i // 2].abs().clamp(max=0.25) + 4 * U * dv[i // 2].abs()) / n[i]
    return total, tt, loss, v_tol * dv.abs() + v_tol ** 2 + 2 * U * loss, coef, c_tol


def check_preference(ctx, dtype, z, t, ref, spans, V, beta=0.1, gamma=0.0, smooth=0.0, mean=False, tau=1.0, dscale=None):
    P = spans.shape[0] // 2
    dscale = 1.0 / P if dscale is None else dscale
    r = Rows(torch.where(t[:, None] < 0, 0.0, z.float()), t, V, tau)
    total, tt, loss, tol, coef, c_tol = exact_preference(r, ref, spans, beta, gamma, smooth, mean)
    seq, got, m, d = run_preference(ctx, dtype, z, t, ref, spans, V, beta, gamma, smooth, mean, tau, dscale)
    within(seq, total, tt, "seq_logp")
    within(got, loss, tol, "pair_loss")
    within(m[0], loss.mean(), tol.mean() + 8 * U * loss.mean(), "mean_loss")
    grad, bound = r.gradient(coef, c_tol, dscale)
    within(d[:, :V], grad, bound + stored(grad, dtype), "dlogits")
    assert not d[:, V:].any()
    again = run_preference(ctx, dtype, z, t, ref, spans, V, beta, gamma, smooth, mean, tau, dscale, in_place=True)
    assert torch.equal(again[1], got) and torch.equal(again[3], d)
    only = run_preference(ctx, dtype, z, t, ref, spans, V, beta, gamma, smooth, mean, tau, dscale, grad=False)
    assert torch.equal(only[1], got) and torch.equal(only[2], m)


def make_spans(M, P, seed):
    """2 P ranges in any order over M rows, some empty, rows between them left out"""
    g = gen(seed)
    cut = torch.sort(torch.randint(0, M + 1, (4 * P,), generator=g, device=DEV)).values.view(2 * P, 2)
    return cut[torch.randperm(2 * P, generator=g, device=DEV)].int().contiguous()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,offset", ROWS)
def test_preference(ctx, dtype, M, V, ld, offset):
    z = make_logits(dtype, M, V, ld, 63 + V, offset, pad=math.nan)
    t = make_targets(M, V, 64 + M, 0.2)
    z[t < 0] = math.nan
    ref = make_policy(Rows(torch.where(t[:, None] < 0, 0.0, z.float()), t, V, 1.0), 65)[1]
    dscale = 64.0 if dtype == "fp16" else None
    for P, args in [(1, dict()), (3, dict(gamma=0.4, smooth=0.2, mean=True, beta=2.0, tau=0.8)), (2, dict(beta=0.02, smooth=0.1))]:
        spans = make_spans(M, P, 66 + P)
        check_preference(ctx, dtype, z, t, ref if P != 3 else None, spans, V, dscale=dscale, **args)


def test_preference_of_long_answers(ctx):
    """One pair over thousands of rows, and hundreds of pairs of a few."""
    M, V = 9000, 300
    z = make_logits("bf16", M, V, 304, 71)
    t = make_targets(M, V, 72, 0.1)
    r = Rows(z, t, V, 1.0)
    ref = make_policy(r, 73)[1]
    spans = torch.tensor([[0, 4000], [4000, 9000]], dtype=torch.int32, device=DEV)
    check_preference(ctx, "bf16", z, t, ref, spans, V, beta=0.01)
    cuts = torch.arange(0, 9001, 15, device=DEV, dtype=torch.int32)
    check_preference(ctx, "bf16", z, t, ref, torch.stack([cuts[:-1], cuts[1:]], 1).contiguous(), V)


def test_preference_of_far_answers(ctx):
    """Differences of a thousand either way: a loss of that size or none, no overflow."""
    V, M = 65, 8
    z = make_logits("fp32", M, V, V, 75)
    t = torch.full((M,), 5, dtype=torch.int32, device=DEV)
    z[:4, 5] = 300.0
    z[4:, 5] = -300.0
    good = torch.tensor([[0, 4], [4, 8]], dtype=torch.int32, device=DEV)
    check_preference(ctx, "fp32", z, t, None, good, V, beta=1.0)
    check_preference(ctx, "fp32", z, t, None, good.flip(0).contiguous(), V, beta=1.0)
    check_preference(ctx, "fp32", z, t, None, good.flip(0).contiguous(), V, beta=1.0, smooth=0.3, gamma=2.0)


def test_preference_flags(ctx):
    V, M = 300, 12
    z = make_logits("fp32", M, V, V, 81)
    t = make_targets(M, V, 82, 0.0)

    def flagged(spans, what="TT_ERR_ARG"):
        run_preference(ctx, "fp32", z, t, None, torch.tensor(spans, dtype=torch.int32, device=DEV), V, 0.1, 0.0, 0.0, False,
                       1.0, 1.0, sync=False)
        with pytest.raises(api.TTError, match=what):
            ctx.sync()

    flagged([[0, 6], [5, 12]])       # a row in two answers
    flagged([[0, 6], [0, 6]])
    flagged([[0, 6], [6, 13]])       # out of range
    flagged([[-1, 6], [6, 12]])
    flagged([[6, 5], [6, 12]])
    flagged([[0, 2 ** 31 - 1], [-2 ** 31, 12]])
    t[3] = V
    flagged([[0, 6], [6, 12]])
    t[3] = 1
    z[2, 7] = math.nan
    flagged([[0, 6], [6, 12]], "TT_ERR_NONFINITE")
    z[2, 7] = 0.0
    # rows without a label may be shared: they count for neither
    t[5] = -1
    check_preference(ctx, "fp32", z, t, None, torch.tensor([[0, 6], [5, 12]], dtype=torch.int32, device=DEV), V)


@pytest.mark.parametrize("V", [40, 3000])
def test_preference_against_differences(ctx, V):
    """as test_policy_against_differences"""
    M = 6
    z = make_logits("fp32", M, V, V, 91, spread=1.5)
    t = torch.tensor([1, V - 1, -1, 3, 0, 2], dtype=torch.int32, device=DEV)
    spans = torch.tensor([[4, 6], [0, 3]], dtype=torch.int32, device=DEV)
    _, _, _, d = run_preference(ctx, "fp32", z, t, None, spans, V, 0.7, 0.2, 0.1, True, 1.2, 1.0)

    def total(x):
        return exact_preference(Rows(x, t, V, 1.2), None, spans, 0.7, 0.2, 0.1, True)[2].sum()

    r = Rows(z, t, V, 1.2)
    coef, c_tol = exact_preference(r, None, spans, 0.7, 0.2, 0.1, True)[4:]
    _, bound = r.gradient(coef, c_tol, 1.0)
    for row, col in [(0, 1), (1, 0), (4, 0), (5, 7), (2, 3), (3, 3)]:
        x = z.double()
        x[row, col] += 1e-5
        up = total(x)
        x[row, col] -= 2e-5
        fd = (up - total(x)) / 2e-5
        assert abs(float(d[row, col]) - float(fd)) <= float(bound[row, col]) + 1e-8


def test_rows_past_32_bits(ctx):
    """More than 2^32 bytes (and 2^31 elements) of logits: the last rows, in place."""
    V, ld = 50257, 50304
    M = 2 ** 31 // ld + 90
    z = torch.zeros(M, ld, dtype=torch.bfloat16, device=DEV)
    last = 40
    z[-last:, :V] = make_logits("bf16", last, V, V, 101)
    t = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    t[-last:] = make_targets(last, V, 102, 0.2)
    r = Rows(z[-last:], t[-last:], V, 1.0)
    lp, _ = run_logprobs(ctx, "bf16", z, t, V, 1.0)
    ctx.sync()
    within(lp[-last:], r.mask(r.lp), r.mask(r.lp_tol), "logp")
    p = [x if x is None else torch.cat([torch.zeros(M - last, device=DEV), x]) for x in make_policy(r, 103)]
    keep = z[-last:].clone()
    row, d = torch.empty(M, device=DEV), z
    ctx.reset()
    ctx.policy("bf16", z, t, p[0], p[1], p[2], p[3], d, None, row, None, M, V, ld, 0.2, 0.3, 0.1, 1.0, 1.0)
    ctx.sync()
    loss, tol, coef, c_tol = exact_policy(r, [x if x is None else x[-last:] for x in p], 0.2, 0.3, 0.1)
    within(row[-last:], r.mask(loss), r.mask(tol), "row_loss")
    grad, bound = r.gradient(coef, c_tol, 1.0)
    within(d[-last:, :V], grad, bound + stored(grad, "bf16"), "policy's gradient")
    z[-last:] = keep
    spans = torch.tensor([[M - last, M - 20], [M - 20, M]], dtype=torch.int32, device=DEV)
    total, tt, loss, tol, coef, c_tol = exact_preference(r, None, spans - (M - last), 0.1, 0.0, 0.0, False)
    seq, pair = torch.empty(2, device=DEV), torch.empty(1, device=DEV)
    ctx.reset()
    ctx.preference("bf16", z, t, None, spans, d, seq, pair, None, M, V, ld, 1, 0.1, 0.0, 0.0, False, 1.0, 1.0)
    ctx.sync()
    within(pair, loss, tol, "pair_loss")
    grad, bound = r.gradient(coef, c_tol, 1.0)
    within(d[-last:, :V], grad, bound + stored(grad, "bf16"), "the pair's gradient")
    del z, d
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- attention over groups
def seen(starts, T):
    """[B, T, T]: does position i see j; [B, T]: which positions count"""
    at = torch.arange(T, device=DEV)
    out = torch.zeros(len(starts), T, T, dtype=torch.bool, device=DEV)
    real = torch.zeros(len(starts), T, dtype=torch.bool, device=DEV)
    for b, s in enumerate(starts):
        part = torch.full((T,), -1, device=DEV)
        part[:s[0]] = 0
        for k, (a, e) in enumerate(zip(s, s[1:])):
            part[a:e] = k + 1
        real[b] = part >= 0
        out[b] = ((part[:, None] == part[None, :]) | (part[None, :] == 0)) & (at[:, None] >= at[None, :])
        out[b] &= real[b][:, None] & real[b][None, :]
    return out, real


def group_refs(dtype, qkv, starts, C, H, y=None, lse=None, dy=None):
    """Forward (dy None) or backward in 64 bits, with a bound for each element."""
    B, T = len(starts), qkv.shape[0] // len(starts)
    D = C // H
    f = torch.finfo(TYPES[dtype])
    h, h2 = (0.0, 0.0) if dtype == "fp32" else (f.eps / 2, f.smallest_normal * f.eps / 2)
    sc = 1.0 / math.sqrt(D)
    ok, real = seen(starts, T)
    ok, live = ok[:, None], real[:, None, :, None]
    heads = lambda x, n: torch.where(live, x.double().view(B, T, n, H, D).permute(2, 0, 3, 1, 4), 0.0)  # noqa: E731
    flat = lambda x: x.permute(0, 2, 1, 3).reshape(B * T, C)  # noqa: E731
    q, k, v = heads(qkv, 3)
    s = (q @ k.transpose(-1, -2)) * sc
    es = (D + 6) * U * (q.abs() @ k.abs().transpose(-1, -2)) * sc + 3 * U * s.abs()  # a score's error, and its scale's
    n = ok.sum(-1, keepdim=True).double()
    if dy is None:
        s = s.masked_fill(~ok, -INF)
        l = torch.logsumexp(s, -1, keepdim=True)
        l0 = torch.where(live, l, 0.0)
        p = torch.where(ok, (s - l0).exp(), 0.0)
        ds = torch.where(ok, es, 0.0).amax(-1, keepdim=True)
        rel = 2 * ds + (n + 80) * U + 3 * U * torch.where(ok, (s - l0).abs().clamp(max=100.0), 0.0)
        out = p @ v
        tol = ((p * rel) @ v.abs()) + (p @ v.abs()) * (rel.amax(-1, keepdim=True) + h) + h2 * (ok.double() @ v.abs())
        lt = ds + (n + 40) * U + 3 * U * l0.abs()
        return flat(out), flat(tol), l0[..., 0], lt[..., 0]
    yy, g = heads(y, 1)[0], heads(dy, 1)[0]
    L = torch.where(live, lse.double()[..., None], 0.0)
    p = torch.where(ok, (s - L).exp(), 0.0)
    dp = torch.where(ok, es + 4 * U * (s.abs() + L.abs()) + 8 * U, 0.0) * p
    Dr = (g * yy).sum(-1, keepdim=True)
    x = g @ v.transpose(-1, -2) - Dr
    ex = (D + 6) * U * (g.abs() @ v.abs().transpose(-1, -2) + (g * yy).abs().sum(-1, keepdim=True)) + 2 * U * x.abs()
    dS, eS = p * x, dp * x.abs() + p * ex + h * (p * x).abs() + 4 * U * (p * x).abs() + h2 * ok
    m = ok.sum(-2, keepdim=True).transpose(-1, -2).double()  # queries of a key
    tr = lambda a: a.transpose(-1, -2)  # noqa: E731
    dq, tq = dS @ k * sc, (eS + (n + 80) * U * dS.abs()) @ k.abs() * sc
    dk, tk = tr(dS) @ q * sc, (tr(eS) + (m + 80) * U * tr(dS).abs()) @ q.abs() * sc
    dv, tv = tr(p) @ g, (tr(dp) + tr(p) * (h + (m + 80) * U) + h2 * tr(ok)) @ g.abs()
    return torch.cat([flat(a) for a in (dq, dk, dv)], 1), torch.cat([flat(a) for a in (tq, tk, tv)], 1)


def group_case(dtype, starts, T, C, seed, pad=math.nan, spread=1.0):
    """qkv with values in the padding that must not matter"""
    B = len(starts)
    qkv = (torch.randn(B, T, 3 * C, generator=gen(seed), device=DEV) * spread).to(TYPES[dtype])
    for b, s in enumerate(starts):
        qkv[b, s[-1]:] = pad
    return qkv.view(B * T, 3 * C), torch.tensor(starts, dtype=torch.int32, device=DEV)


def run_group_fwd(ctx, dtype, qkv, st, T, C, H, sync=True):
    B, K = st.shape[0], st.shape[1] - 1
    y = torch.full((B * T, C), 7.0, dtype=TYPES[dtype], device=DEV)
    lse = torch.full((B, H, T), 7.0, device=DEV)
    ctx.reset()
    ctx.group_attention_fwd(dtype, qkv, st, y, lse, B, T, C, H, K)
    if sync:
        ctx.sync()
    return y, lse


def run_group_bwd(ctx, dtype, qkv, st, y, lse, dy, T, C, H, sync=True):
    B, K = st.shape[0], st.shape[1] - 1
    d = torch.full((B * T, 3 * C), 7.0, dtype=TYPES[dtype], device=DEV)
    ctx.reset()
    ctx.group_attention_bwd(dtype, qkv, st, y, lse, dy, d, B, T, C, H, K)
    if sync:
        ctx.sync()
    return d


def check_group(ctx, dtype, starts, T, C, H, seed=1, spread=1.0):
    qkv, st = group_case(dtype, starts, T, C, seed, spread=spread)
    y, lse = run_group_fwd(ctx, dtype, qkv, st, T, C, H)
    want, tol, l, lt = group_refs(dtype, qkv, starts, C, H)
    within(y, want, tol + stored(want, dtype), "y")
    within(lse, l, lt, "lse")
    _, real = seen(starts, T)
    off = ~real.reshape(-1)
    assert not y[off].any() and not lse.transpose(1, 2).reshape(-1, H)[off].any()
    dy = torch.randn(y.shape, generator=gen(seed + 1), device=DEV).to(TYPES[dtype])
    y2, l2 = y.clone(), lse.clone()
    dy[off], y2[off] = math.nan, math.inf
    l2.transpose(1, 2)[~real] = math.nan
    d = run_group_bwd(ctx, dtype, qkv, st, y2, l2, dy, T, C, H)
    want, tol = group_refs(dtype, qkv, starts, C, H, y, lse, dy)
    within(d, want, tol + stored(want, dtype), "dqkv")
    assert not d[off].any()
    assert torch.equal(run_group_bwd(ctx, dtype, qkv, st, y2, l2, dy, T, C, H), d)  # the same bits again
    return y, lse, d


GROUPS = [  # T, starts
    (1, [[0, 1]]), (1, [[1, 1]]), (1, [[0, 0]]), (2, [[1, 2], [0, 1]]), (3, [[1, 2, 3]]),
    (37, [[10, 20, 30], [0, 0, 37]]), (64, [[64, 64, 64]]), (65, [[64, 65, 65], [1, 64, 65]]),
    (100, [[30, 50, 50, 99], [0, 10, 20, 30], [99, 99, 99, 99]]), (128, [[0, 128, 128]]), (129, [[65, 70, 128]]),
    (200, [[0, 50, 100, 150, 200]]), (257, [[100, 150, 200, 201, 256], [0, 0, 0, 0, 0]]),
    (300, [[0, 64, 128, 192, 256, 300], [5, 5, 5, 5, 5, 5]]), (384, [[130, 200, 384]]), (500, [[1, 127, 255, 256, 257, 500]]),
    (700, [[64, 320, 321, 449, 690], [300, 300, 500, 600, 700]]), (1000, [[10, 300, 620, 950], [700, 800, 900, 1000]]),
]


@pytest.mark.parametrize("dtype,C,H", [("bf16", 128, 2), ("fp16", 64, 1), ("fp32", 64, 1), ("fp32", 64, 4), ("bf16", 64, 2),
                                       ("fp16", 48, 3), ("fp32", 96, 3)])
@pytest.mark.parametrize("T,starts", GROUPS)
def test_group_attention(ctx, dtype, C, H, T, starts):
    check_group(ctx, dtype, starts, T, C, H, seed=T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_group_attention_of_random_groups(ctx, dtype):
    """Random lengths, empty parts among them, in two bands of the tensor-core kernels' grid."""
    g = gen(5)
    for i in range(6):
        T = int(torch.randint(60, 420, (1,), generator=g, device=DEV))
        B, K = 3, int(torch.randint(1, 9, (1,), generator=g, device=DEV))
        starts = [sorted(torch.randint(0, T + 1, (K + 1,), generator=g, device=DEV).tolist()) for _ in range(B)]
        check_group(ctx, dtype, starts, T, 64, 1, seed=10 + i)
    starts = [[40 + b, 80, 100 + b, 130 - b] for b in range(6)]
    check_group(ctx, dtype, starts, 130, 768, 12, seed=20)


@pytest.mark.parametrize("dtype,spread", [("bf16", 4.0), ("fp16", 3.0), ("fp32", 4.0), ("bf16", 0.0)])
def test_group_attention_of_sharp_and_flat_scores(ctx, dtype, spread):
    """Scores whose maximum moves by far more than a block's (the accumulators are rescaled), and equal ones."""
    check_group(ctx, dtype, [[100, 180, 290], [0, 150, 300]], 300, 64, 1, seed=31, spread=spread)


@pytest.mark.parametrize("dtype,T", [("bf16", 70), ("bf16", 256), ("fp32", 100)])
def test_one_answer_is_causal_attention(ctx, dtype, T):
    """One answer that fills the sequence: tt_op_attention, in 16 bits bit for
    bit (the same kernels), in fp32 within both bounds."""
    B, C, H = 2, 128, 2
    for cut in (0, T // 3, T):
        qkv, st = group_case(dtype, [[cut, T]] * B, T, C, 41)
        y, lse = run_group_fwd(ctx, dtype, qkv, st, T, C, H)
        y0, l0 = torch.empty_like(y), torch.empty_like(lse)
        ctx.attention_fwd(dtype, qkv, y0, l0, B, T, C, H)
        dy = torch.randn(y.shape, generator=gen(42), device=DEV).to(TYPES[dtype])
        d0 = torch.empty_like(qkv)
        ctx.attention_bwd(dtype, qkv, y0, l0, dy, d0, B, T, C, H)
        ctx.sync()
        d = run_group_bwd(ctx, dtype, qkv, st, y0, l0, dy, T, C, H)
        if dtype == "bf16":
            assert torch.equal(y, y0) and torch.equal(lse, l0) and torch.equal(d, d0)
        else:
            want, tol, l, lt = group_refs(dtype, qkv, [[cut, T]] * B, C, H)
            within(y0, want, tol + stored(want, dtype), "y")
            want, tol = group_refs(dtype, qkv, [[cut, T]] * B, C, H, y0, l0, dy)
            within(d, want, tol + stored(want, dtype), "dqkv")


def test_a_group_is_its_answers_one_by_one(ctx):
    """The prompt computed once gives what each prompt-and-answer gives as a sequence of its own."""
    C, H, P, n = 128, 2, 90, 70
    T = P + 3 * n
    qkv, st = group_case("fp32", [[P, P + n, P + 2 * n, T]], T, C, 51)
    y, lse = run_group_fwd(ctx, "fp32", qkv, st, T, C, H)
    for k in range(3):
        at = list(range(P)) + list(range(P + k * n, P + (k + 1) * n))
        own = qkv[at].contiguous()
        y0, l0 = torch.empty(P + n, C, device=DEV), torch.empty(1, H, P + n, device=DEV)
        ctx.attention_fwd("fp32", own, y0, l0, 1, P + n, C, H)
        ctx.sync()
        want, tol, l, lt = group_refs("fp32", own, [[P + n, P + n]], C, H)
        within(y[at], want, tol + stored(want, "fp32"), "in the group")
        within(y0, want, tol + stored(want, "fp32"), "alone")
        within(lse[:, :, at], l, lt, "lse")


def test_group_attention_against_differences(ctx):
    """d sum(y w) / d qkv of the 64-bit forward by central differences at a
    step of 1e-5 (error below 1e-8 at these sizes)."""
    T, C, H = 9, 32, 2
    starts = [[3, 5, 8]]
    qkv, st = group_case("fp32", starts, T, C, 61, pad=0.0)
    w = torch.randn(T, C, generator=gen(62), device=DEV)
    y, lse = run_group_fwd(ctx, "fp32", qkv, st, T, C, H)
    d = run_group_bwd(ctx, "fp32", qkv, st, y, lse, w, T, C, H)
    _, tol = group_refs("fp32", qkv, starts, C, H, y, lse, w)
    total = lambda x: (group_refs("fp32", x, starts, C, H)[0] * w.double()).sum()  # noqa: E731
    for i, c in [(0, 0), (0, C + 3), (2, 2 * C + 5), (3, 7), (4, C), (5, 2 * C), (7, 3 * C - 1), (8, 1), (8, C), (1, C + 9)]:
        x = qkv.double()
        x[i, c] += 1e-5
        up = total(x)
        x[i, c] -= 2e-5
        fd = (up - total(x)) / 2e-5
        # y's own rounding enters D: at most a few u of what the sums hold
        assert abs(float(d[i, c]) - float(fd)) <= float(tol[i, c]) + 40 * U * float(w.abs().max()) * 10 + 1e-7


def test_group_attention_flags_bad_starts(ctx):
    T = 100
    for dtype, C, H in (("bf16", 64, 1), ("fp32", 64, 4)):
        for s in ([-1, 50, 100], [10, 50, 101], [60, 50, 100], [2 ** 31 - 1, 5, -2 ** 31], [50, 100, 99]):
            qkv, st = group_case(dtype, [[0, 50, 100], [0, 50, 100]], T, C, 71, pad=0.0)
            st[1] = torch.tensor(s, dtype=torch.int32)
            y, lse = run_group_fwd(ctx, dtype, qkv, st, T, C, H, sync=False)
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                ctx.sync()
            run_group_bwd(ctx, dtype, qkv, st, y, lse, y, T, C, H, sync=False)
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                ctx.sync()
            want, tol, _, _ = group_refs(dtype, qkv[:T], [[0, 50, 100]], C, H)
            within(y[:T], want, tol + stored(want, dtype), "the other group")
    ctx.reset()


@pytest.mark.parametrize("dtype,C,H", [("bf16", 128, 2), ("fp16", 96, 3), ("bf16", 32, 2), ("fp32", 128, 2), ("fp32", 64, 2),
                                       ("fp32", 32, 2)])
def test_group_attention_of_many_answers(ctx, dtype, C, H):
    """Hundreds of answers of a few tokens, many of them empty, past a prompt of several blocks and past none."""
    g = gen(91)
    many = lambda first, T: [first] + sorted(torch.randint(first, T + 1, (300,), generator=g, device=DEV).tolist())  # noqa: E731
    check_group(ctx, dtype, [many(150, 640), many(0, 640), list(range(301)), [640] * 301], 640, C, H, seed=92)


@pytest.mark.parametrize("dtype,D", [("bf16", 16), ("fp16", 32), ("bf16", 64), ("fp32", 16), ("fp32", 32), ("fp32", 64)])
def test_group_attention_of_many_heads(ctx, dtype, D):
    """More (sequence, head) pairs than a band of the grid holds, the last band with a few."""
    B, H = 5, 14
    check_group(ctx, dtype, [[20 + 20 * b, 100, 140 + b, 150] for b in range(B)], 151, H * D, H, seed=93)


@pytest.mark.parametrize("dtype,H,D", [("bf16", 1, 16), ("fp16", 1, 32), ("bf16", 5, 16), ("fp16", 3, 32), ("bf16", 6, 16), ("fp32", 1, 16)])
def test_group_attention_of_widths_beside_64(ctx, dtype, H, D):
    """Channels that 64 does not divide, one narrow head alone among them; a NaN in another head's columns stays there."""
    T, starts, C = 200, [[60, 100, 190], [0, 70, 200], [130, 130, 131]], H * D
    y, lse, d = check_group(ctx, dtype, starts, T, C, H, seed=99)
    if H == 1:
        return
    qkv, st = group_case(dtype, starts, T, C, 99)
    qkv.view(-1, 3, H, D)[:, :, H - 1] = math.nan
    y2, l2 = run_group_fwd(ctx, dtype, qkv, st, T, C, H)
    own = slice(0, (H - 1) * D)
    assert torch.equal(y2[:, own], y[:, own]) and torch.equal(l2[:, :H - 1], lse[:, :H - 1])
    dy = torch.randn(y.shape, generator=gen(100), device=DEV).to(TYPES[dtype])
    d2 = run_group_bwd(ctx, dtype, qkv, st, y2, l2, dy, T, C, H)
    assert torch.equal(d2.view(-1, 3, C)[:, :, own], d.view(-1, 3, C)[:, :, own])


@pytest.mark.parametrize("dtype,D,spread", [("bf16", 16, 5.0), ("fp16", 32, 4.0), ("fp32", 16, 5.0), ("fp32", 32, 0.0)])
def test_narrow_heads_of_sharp_and_flat_scores(ctx, dtype, D, spread):
    check_group(ctx, dtype, [[100, 180, 290], [0, 150, 300]], 300, 2 * D, 2, seed=94, spread=spread)


def test_narrow_heads_flag_bad_starts(ctx):
    T = 100
    for dtype, C, H in (("bf16", 48, 3), ("fp16", 64, 2), ("fp32", 64, 2), ("fp32", 64, 1)):
        for s in ([-1, 50, 100], [10, 50, 101], [60, 50, 100], [2 ** 31 - 1, 5, -2 ** 31], [50, 100, 99]):
            qkv, st = group_case(dtype, [[0, 50, 100], [0, 50, 100]], T, C, 95, pad=0.0)
            st[1] = torch.tensor(s, dtype=torch.int32)
            y, lse = run_group_fwd(ctx, dtype, qkv, st, T, C, H, sync=False)
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                ctx.sync()
            run_group_bwd(ctx, dtype, qkv, st, y, lse, y, T, C, H, sync=False)
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                ctx.sync()
            want, tol, _, _ = group_refs(dtype, qkv[:T], [[0, 50, 100]], C, H)
            within(y[:T], want, tol + stored(want, dtype), "the other group")
    ctx.reset()


@pytest.mark.parametrize("dtype,C,H", [("bf16", 64, 1), ("fp16", 64, 2), ("fp32", 64, 1)])
def test_groups_at_16_byte_boundaries(ctx, dtype, C, H):
    """Every tensor 16 bytes past a longer boundary, its neighbours left as they are."""
    T, starts = 90, [[20, 50, 85], [0, 45, 90]]
    M, n = 2 * T, 16 // torch.empty(0, dtype=TYPES[dtype]).element_size()
    qkv, st = group_case(dtype, starts, T, C, 96)
    y0, l0, d0 = check_group(ctx, dtype, starts, T, C, H, seed=96)

    def off(x, fill=7.0, n=n):
        b = torch.full((x.numel() + 2 * n,), fill, dtype=x.dtype, device=DEV)
        b[n:-n] = x.reshape(-1)
        return b, b[n:-n].view(x.shape)

    (_, q), (_, s) = off(qkv), off(st, 0, 1)
    (yb, y), (lb, lse), (db, d) = off(torch.zeros_like(y0)), off(torch.zeros_like(l0), n=1), off(torch.zeros_like(d0))
    ctx.reset()
    ctx.group_attention_fwd(dtype, q, s, y, lse, 2, T, C, H, 2)
    ctx.sync()
    assert torch.equal(y, y0) and torch.equal(lse, l0)
    dy = torch.randn(M, C, generator=gen(97), device=DEV).to(TYPES[dtype])
    ctx.group_attention_bwd(dtype, q, s, y, lse, off(dy)[1], d, 2, T, C, H, 2)
    ctx.sync()
    assert torch.equal(d, d0)
    for b, k in ((yb, n), (lb, 1), (db, n)):
        assert (b[:k] == 7).all() and (b[-k:] == 7).all()


@pytest.mark.parametrize("B,K,T,H", [(8, 4, 2048, 12), (32, 1, 1024, 12), (3, 7, 700, 5)])
def test_no_wait_of_a_thousand_calls_runs_out(ctx, B, K, T, H):
    """The tensor-core kernels' warps hand blocks to each other by barriers; one that misses a phase runs into its
    wait's limit, which tt_ctx_sync reports. Each call gives the first one's bits."""
    C = 64 * H
    starts = [[T // 2 + (T // 2 - b) * k // K for k in range(K + 1)] for b in range(B)]
    qkv, st = group_case("bf16", starts, T, C, 98, pad=0.0)
    y, lse = run_group_fwd(ctx, "bf16", qkv, st, T, C, H)
    d = run_group_bwd(ctx, "bf16", qkv, st, y, lse, y, T, C, H)
    y2, l2, d2 = torch.empty_like(y), torch.empty_like(lse), torch.empty_like(d)
    for _ in range(10):
        for _ in range(100):
            ctx.group_attention_fwd("bf16", qkv, st, y2, l2, B, T, C, H, K)
            ctx.group_attention_bwd("bf16", qkv, st, y2, l2, y2, d2, B, T, C, H, K)
        ctx.sync()
        assert torch.equal(y2, y) and torch.equal(l2, lse) and torch.equal(d2, d)


def test_groups_past_32_bits(ctx):
    """More than 2^31 elements of qkv: the last group's values and gradients."""
    T, C, H, K = 8192, 1024, 16, 128
    B = 2 ** 31 // (T * 3 * C) + 2
    cuts = list(range(0, T + 1, T // K))
    qkv = torch.zeros(B * T, 3 * C, dtype=torch.bfloat16, device=DEV)
    small = torch.randn(T, 3 * C, generator=gen(81), device=DEV).bfloat16()
    qkv[-T:] = small
    st = torch.tensor([cuts] * B, dtype=torch.int32, device=DEV)
    y, lse = run_group_fwd(ctx, "bf16", qkv, st, T, C, H)
    y0, l0 = run_group_fwd(ctx, "bf16", small, st[:1].contiguous(), T, C, H)
    assert torch.equal(y[-T:], y0) and torch.equal(lse[-1:], l0) and not y[:-T].any()
    dy = torch.ones_like(y)
    big = api.Context(16 * B * H * T)
    d = torch.empty_like(qkv)
    big.group_attention_bwd("bf16", qkv, st, y, lse, dy, d, B, T, C, H, K)
    big.sync()
    d0 = torch.empty_like(small)
    big.group_attention_bwd("bf16", small, st[:1].contiguous(), y0, l0, dy[:T], d0, 1, T, C, H, K)
    big.sync()
    big.close()
    assert torch.equal(d[-T:], d0)
    cols = torch.cat([torch.arange(64) + i * C for i in range(3)]).to(DEV)
    want, tol, _, _ = group_refs("bf16", small[:256, cols].contiguous(), [cuts[:5]], 64, 1)
    within(y[-T:-T + 256, :64], want, tol + stored(want, "bf16"), "y")
    del qkv, d, y
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- together
def test_recorded_calls_replay(ctx):
    """Recorded once, replayed on new inputs: the same as the calls; scratch is not shared with calls after it."""
    c = api.Context(32 << 20)
    M, V, P, T, C, H = 60, 3000, 2, 130, 64, 1
    z = make_logits("bf16", M, V, V, 1)
    t = make_targets(M, V, 2, 0.1)
    p = make_policy(Rows(z, t, V, 1.0), 3)
    spans = make_spans(M, P, 4)
    qkv, st = group_case("bf16", [[30, 80, 120]], T, C, 5, pad=0.0)
    dy = torch.randn(T, C, generator=gen(6), device=DEV).bfloat16()
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    b = lambda *s: torch.zeros(*s, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    o = dict(lp=f(M), row=f(M), mean=f(1), d=b(M, V), seq=f(2 * P), pair=f(P), d2=b(M, V), y=b(T, C), lse=f(1, H, T), dqkv=b(T, 3 * C))

    def calls(x, o):
        x.logprobs("bf16", z, t, o["lp"], None, M, V, V)
        x.policy("bf16", z, t, p[0], p[1], p[2], p[3], o["d"], None, o["row"], o["mean"], M, V, V, 0.2, 0.3, 0.1, 1.0, 1.0)
        x.preference("bf16", z, t, o["lp"], spans, o["d2"], o["seq"], o["pair"], None, M, V, V, P, 0.3, 0.1, 0.1, False, 1.0, 1.0)
        x.group_attention_fwd("bf16", qkv, st, o["y"], o["lse"], 1, T, C, H, 2)
        x.group_attention_bwd("bf16", qkv, st, o["y"], o["lse"], dy, o["dqkv"], 1, T, C, H, 2)

    c.reset()
    c.record(lambda: calls(c, o))
    used = c.used
    assert used > 0  # the recording keeps its scratch
    for seed in (7, 8):
        z.copy_(make_logits("bf16", M, V, V, seed))
        qkv.copy_(group_case("bf16", [[30, 80, 120]], T, C, seed, pad=0.0)[0])
        c.replay()
        c.sync()
        got = {k: v.clone() for k, v in o.items()}
        other = {k: torch.zeros_like(v) for k, v in o.items()}
        calls(c, other)  # beside the recording, in the same context
        c.sync()
        for k in o:
            assert torch.equal(got[k], other[k]), k
        c.replay()
        c.sync()
        for k in o:
            assert torch.equal(o[k], got[k]), k
    c.close()


def test_two_contexts_at_once(ctx):
    """Two contexts on two streams, their calls in flight together."""
    M, V, T, C, H = 400, 9001, 600, 128, 2
    jobs = []
    for i in range(2):
        s = torch.cuda.Stream()
        z = make_logits("bf16", M, V, V, 11 + i)
        t = make_targets(M, V, 12 + i)
        spans = make_spans(M, 3, 13 + i)
        qkv, st = group_case("bf16", [[200 + i, 300, 590]], T, C, 14 + i, pad=0.0)
        jobs.append((s, z, t, spans, qkv, st, api.Context(32 << 20, stream=s.cuda_stream)))
    torch.cuda.synchronize()

    def go(c, z, t, spans, qkv, st):
        d, seq, pair = torch.empty_like(z), torch.empty(6, device=DEV), torch.empty(3, device=DEV)
        y, lse = torch.empty(T, C, device=DEV, dtype=torch.bfloat16), torch.empty(1, H, T, device=DEV)
        dq = torch.empty_like(qkv)
        torch.cuda.synchronize()
        return c, (z, t, spans, qkv, st, d, seq, pair, y, lse, dq)

    def launch(c, a):
        z, t, spans, qkv, st, d, seq, pair, y, lse, dq = a
        c.preference("bf16", z, t, None, spans, d, seq, pair, None, M, V, V, 3, 0.1, 0.0, 0.0, False, 1.0, 1.0)
        c.group_attention_fwd("bf16", qkv, st, y, lse, 1, T, C, H, 2)
        c.group_attention_bwd("bf16", qkv, st, y, lse, y, dq, 1, T, C, H, 2)

    alone = []
    for s, z, t, spans, qkv, st, c in jobs:
        x = go(c, z, t, spans, qkv, st)
        launch(*x)
        c.sync()
        alone.append(x[1][5:])
    both = [go(c, z, t, spans, qkv, st) for s, z, t, spans, qkv, st, c in jobs]
    for _ in range(5):
        for x in both:
            launch(*x)
    for (s, *_, c), x, a in zip(jobs, both, alone):
        c.sync()
        for u, v in zip(x[1][5:], a):
            assert torch.equal(u, v)
        c.close()


def test_refusals(ctx):
    """Arguments that the calls refuse on the host, before anything is launched."""
    M, V, T, C, H = 8, 300, 16, 64, 1
    z = make_logits("fp32", M, V, V, 1)
    t = make_targets(M, V, 2)
    f = torch.zeros(64, device=DEV)
    spans = torch.tensor([[0, 4], [4, 8]], dtype=torch.int32, device=DEV)
    d = torch.empty_like(z)
    odd = f.data_ptr() + 2
    ctx.reset()
    n0 = ctx.launches

    def refused(fn, *bad, status="TT_ERR_ARG"):
        for b in bad:
            with pytest.raises(api.TTError, match=status):
                fn(**b)

    def lp(dtype="fp32", z=z, t=t, o=f, l=None, M=M, V=V, ld=V, tau=1.0):
        ctx.logprobs(dtype, z, t, o, l, M, V, ld, tau)

    rows = [dict(z=None), dict(t=None), dict(M=0), dict(M=-1), dict(V=0), dict(ld=V - 1), dict(V=400001, ld=400001),
            dict(z=z.data_ptr() + 2), dict(t=odd), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan), dict(tau=INF),
            dict(tau=1e-39)]
    refused(lp, *rows, dict(o=None), dict(o=odd), dict(l=odd))

    def pol(z=z, t=t, old=f, ref=f, adv=f, w=f, d=d, lp=f, row=f, mean=f, M=M, V=V, ld=V, lo=0.2, hi=0.2, beta=0.1, tau=1.0):
        ctx.policy("fp32", z, t, old, ref, adv, w, d, lp, row, mean, M, V, ld, lo, hi, beta, tau, 1.0)

    refused(pol, *rows, dict(adv=None), dict(row=None), dict(ref=None), dict(lo=-0.1), dict(lo=1.0), dict(hi=-0.1), dict(hi=INF),
            dict(beta=-1.0), dict(beta=INF), dict(lo=math.nan), dict(hi=math.nan), dict(beta=math.nan),
            dict(d=d.data_ptr() + 1), *[{k: odd} for k in ("old", "ref", "adv", "w", "lp", "row", "mean")])

    def pref(z=z, t=t, ref=f, spans=spans, d=d, seq=f, pair=f, mean=f, M=M, V=V, ld=V, P=1, beta=0.1, gamma=0.0, s=0.0, tau=1.0):
        ctx.preference("fp32", z, t, ref, spans, d, seq, pair, mean, M, V, ld, P, beta, gamma, s, False, tau, 1.0)

    refused(pref, *rows, dict(spans=None), dict(pair=None), dict(P=0), dict(P=-1), dict(beta=0.0), dict(beta=-1.0),
            dict(beta=INF), dict(beta=math.nan), dict(gamma=INF), dict(gamma=math.nan), dict(s=0.5), dict(s=-0.1),
            dict(s=math.nan), *[{k: odd} for k in ("ref", "spans", "seq", "pair", "mean")])
    q = torch.zeros(T, 3 * C, device=DEV)
    y = torch.zeros(T, C, device=DEV)
    st = torch.tensor([[4, 8, 16]], dtype=torch.int32, device=DEV)

    def fwd(q=q, st=st, y=y, l=f, B=1, T=T, C=C, H=H, K=2):
        ctx.group_attention_fwd("fp32", q, st, y, l, B, T, C, H, K)

    shapes = [dict(q=None), dict(st=None), dict(y=None), dict(l=None), dict(B=0), dict(T=0), dict(C=0), dict(H=0), dict(K=0),
              dict(C=65), dict(H=3), dict(C=128), dict(C=40, H=5), dict(B=2 ** 20, T=2 ** 12), dict(T=65535 * 64 + 1),
              dict(K=2 ** 30), dict(q=q.data_ptr() + 8), dict(y=y.data_ptr() + 4), dict(st=odd), dict(l=odd)]
    refused(fwd, *shapes)

    def bwd(q=q, st=st, y=y, l=f, dy=y, dq=q, B=1, T=T, C=C, H=H, K=2):
        ctx.group_attention_bwd("fp32", q, st, y, l, dy, dq, B, T, C, H, K)

    refused(bwd, *shapes, dict(dy=None), dict(dq=None), dict(dy=y.data_ptr() + 4), dict(dq=q.data_ptr() + 8))
    lib = api.lib()
    assert lib.tt_op_logprobs(ctx.h, 7, z.data_ptr(), t.data_ptr(), f.data_ptr(), None, M, V, V, 1.0) == -2
    assert lib.tt_op_group_attention_fwd(ctx.h, 7, q.data_ptr(), st.data_ptr(), y.data_ptr(), f.data_ptr(), 1, T, C, H, 2) == -2
    small = api.Context(256)
    for call in (lambda: small.preference("fp32", z, t, f, spans, d, f, f, f, M * 8, V, V, 1, 0.1, 0.0, 0.0, False, 1.0, 1.0),
                 lambda: small.group_attention_bwd("fp32", q, st, y, f, y, q, 1, 2 ** 12, C, H, 2)):
        with pytest.raises(api.TTError, match="TT_ERR_ARENA_OOM"):
            call()
    small.close()
    assert ctx.launches == n0
    ctx.sync()
