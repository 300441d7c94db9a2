"""The operators on lists of logits against plain implementations in 64 bits:
top logits, distillation (loss and gradient), beam selection and reordering,
at the sizes, alignments and masks where they can go wrong.

Tolerances.  Lists, parents and tokens are exact.  With u = 2^-24 (half a step
of fp32):
 - a sum of n exponentials is off by at most (depth + 4 + A) u relative, depth
   the longest chain of additions of one value (a thread's share of the row
   plus a tree, under 160) and A the largest |argument| of an exponential that
   counts (its rounding); exponentials below e^-30 of the largest do not count.
   The log-sum-exp inherits it absolutely, plus its own rounding.
 - a loss is a sum of terms p (ln p - ln q), each off by a few u times the size
   of what is subtracted.
 - a gradient element is off by half a step of its storage type plus the same
   relative errors of the terms that it is made of.
The functions below write these out."""
import math

import numpy as np
import pytest
import torch

from autograd_arena_allocated_gb300 import api, synth
from autograd_arena_allocated_gb300 import build as native_build

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
DEPTH = 160  # additions in a row on the way of one term into its sum
INF = math.inf


@pytest.fixture(scope="module")
def ctx():
    native_build.build()
    c = api.Context(64 << 20)
    yield c
    c.close()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make_logits(dtype, M, V, ld, seed, offset=0, spread=2.5, pad=None):
    """[M, ld] logits, `offset` elements into their buffer, the padding filled
    with values that must not matter."""
    buf = torch.empty(M * ld + offset, dtype=TYPES[dtype], device=DEV)
    z = buf[offset:].view(M, ld)
    z.copy_(torch.randn(M, ld, generator=gen(seed), device=DEV) * spread)
    if ld > V:
        z[:, V:] = INF if pad is None else pad
    return z


def lse_tol(lse, A):
    return (DEPTH + 4 + A) * U + 2 * U * lse.abs()


# ---------------------------------------------------------------- top logits
def ref_top(z, V, k, tau):
    x = z[:, :V].double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x) + 0.0
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    return np.take_along_axis(x, order, 1), order, torch.logsumexp(z[:, :V].double() / tau, 1)


def check_top(ctx, dtype, z, V, k, tau=1.0, with_lse=True):
    M, ld = z.shape
    vals = torch.full((M, k), 123.0, device=DEV)
    idx = torch.full((M, k), -7, dtype=torch.int32, device=DEV)
    lse = torch.full((M,), 123.0, device=DEV) if with_lse else None
    ctx.reset()
    ctx.top_logits(dtype, z, vals, idx, lse, M, V, ld, k, tau)
    ctx.sync()
    rv, ri, rl = ref_top(z, V, k, tau)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(vals.double().cpu().numpy(), rv)
    if with_lse:
        assert torch.equal(torch.isnan(rl), torch.isnan(lse))
        fin = torch.isfinite(rl)
        assert torch.equal(lse[~fin & ~torch.isnan(rl)].double(), rl[~fin & ~torch.isnan(rl)])
        err = (lse.double() - rl).abs()[fin]
        assert bool((err <= lse_tol(rl[fin], 30.0)).all()), float(err.max())


TOP_CASES = [  # M, V, ld, k, offset
    (1, 1, 1, 1, 0), (3, 2, 5, 2, 1), (5, 7, 8, 7, 0), (9, 65, 128, 65, 0), (16, 256, 256, 10, 3),
    (4, 1000, 1000, 128, 0), (33, 1025, 1031, 1, 5), (2, 4097, 4100, 64, 2), (7, 8191, 8192, 33, 0),
    (1, 50257, 50304, 4, 0), (3, 50257, 50257, 128, 1), (170, 50257, 50304, 50, 0), (2, 151936, 151936, 16, 0),
    (1, 300001, 300001, 100, 7),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,k,offset", TOP_CASES)
def test_top_logits(ctx, dtype, M, V, ld, k, offset):
    z = make_logits(dtype, M, V, ld, 11 + M + V, offset)
    check_top(ctx, dtype, z, V, k, tau=1.0 if M % 2 else 2.5)
    check_top(ctx, dtype, z, V, k, with_lse=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [65, 3000, 50257])
def test_top_logits_hard_rows(ctx, dtype, V):
    """Rows whose list is hard to find: all equal, sorted either way, a few
    columns left by a mask, nothing left, signed zeros, NaN and infinities,
    the best values all in one stretch or on one residue."""
    z = make_logits(dtype, 14, V, V + 3, 5)
    z[0, :V] = 0.25
    z[1, :V] = torch.sort(z[1, :V]).values
    z[2, :V] = torch.sort(z[2, :V], descending=True).values
    z[3, :V] = -INF
    z[3, V // 2:V // 2 + 5] = torch.tensor([1.0, 2.0, 2.0, -1.0, 2.0])
    z[4, :V] = -INF
    z[5, :V] = 0.0
    z[5, 1:V:2] = -0.0
    z[6, 3] = math.nan
    z[6, 4] = INF
    z[7, V - 1] = INF
    z[8, :V] = torch.finfo(TYPES[dtype]).min
    z[9, V // 3:V // 3 + 40] += 30.0
    z[10, ::8] += 30.0
    z[11, 0] = math.nan
    z[12, :V] = (torch.arange(V, device=DEV) % 3).float()
    z[13, :V] = -INF
    z[13, 0:V:max(1, V // 40)] = 1.5
    z[:, V:] = math.nan
    for k in (1, 40, 65):
        check_top(ctx, dtype, z, V, k)


@pytest.mark.parametrize("dtype,M,V,ld,k,offset", [("bf16", 2500, 5003, 5003, 64, 1), ("fp32", 2100, 4500, 4500, 128, 0),
                                                   ("fp16", 2000, 33000, 33024, 7, 0), ("bf16", 1900, 50257, 50304, 128, 0),
                                                   ("fp32", 1900, 20000, 20001, 1, 3)])
def test_top_logits_of_many_rows(ctx, dtype, M, V, ld, k, offset):
    """More rows than the SMs hold at once: ordinary ones, and among them rows
    whose list is hard to find."""
    z = make_logits(dtype, M, V, ld, 13 + V, offset, pad=math.nan)
    z[0, :V] = 0.25
    z[1, :V] = torch.sort(z[1, :V]).values
    z[2, :V] = -INF
    z[3, :V] = -INF
    z[3, V // 2:V // 2 + 5] = torch.tensor([1.0, 2.0, 2.0, -1.0, 2.0])
    z[4, 7] = math.nan
    z[5, V - 1] = INF
    z[6, 0], z[6, 1] = INF, math.nan
    z[7, :V] = torch.finfo(TYPES[dtype]).min
    z[8, :V] = (torch.arange(V, device=DEV) % 3).float()
    z[9, V // 3:V // 3 + 300] = 30.0
    z[10, :V] = math.nan
    z[11, :V] = -0.0
    z[11, 5:V:9] = 0.0
    z[12, :V] += 3000.0
    z[M - 1, :V] = -INF
    z[M - 1, 0:V:max(1, V // 60)] = 1.5
    check_top(ctx, dtype, z, V, k, tau=2.0)
    check_top(ctx, dtype, z, V, k, with_lse=False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("V,ld,k", [(1, 1, 1), (31, 33, 31), (32, 32, 5), (33, 40, 33), (64, 64, 64), (65, 65, 1),
                                    (127, 130, 100), (128, 128, 128), (129, 129, 128)])
def test_top_logits_of_short_rows(ctx, dtype, V, ld, k):
    """Many rows of few logits: plain ones, whole numbers (ties), rows of -inf,
    of the lowest value, with infinities and NaN."""
    M = 3000
    z = make_logits(dtype, M, V, ld, 5 + V, 1)
    z[::7, :V] = torch.round(z[::7, :V])
    check_top(ctx, dtype, z, V, k, tau=1.3)
    z[3::9, :V] = -INF
    z[4::9, :V] = torch.finfo(TYPES[dtype]).min
    z[5::9, : V // 2] = -INF
    z[6::9, V - 1] = math.nan
    z[7::9, V // 2] = INF
    z[8::9, :V] = 0.25
    check_top(ctx, dtype, z, V, k)
    check_top(ctx, dtype, z, V, k, with_lse=False)


# ---------------------------------------------------------------- distillation
def ref_distill(z, V, t_vals, t_idx, t_lse, targets, alpha, tau, want_scale=False):
    """Row losses in 64 bits (differentiable in z [M, V]); with want_scale also
    the size of what each row's loss is made of, for its tolerance."""
    M = z.shape[0]
    used = (t_idx >= 0)
    at = t_idx.long().clamp(min=0)
    logq = torch.log_softmax(z / tau, 1)
    t = torch.where(used, t_vals.double() / tau, torch.tensor(-INF, dtype=torch.float64, device=z.device))
    any_ = used.any(1)
    base = t_lse.double()[:, None] if t_lse is not None else torch.logsumexp(t, 1, keepdim=True)
    logp = torch.where(used & any_[:, None], t - base, torch.tensor(-INF, dtype=torch.float64, device=z.device))
    p = logp.exp()
    lq = logq.gather(1, at)
    on = p > 0
    kl = torch.where(on, p * (torch.where(on, logp, torch.zeros_like(p)) - torch.where(on, lq, torch.zeros_like(p))),
                     torch.zeros_like(p)).sum(1)
    size = (p * (t_vals.double().abs().nan_to_num(posinf=0.0) / tau + base.nan_to_num(neginf=0.0).abs()
                 + (z.detach() / tau).gather(1, at).abs().nan_to_num(posinf=0.0) + 20)).sum(1)
    size = size + torch.logsumexp(z.detach() / tau, 1).abs().nan_to_num(posinf=0.0, neginf=0.0, nan=0.0)
    if t_lse is not None:
        mask = torch.zeros(M, V + 1, dtype=torch.bool, device=z.device)
        mask.scatter_(1, torch.where(used, at, torch.full_like(at, V)), True)
        off = ~mask[:, :V]
        pr = (1 - p.sum(1)).clamp(min=0)
        qr = torch.where(off, logq.exp(), torch.zeros_like(logq)).sum(1)
        ok = (qr > 0) & (pr > 0) & any_
        lr = torch.where(ok, torch.where(ok, pr, 1.0).log() - torch.where(ok, qr, 1.0).log(), torch.zeros_like(pr))
        kl = kl + pr * lr
        size = size * (1 + lr.detach().abs())
    kl = torch.where(any_, kl, torch.zeros_like(kl))
    loss = alpha * tau * tau * kl
    size = alpha * tau * tau * size
    if targets is not None and alpha < 1:
        y = targets.long()
        ce = -torch.log_softmax(z, 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
        loss = loss + (1 - alpha) * torch.where(y >= 0, ce, torch.zeros_like(ce))
        size = size + (1 - alpha) * (torch.logsumexp(z.detach(), 1).abs() + 20)
    return (loss, size) if want_scale else loss


def make_lists(M, V, k, seed, unused=True):
    g = gen(seed)
    idx = torch.rand(M, V, generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32)
    vals = torch.randn(M, k, generator=g, device=DEV) * 2.0 + 3.0
    lse = torch.logsumexp(vals.double(), 1).float() + 0.05 + torch.rand(M, generator=g, device=DEV)
    if unused and k > 2:
        idx[::3, k - 1] = -1
    return vals, idx.contiguous(), lse


def run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, grad=True, in_place=False, dscale=None, sync=True):
    M, ld = z.shape
    vals, idx, lse = lists
    dscale = 1.0 / M if dscale is None else dscale
    row = torch.full((M,), math.nan, device=DEV)
    mean = torch.full((1,), math.nan, device=DEV)
    d = None
    src = z
    if in_place:
        src = torch.empty(z.storage_offset() + z.numel(), dtype=z.dtype, device=DEV)[z.storage_offset():].view(M, ld)
        src.copy_(z)
        d = src
    elif grad:
        d = torch.full_like(z, 77.0)
    ctx.reset()
    ctx.distill(dtype, src, vals, idx, lse if rest else None, targets, d, row, mean, M, V, ld, idx.shape[1], alpha, tau,
                dscale)
    if sync:
        ctx.sync()
    return row, mean, d


def check_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, skip_rows=(), **kw):
    M, ld = z.shape
    vals, idx, lse = lists
    dscale = kw.pop("dscale", 1.0 / M)
    row, mean, d = run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=dscale, **kw)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    for r in skip_rows:
        keep[r] = False
    x = z[:, :V].double().clone()
    x[~keep] = 0.0
    x.requires_grad_(True)
    loss, size = ref_distill(x, V, vals, idx, lse if rest else None, targets, alpha, tau, want_scale=True)
    A = min(30.0, float((x.detach().amax() - x.detach().clamp(min=-1e4).amin()) / min(tau, 1.0)))
    rel = (2 * DEPTH + 4 * A + 64) * U
    ref = loss.detach()
    err = (row.double() - ref).abs()[keep]
    # loss terms: a sum of up to k + 2 products, each off by `rel` of its size at most
    assert bool((err <= rel * size.detach()[keep] + 2 * U * ref.abs()[keep]).all()), (
        float((err / (rel * size.detach()[keep] + 1e-30)).max()))
    m = ref.mean()
    if not skip_rows:
        assert abs(float(mean) - float(m)) <= rel * float(size.mean()) + (M / 1024 + 20) * U * float(ref.abs().mean())
    if d is None:
        return row, mean, d
    (gx,) = torch.autograd.grad(loss.sum(), x)
    gx = gx * dscale
    # what an element is made of, for its absolute part
    with torch.no_grad():
        q = torch.softmax(x / tau, 1)
        part = alpha * tau * 2 * q
        used = idx >= 0
        t = torch.where(used, vals.double() / tau, torch.tensor(-INF, dtype=torch.float64, device=DEV))
        p = (t - (lse.double()[:, None] if rest else torch.logsumexp(t, 1, keepdim=True))).exp().nan_to_num(nan=0.0)
        part.scatter_add_(1, idx.long().clamp(min=0), alpha * tau * p)
        if rest:
            mask = torch.zeros(M, V + 1, dtype=torch.bool, device=DEV)
            mask.scatter_(1, torch.where(used, idx.long(), torch.full_like(idx.long(), V)), True)
            qr = torch.where(mask[:, :V], torch.zeros_like(q), q).sum(1, keepdim=True)
            # p_r is a difference from 1: it is off by a few u absolutely
            part = part + alpha * tau * (q / qr.clamp(min=1e-300)).nan_to_num(posinf=0.0) * 2
        if targets is not None and alpha < 1:
            part += (1 - alpha) * 2 * torch.softmax(x, 1)
            hot = torch.zeros_like(q).scatter_(1, targets.long().clamp(min=0)[:, None], 1.0)
            part += (1 - alpha) * hot
    half = torch.finfo(TYPES[dtype]).eps / 2
    tiny = torch.finfo(TYPES[dtype]).smallest_normal * torch.finfo(TYPES[dtype]).eps
    bound = half * gx.abs() * 1.001 + rel * part * abs(dscale) + tiny / 2 + 1e-37
    err = (d[:, :V].double() - gx).abs()
    bad = (err > bound)[keep]
    assert not bool(bad.any()), (int(bad.sum()), float((err / bound)[keep].max()))
    assert bool((d[:, V:] == 0).all())
    for r in skip_rows:
        assert float(row[r]) == 0.0 and bool((d[r] == 0).all())
    return row, mean, d


DISTILL_CASES = [  # M, V, ld, k, offset, alpha, tau, rest
    (1, 1, 1, 1, 0, 1.0, 1.0, False), (3, 2, 3, 1, 1, 0.5, 2.0, True), (4, 5, 8, 5, 0, 0.7, 1.5, True),
    (6, 65, 128, 8, 0, 0.5, 2.0, False), (5, 65, 67, 64, 3, 1.0, 3.0, True), (40, 256, 256, 128, 0, 0.9, 0.7, True),
    (3, 1000, 1000, 10, 0, 0.0, 2.0, False), (9, 1023, 1024, 33, 5, 0.5, 1.0, True), (2, 2051, 2053, 7, 1, 0.3, 4.0, False),
    (7, 8192, 8192, 100, 0, 0.5, 2.0, True), (1, 50257, 50304, 64, 0, 0.5, 2.0, True),
    (3, 50257, 50257, 64, 3, 0.25, 2.0, True), (160, 50257, 50304, 16, 0, 1.0, 2.0, False),
    (5, 32000, 32000, 128, 0, 0.5, 1.0, True), (2, 151936, 151936, 20, 0, 0.5, 2.0, True),
    (1, 262144, 262147, 50, 1, 0.8, 1.3, True),
    (320, 2048, 2048, 128, 0, 0.5, 2.0, True), (310, 1500, 1503, 16, 1, 0.4, 1.3, False), (40, 700, 704, 20, 0, 1.0, 3.0, True),
    (320, 9000, 9000, 30, 0, 0.5, 4.0, False), (161, 40001, 40001, 12, 1, 0.6, 3.0, True),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,k,offset,alpha,tau,rest", DISTILL_CASES)
def test_distill(ctx, dtype, M, V, ld, k, offset, alpha, tau, rest):
    z = make_logits(dtype, M, V, ld, 3 + M + V, offset)
    lists = make_lists(M, V, k, 17 + V)
    targets = torch.randint(0, V, (M,), generator=gen(4), device=DEV, dtype=torch.int32) if alpha < 1 else None
    if targets is not None:
        targets[0] = lists[1][0, 0]  # a target on the list
    scale = 1024.0 / M if dtype == "fp16" else 1.0 / M
    row, _, d = check_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=scale)
    r2, _, d2 = run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=scale, in_place=True)
    assert torch.equal(row, r2) and torch.equal(d, d2)
    r3, _, none = run_distill(ctx, dtype, z, V, lists, targets, alpha, tau, rest, dscale=scale, grad=False)
    assert none is None and torch.equal(row, r3)


DISTILL_STREAMED = [  # rows in such numbers that they are not held on chip
    (420, 2049, 2049, 128, 0, 0.5, 2.0, True), (400, 2100, 2103, 9, 1, 1.0, 1.0, False),
    (333, 4097, 4100, 50, 2, 0.4, 3.0, True), (310, 9001, 9088, 1, 0, 0.5, 4.0, True),
    (700, 5000, 5000, 20, 0, 0.0, 2.0, False), (307, 10007, 10007, 64, 3, 0.7, 0.8, True),
    (153, 60001, 60001, 64, 1, 0.5, 2.0, True), (160, 58000, 58112, 10, 0, 1.0, 2.5, False),
    (80, 120011, 120013, 100, 0, 0.3, 1.0, True), (60, 151936, 151936, 16, 0, 0.5, 1.7, True),
    (60, 300001, 300003, 7, 1, 0.5, 4.0, True),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("M,V,ld,k,offset,alpha,tau,rest", DISTILL_STREAMED)
def test_distill_of_many_rows(ctx, dtype, M, V, ld, k, offset, alpha, tau, rest):
    test_distill(ctx, dtype, M, V, ld, k, offset, alpha, tau, rest)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V,copies", [(3000, 40), (60000, 20)])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_masks_of_many_rows(ctx, dtype, V, copies, rest):
    """The rows of test_distill_masks in such numbers that they are not held on
    chip; every copy of a row receives the same, bit by bit (its rows lie at
    one place of a 16-byte line)."""
    M, k, ld = 12, 20, V + 8
    z = make_logits(dtype, M, V, ld, 21, pad=math.nan)
    vals, idx, lse = make_lists(M, V, k, 22)
    y = torch.randint(0, V, (M,), generator=gen(6), device=DEV, dtype=torch.int32)
    idx[1] = -1
    y[2] = -1
    idx[3], y[3] = -1, -1
    z[3] = math.nan
    free = torch.ones(V, dtype=torch.bool, device=DEV)
    free[idx[4].long().clamp(min=0)] = False
    free[y[4].long()] = False
    z[4, :V][free] = -INF
    vals[5, 3:7] = -INF
    z[6, :V] = 0.5
    z[7, :V] += 3000.0
    z[8, :V] = torch.finfo(TYPES[dtype]).min / 4
    z[8, idx[8, 0].long()] = 1.0
    vals[8, 1:] = -INF
    z[8, y[8].long()] = 0.5
    idx[9, 1:] = -1
    lse[9] = vals[9, 0] / 2.0
    lse[10] = 200.0
    z[11, :V] = torch.finfo(TYPES[dtype]).min  # a whole row of the lowest value
    many = z.repeat(copies, 1)
    lists = tuple(t.repeat(copies, *([1] * (t.dim() - 1))) for t in (vals, idx, lse))
    for alpha in (0.5, 1.0):
        empty = (3,) if alpha < 1 else (1, 3)
        skip = tuple(r + 12 * c for c in range(copies) for r in empty)
        row, _, d = check_distill(ctx, dtype, many, V, lists, y.repeat(copies), alpha, 2.0, rest, skip_rows=skip)
        assert bool((row.view(copies, M) == row[:M]).all())
        assert bool((d.view(copies, M, ld) == d[:M]).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,V", [(40, 65), (40, 900), (12, 3000), (400, 3000), (3, 120000), (160, 60000)])
def test_distill_of_labels_only_with_a_known_normaliser(ctx, dtype, M, V):
    """alpha 0: the list has no weight, but its columns still count in the cross entropy."""
    z = make_logits(dtype, M, V, V + 1, 8)
    lists = make_lists(M, V, 30, 9)
    y = torch.randint(0, V, (M,), generator=gen(10), device=DEV, dtype=torch.int32)
    y[::2] = lists[1][::2, 3]
    z[1, lists[1][1, :20].long()] += 12.0  # most of the mass is on the list
    for tau in (1.0, 2.0):
        a = check_distill(ctx, dtype, z, V, lists, y, 0.0, tau, True)
        b = check_distill(ctx, dtype, z, V, lists, y, 0.0, tau, False)
        assert bool(((a[0] - b[0]).abs() <= 4 * (DEPTH + 64) * U * (20 + b[0].abs())).all())


@pytest.mark.parametrize("V,M", [(3000, 400), (70000, 160)])
def test_distill_of_many_rows_other_alignment_and_flags(ctx, V, M):
    """dlogits that starts at another place of a line; bad columns and labels."""
    ld, k = V + 2, 9
    z = make_logits("bf16", M, V, ld, 9, offset=1)
    lists = make_lists(M, V, k, 2)
    y = torch.randint(0, V, (M,), generator=gen(5), device=DEV, dtype=torch.int32)
    _, _, want = run_distill(ctx, "bf16", z, V, lists, y, 0.5, 2.0, True)
    for off in (0, 7):
        buf = torch.full((M * ld + 72,), 55.0, dtype=torch.bfloat16, device=DEV)
        d = buf[off:off + M * ld].view(M, ld)
        row = torch.empty(M, device=DEV)
        ctx.reset()
        ctx.distill("bf16", z, *lists, y, d, row, None, M, V, ld, k, 0.5, 2.0, 1.0 / M)
        ctx.sync()
        assert torch.equal(d, want)
        assert bool((buf[:off] == 55).all()) and bool((buf[off + M * ld:] == 55).all())
    for name in ("column", "twice", "label"):
        idx, t = lists[1].clone(), y.clone()
        if name == "column":
            idx[M - 1, 3] = V
        elif name == "twice":
            idx[M - 2, 4] = idx[M - 2, 1]
        else:
            t[M - 1] = -2
        run_distill(ctx, "bf16", z, V, (lists[0], idx, lists[2]), t, 0.5, 1.0, True, sync=False)
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.sync()
    check_distill(ctx, "bf16", z, V, lists, y, 0.5, 2.0, True)


@pytest.mark.parametrize("V", [65, 5000, 50257])
def test_distill_gradient_buffer_of_another_alignment(ctx, V):
    """logits and dlogits that start at different places of a 16-byte line."""
    M, ld = 5, V + 2
    z = make_logits("bf16", M, V, ld, 9, offset=1)
    lists = make_lists(M, V, 9, 2)
    _, _, want = run_distill(ctx, "bf16", z, V, lists, None, 1.0, 2.0, True)
    for off in (0, 2, 7):
        buf = torch.full((M * ld + 8 + 64,), 55.0, dtype=torch.bfloat16, device=DEV)
        d = buf[off:off + M * ld].view(M, ld)
        row = torch.empty(M, device=DEV)
        ctx.reset()
        ctx.distill("bf16", z, lists[0], lists[1], lists[2], None, d, row, None, M, V, ld, 9, 1.0, 2.0, 1.0 / M)
        ctx.sync()
        assert torch.equal(d, want)
        assert bool((buf[:off] == 55).all()) and bool((buf[off + M * ld:] == 55).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [65, 3000, 50257])
@pytest.mark.parametrize("rest", [True, False])
def test_distill_masks(ctx, dtype, V, rest):
    """Masked logits, empty lists, rows without a label, rows with neither
    (whatever they hold), entries of probability 0, huge and equal logits."""
    M, k = 12, 20
    z = make_logits(dtype, M, V, V + 5, 21, pad=math.nan)
    vals, idx, lse = make_lists(M, V, k, 22)
    y = torch.randint(0, V, (M,), generator=gen(6), device=DEV, dtype=torch.int32)
    idx[1] = -1                      # no list: cross entropy only
    y[2] = -1                        # no label: the list only
    idx[3], y[3] = -1, -1            # neither: nothing is read
    z[3] = math.nan
    free = torch.ones(V, dtype=torch.bool, device=DEV)
    free[idx[4].long().clamp(min=0)] = False
    free[y[4].long()] = False
    z[4, :V][free] = -INF            # the student has nothing off the list
    vals[5, 3:7] = -INF              # entries that the teacher rules out
    z[6, :V] = 0.5                   # all equal
    z[7, :V] += 3000.0               # far from zero
    z[8, :V] = torch.finfo(TYPES[dtype]).min / 4
    z[8, idx[8, 0].long()] = 1.0
    vals[8, 1:] = -INF
    z[8, y[8].long()] = 0.5
    idx[9, 1:] = -1                  # one entry
    lse[9] = vals[9, 0] / 2.0
    lse[10] = 200.0                  # the teacher knows almost nothing of the list
    for alpha in (0.5, 1.0):
        skip = (3,) if alpha < 1 else (1, 3)
        check_distill(ctx, dtype, z, V, (vals, idx, lse), y, alpha, 2.0, rest, skip_rows=skip)


def test_distill_against_differences(ctx):
    """The gradient against central differences of the call's own loss, fp32.
    h = 2^-6: the third derivative of a row's loss is at most alpha tau^2 / tau^3
    + (1 - alpha) <= 1, so the difference is off by h^2 / 6 at most, plus the
    loss's own error over h."""
    M, V, k, alpha, tau, h = 1, 37, 6, 0.6, 1.7, 2.0 ** -6
    z = make_logits("fp32", M, V, V, 31)
    lists = make_lists(M, V, k, 32)
    y = torch.tensor([int(lists[1][0, 2])], dtype=torch.int32, device=DEV)
    for rest in (True, False):
        _, _, d = run_distill(ctx, "fp32", z, V, lists, y, alpha, tau, rest, dscale=1.0)
        both = z.repeat(2 * V, 1)
        both[torch.arange(V), torch.arange(V)] += h
        both[V + torch.arange(V), torch.arange(V)] -= h
        many = tuple(x.repeat(2 * V, *([1] * (x.dim() - 1))) for x in lists)
        row, _, _ = run_distill(ctx, "fp32", both, V, many, y.repeat(2 * V), alpha, tau, rest, grad=False)
        diff = (row[:V].double() - row[V:].double()) / (2 * h)
        tol = h * h / 6 * 4 + 64 * U * 20 * tau * tau / h
        assert float((diff - d[0].double()).abs().max()) <= tol


def test_distill_own_list_gives_nothing(ctx):
    """A student equal to its teacher: loss and gradient vanish to rounding."""
    M, V, k, tau = 7, 50257, 64, 2.0
    z = make_logits("bf16", M, V, 50304, 41)
    vals = torch.empty(M, k, device=DEV)
    idx = torch.empty(M, k, dtype=torch.int32, device=DEV)
    lse = torch.empty(M, device=DEV)
    ctx.reset()
    ctx.top_logits("bf16", z, vals, idx, lse, M, V, 50304, k, tau)
    row, mean, d = run_distill(ctx, "bf16", z, V, (vals, idx, lse), None, 1.0, tau, True, dscale=1.0)
    tol = (2 * DEPTH + 200) * U * 40 * tau * tau
    assert float(row.abs().max()) <= tol and float(d.float().abs().max()) <= tol


def test_distill_of_the_most_rows(ctx):
    """2^31 - 1 rows of one logit: a softmax over one column has no loss."""
    M = 2 ** 31 - 1
    z = torch.ones(M, 1, dtype=torch.float16, device=DEV)
    vals = torch.ones(M, 1, device=DEV)
    idx = torch.zeros(M, 1, dtype=torch.int32, device=DEV)
    row = torch.full((M,), 7.0, device=DEV)
    mean = torch.full((1,), 7.0, device=DEV)
    ctx.reset()
    ctx.distill("fp16", z, vals, idx, None, None, None, row, mean, M, 1, 1, 1, 1.0, 2.0, 1.0)
    ctx.sync()
    assert float(row.max()) == 0.0 and float(row.min()) == 0.0 and float(mean) == 0.0
    del z, vals, idx, row
    torch.cuda.empty_cache()


def test_rows_past_32_bits(ctx):
    """More than 2^31 logits: the last rows of each operator over them."""
    V, ld, k = 50257, 50304, 8
    M = 2 ** 31 // ld + 40
    z = torch.zeros(M, ld, dtype=torch.bfloat16, device=DEV)
    last = 64
    z[-last:] = make_logits("bf16", last, V, ld, 21)
    tail = z[-last:].clone()
    vals, idx = torch.empty(M, k, device=DEV), torch.empty(M, k, dtype=torch.int32, device=DEV)
    lse = torch.empty(M, device=DEV)
    ctx.reset()
    ctx.top_logits("bf16", z, vals, idx, lse, M, V, ld, k, 1.0)
    ctx.sync()
    rv, ri, rl = ref_top(tail, V, k, 1.0)
    assert np.array_equal(idx[-last:].cpu().numpy(), ri) and np.array_equal(vals[-last:].double().cpu().numpy(), rv)
    assert bool(((lse[-last:].double() - rl).abs() <= lse_tol(rl, 30.0)).all())
    # the choice of the last sequence
    B, K = M // 4, 4
    scores = -torch.rand(B, K, generator=gen(22), device=DEV)
    par, tok = torch.empty(B, K, dtype=torch.int32, device=DEV), torch.empty(B, K, dtype=torch.int32, device=DEV)
    sc = torch.empty(B, K, device=DEV)
    ctx.beam_select("bf16", z, scores, None, par, tok, sc, None, B, K, V, ld, K, -1)
    ctx.sync()
    rows = z[(B - 8) * K:B * K]
    rp, rt, _, _ = ref_select(rows, scores[-8:], None, K, V, K, -1)
    assert torch.equal(par[-8:], rp) and torch.equal(tok[-8:], rt)
    # a model's own whole list gives (nearly) no loss; in place
    row = torch.full((M,), 7.0, device=DEV)
    ctx.distill("bf16", z, vals, idx, lse, None, z, row, None, M, V, ld, k, 1.0, 1.0, 1.0)
    ctx.sync()
    tol = (2 * DEPTH + 200) * U * 40
    assert float(row[-last:].abs().max()) <= tol and float(z[-last:, :V].float().abs().max()) <= tol
    assert float(z[-last:, V:].float().abs().max()) == 0.0
    del z
    torch.cuda.empty_cache()


def test_distill_flags(ctx):
    M, V, k = 4, 300, 5
    z = make_logits("fp32", M, V, V, 51)
    good = make_lists(M, V, k, 52, unused=False)
    y = torch.zeros(M, dtype=torch.int32, device=DEV)

    def flagged(idx, targets, alpha=0.5):
        run_distill(ctx, "fp32", z, V, (good[0], idx, good[2]), targets, alpha, 1.0, True, sync=False)
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.sync()

    for bad in (V, -2, 1 << 30):
        idx = good[1].clone()
        idx[2, 1] = bad
        flagged(idx, y)
        t = y.clone()
        t[3] = bad
        flagged(good[1], t)
    idx = good[1].clone()
    idx[0, 4] = idx[0, 1]
    flagged(idx, y)
    bad = make_logits("fp32", M, V, V, 51)
    bad[1, 7] = math.nan
    run_distill(ctx, "fp32", bad, V, good, y, 0.5, 1.0, True, sync=False)
    with pytest.raises(api.TTError, match="TT_ERR_NONFINITE"):
        ctx.sync()
    check_distill(ctx, "fp32", z, V, good, y, 0.5, 1.0, True)  # usable afterwards


# ---------------------------------------------------------------- beam search
def ref_select(z, scores, done, K, V, n, eos):
    B = scores.shape[0]
    x = z[:, :V].double().view(B, K, V)
    cand = scores.double()[:, :, None] + (x - torch.logsumexp(x, 2, keepdim=True))
    cand = torch.where(torch.isnan(cand), -INF, cand)
    if done is not None:
        only = (torch.arange(V, device=DEV) == eos)[None, None, :]
        cand = torch.where(done[:, :, None] != 0,
                           torch.where(only, scores.double()[:, :, None], -INF), cand)
    cand = cand.reshape(B, K * V)
    best, at = torch.sort(cand, dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    par, tok = at // V, at % V
    d = tok == eos
    if done is not None:
        d = d | (done.gather(1, par) != 0)
    return par.int(), tok.int(), best, d.int()


def check_select(ctx, dtype, z, scores, done, K, V, n, eos, flag=False):
    B, ld = scores.shape[0], z.shape[1]
    par = torch.full((B, n), -9, dtype=torch.int32, device=DEV)
    tok, od = par.clone(), par.clone()
    sc = torch.full((B, n), 9.0, device=DEV)
    ctx.reset()
    ctx.beam_select(dtype, z, scores, done, par, tok, sc, od, B, K, V, ld, n, eos)
    if flag:
        with pytest.raises(api.TTError, match="TT_ERR_NONFINITE"):
            ctx.sync()
    else:
        ctx.sync()
    rp, rt, rs, rd = ref_select(z, scores, done, K, V, n, eos)
    assert torch.equal(par, rp) and torch.equal(tok, rt) and torch.equal(od, rd)
    fin = torch.isfinite(rs)
    assert torch.equal(fin, torch.isfinite(sc))
    # the log-sum-exp's error, then one rounding to fp32
    tol = (DEPTH + 4 + 30) * U + 1.01 * U * rs[fin].abs()
    assert bool(((sc[fin].double() - rs[fin]).abs() <= tol).all())


SELECT_CASES = [  # B, K, V, ld, n, offset
    (1, 1, 1, 1, 1, 0), (1, 1, 50257, 50304, 5, 0), (1, 4, 50257, 50304, 4, 0), (2, 3, 65, 128, 6, 0),
    (5, 2, 3, 7, 6, 1), (3, 5, 1001, 1001, 10, 3), (1, 32, 4000, 4000, 64, 0), (33, 8, 300, 301, 16, 0),
    (2, 16, 151936, 151936, 16, 0), (64, 4, 8192, 8192, 8, 0), (1, 2, 300001, 300003, 4, 1),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("B,K,V,ld,n,offset", SELECT_CASES)
def test_beam_select(ctx, dtype, B, K, V, ld, n, offset):
    z = make_logits(dtype, B * K, V, ld, 61 + V, offset)
    scores = torch.randn(B, K, generator=gen(62), device=DEV) - 40.0
    check_select(ctx, dtype, z, scores, None, K, V, n, -1)
    done = (torch.rand(B, K, generator=gen(63), device=DEV) < 0.4).int()
    check_select(ctx, dtype, z, scores, done, K, V, n, V - 1)
    check_select(ctx, dtype, z, scores, done, K, V, n, 0)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("allowed", [0, 1, 5, 40])
def test_beam_select_of_few_allowed_tokens(ctx, dtype, allowed):
    """A vocabulary masked down to a few tokens (decoding after a grammar):
    the candidates beyond them are the first masked columns."""
    B, K, V, n = 3, 4, 50257, 8
    z = make_logits(dtype, B * K, V, V + 1, 75)
    keep = torch.randperm(V, generator=gen(76), device=DEV)[:allowed]
    hide = torch.ones(V, dtype=torch.bool, device=DEV)
    hide[keep] = False
    z[:, :V][:, hide] = -INF
    scores = -1.0 - torch.rand(B, K, generator=gen(77), device=DEV)
    check_select(ctx, dtype, z, scores, None, K, V, n, -1)
    check_top(ctx, dtype, z, V, 64)


@pytest.mark.parametrize("V", [65, 6000, 50257])
def test_beam_select_ties_and_masks(ctx, V):
    """Equal beams, whole-number logits (many ties), masked vocabularies, slots
    without a hypothesis, every beam finished."""
    B, K, n = 4, 4, 8
    z = make_logits("fp32", B * K, V, V, 71)
    z[0:4] = (torch.arange(V, device=DEV) % 5).float()  # sequence 0: the same logits in every beam
    z[4:8, :] = -INF
    z[4:8, 3:6] = 1.0                                   # sequence 1: three columns left
    z[5] = -INF                                         # ... and a beam with none
    scores = torch.tensor([[-1.0, -1.0, -1.0, -1.0], [-2.0, -3.0, -2.0, -INF], [-INF, -INF, -1.0, -INF],
                           [-5.0, -4.0, -4.0, -INF]], device=DEV)
    check_select(ctx, "fp32", z, scores, None, K, V, n, -1)
    done = torch.zeros(B, K, dtype=torch.int32, device=DEV)
    done[3] = 1
    done[0, 2] = 1
    check_select(ctx, "fp32", z, scores, done, K, V, n, 2)
    z[9, 1] = math.nan
    z[13, 0] = INF
    check_select(ctx, "fp32", z, scores, None, K, V, n, -1, flag=True)


def test_beam_select_in_place_and_far_scores(ctx):
    """Outputs over the inputs' arrays; scores so low that 32 bits would tie
    what differs."""
    B, K, V = 6, 8, 2000
    z = make_logits("fp32", B * K, V, V, 81)
    scores = -3000.0 + torch.rand(B, K, generator=gen(82), device=DEV)
    done = (torch.rand(B, K, generator=gen(83), device=DEV) < 0.3).int()
    rp, rt, rs, rd = ref_select(z, scores, done, K, V, K, 7)
    par = torch.empty(B, K, dtype=torch.int32, device=DEV)
    tok = torch.empty_like(par)
    ctx.reset()
    ctx.beam_select("fp32", z, scores, done, par, tok, scores, done, B, K, V, V, K, 7)
    ctx.sync()
    assert torch.equal(par, rp) and torch.equal(tok, rt) and torch.equal(done, rd)
    assert bool(((scores.double() - rs).abs() <= 1e-4 * 3 + U * rs.abs() * 1.01).all())


def test_beam_select_of_nearly_equal_beams(ctx):
    """Two beams with the same score and the same best tokens, whose
    distributions differ by 3e-4 under logits of a thousand: no tie."""
    V, n = 1000, 4
    z = torch.full((2, V), 1000.0, device=DEV)
    z[:, 5] = 1010.0
    z[:, 9] = 1009.0
    z[1, 100:110] = 900.0
    check_select(ctx, "fp32", z, torch.full((1, 2), -7.0, device=DEV), None, 2, V, n, -1)


@pytest.mark.parametrize("over", [False, True])
def test_beam_select_of_scores_that_are_not_finite(ctx, over):
    """Such beams offer -inf only, finished or not."""
    B, K, V, n = 2, 4, 700, 4
    z = make_logits("fp32", B * K, V, V, 84)
    scores = torch.tensor([[INF, -1.0, -2.0, math.nan], [-3.0, math.nan, INF, -2.5]], device=DEV)
    done = torch.full((B, K), int(over), dtype=torch.int32, device=DEV)
    par = torch.empty(B, n, dtype=torch.int32, device=DEV)
    tok, sc = par.clone(), torch.empty(B, n, device=DEV)
    ctx.reset()
    ctx.beam_select("fp32", z, scores, done, par, tok, sc, None, B, K, V, V, n, 3)
    ctx.sync()
    rp, rt, rs, _ = ref_select(z, torch.where(torch.isfinite(scores), scores, -INF), done, K, V, n, 3)
    assert torch.equal(par, rp) and torch.equal(tok, rt)
    fin = torch.isfinite(rs)
    assert torch.equal(fin, torch.isfinite(sc)) and not bool(torch.isnan(sc).any() | (sc == INF).any())


def check_reorder(ctx, state, parents, first, count):
    N, B, K, row = state.shape
    want = state.clone()
    for b in range(B):
        for j in range(K):
            want[:, b, j, first:first + count] = state[:, b, int(parents[b, j]), first:first + count]
    ctx.reset()
    ctx.beam_reorder(state, parents, N, B, K, row, first, count)
    ctx.sync()
    assert torch.equal(state, want)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8, 13, 16, 31, 32])
@pytest.mark.parametrize("row,first,count", [(4096, 0, 4096), (640, 64, 500), (36, 4, 20), (33, 5, 17), (7, 0, 7),
                                             (100000, 16, 99984), (64, 64, 0), (2, 0, 1)])
def test_beam_reorder(ctx, K, row, first, count):
    g = gen(90 + K)
    for N, B in ((1, 1), (3, 5)):
        state = torch.randint(0, 256, (N, B, K, row), generator=g, device=DEV, dtype=torch.uint8)
        for kind in range(3):
            if kind == 0:  # any mapping
                parents = torch.randint(0, K, (B, K), generator=g, device=DEV, dtype=torch.int32)
            elif kind == 1:  # one cycle
                parents = ((torch.arange(K, device=DEV, dtype=torch.int32) + 1) % K).repeat(B, 1)
            else:  # nothing moves
                parents = torch.arange(K, device=DEV, dtype=torch.int32).repeat(B, 1)
            check_reorder(ctx, state, parents.contiguous(), first, count)


def test_beam_reorder_past_32_bits(ctx):
    """Rows whose offsets pass 2^32 bytes."""
    N, B, K, row = 3, 1, 2, 1 << 30
    state = torch.zeros(N, B, K, row, dtype=torch.uint8, device=DEV)
    for n in range(N):
        state[n, 0, 0, -4096:] = 10 + n
        state[n, 0, 1, -4096:] = 20 + n
    parents = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    ctx.reset()
    ctx.beam_reorder(state, parents, N, B, K, row, row - 2048, 2048)
    ctx.sync()
    for n in range(N):
        assert bool((state[n, 0, 0, -2048:] == 20 + n).all()) and bool((state[n, 0, 1, -2048:] == 10 + n).all())
        assert bool((state[n, 0, 0, -4096:-2048] == 10 + n).all())


def test_beam_reorder_flags_a_bad_parent(ctx):
    state = torch.arange(4 * 64, device=DEV).to(torch.uint8).view(1, 1, 4, 64)
    want = state.clone()
    want[0, 0, 0] = state[0, 0, 3]
    for bad in (4, -1):
        s = state.clone()
        ctx.reset()
        ctx.beam_reorder(s, torch.tensor([[3, bad, 2, 3]], dtype=torch.int32, device=DEV), 1, 1, 4, 64, 0, 64)
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.sync()
        assert torch.equal(s, want)


# ---------------------------------------------------------------- refusals
def test_refusals(ctx):
    M, V, k = 4, 50, 5
    z = make_logits("fp32", M, V, V, 1)
    vals, idx, lse = make_lists(M, V, k, 2)
    row = torch.empty(M, device=DEV)
    y = torch.zeros(M, dtype=torch.int32, device=DEV)
    par = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    tok, sc = par.clone(), torch.zeros(2, 2, device=DEV)

    def top(**kw):
        a = dict(logits=z, vals=vals, idx=idx, lse=None, M=M, V=V, ld=V, k=k, tau=1.0)
        a.update(kw)
        ctx.top_logits("fp32", **a)

    def dis(**kw):
        a = dict(logits=z, t_vals=vals, t_idx=idx, t_lse=None, targets=y, dlogits=None, row_loss=row, mean_loss=None,
                 M=M, V=V, ld=V, k=k, alpha=0.5, tau=1.0, dscale=1.0)
        a.update(kw)
        ctx.distill("fp32", **a)

    def sel(**kw):
        a = dict(logits=z, scores=sc, done=None, parent=par, token=tok, out_scores=sc, out_done=None, B=2, K=2, V=V,
                 ld=V, n=2, eos=-1)
        a.update(kw)
        ctx.beam_select("fp32", **a)

    def reo(**kw):
        a = dict(state=z, parents=par, N=1, B=2, K=2, row_bytes=200, first=0, count=200)
        a.update(kw)
        ctx.beam_reorder(**a)

    ctx.reset()
    n0 = ctx.launches
    for call, bads in [
        (top, [dict(logits=None), dict(vals=None), dict(idx=None), dict(M=0), dict(V=0), dict(ld=V - 1), dict(k=0),
               dict(k=129, V=200, ld=200), dict(k=V + 1), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan),
               dict(tau=INF), dict(tau=1e-42), dict(V=1 << 20, ld=1 << 20)]),
        (dis, [dict(logits=None), dict(t_vals=None), dict(t_idx=None), dict(row_loss=None), dict(targets=None),
               dict(alpha=-0.1), dict(alpha=1.1), dict(alpha=math.nan), dict(tau=0.0), dict(k=0), dict(k=51),
               dict(M=-1), dict(ld=V - 1)]),
        (sel, [dict(logits=None), dict(scores=None), dict(parent=None), dict(token=None), dict(out_scores=None),
               dict(B=0), dict(K=0), dict(K=33), dict(n=0), dict(n=65), dict(n=7, K=2, V=3, ld=3), dict(eos=V),
               dict(eos=-2), dict(done=par), dict(ld=V - 1)]),
        (reo, [dict(state=None), dict(parents=None), dict(N=0), dict(B=0), dict(K=0), dict(K=33), dict(first=201),
               dict(count=201), dict(first=100, count=101)]),
    ]:
        for bad in bads:
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                call(**bad)
    with pytest.raises(api.TTError, match="TT_ERR_ARG"):
        ctx._check(api.lib().tt_op_top_logits(ctx.h, 7, z.data_ptr(), vals.data_ptr(), idx.data_ptr(), None, M, V, V, k,
                                              1.0))
    assert ctx.launches == n0
    for call, name in ((top, "logits"), (dis, "logits"), (dis, "dlogits"), (sel, "logits")):
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):  # off an element's boundary
            call(**{name: z.data_ptr() + 2})
    assert ctx.launches == n0
    with pytest.raises(ValueError, match="contiguous"):
        top(logits=make_logits("fp32", M, V, 2 * V, 1)[:, ::2])
    small = api.Context(256)  # 4 rows of 50 entries need 1632 bytes
    p64, s64 = torch.zeros(2, 64, dtype=torch.int32, device=DEV), torch.zeros(2, 64, device=DEV)
    with pytest.raises(api.TTError, match="TT_ERR_ARENA_OOM"):
        small.beam_select("fp32", z, sc, None, p64, p64.clone(), s64, None, 2, 2, V, V, 64, -1)
    small.close()
    ctx.sync()


# ---------------------------------------------------------------- together
def test_recorded_calls_replay(ctx):
    """The calls of one search step and one distillation, recorded and replayed
    on changed inputs, give what the calls give."""
    B, K, V, n = 2, 3, 3001, 3
    z = make_logits("bf16", B * K, V, V, 91)
    scores = torch.randn(B, K, generator=gen(92), device=DEV)
    par = torch.empty(B, n, dtype=torch.int32, device=DEV)
    tok, sc = torch.empty_like(par), torch.empty(B, n, device=DEV)
    state = torch.randint(0, 256, (2, B, K, 320), generator=gen(93), device=DEV, dtype=torch.uint8)
    vals, idx, lse = make_lists(B * K, V, 8, 94)
    tv, ti, tl = torch.empty_like(vals), torch.empty_like(idx), torch.empty_like(lse)
    row, mean, d = torch.empty(B * K, device=DEV), torch.empty(1, device=DEV), torch.empty_like(z)
    stream = torch.cuda.Stream()

    with api.Context(8 << 20, stream=stream.cuda_stream) as c:
        def calls():
            c.beam_select("bf16", z, scores, None, par, tok, sc, None, B, K, V, V, n)
            c.beam_reorder(state, par, 2, B, K, 320, 32, 256)
            c.top_logits("bf16", z, tv, ti, tl, B * K, V, V, 8, 2.0)
            c.distill("bf16", z, tv, ti, tl, None, d, row, mean, B * K, V, V, 8, 1.0, 3.0, 1.0)

        torch.cuda.synchronize()
        start = state.clone()
        c.record(calls)
        z.copy_(make_logits("bf16", B * K, V, V, 95))
        scores.copy_(torch.randn(B, K, generator=gen(96), device=DEV))
        torch.cuda.synchronize()
        c.replay(1)
        c.sync()
        got = [x.clone() for x in (par, tok, sc, state, tv, ti, tl, row, mean, d)]
        for x in (par, tok, sc, tv, ti, tl, row, mean, d):
            x.zero_()
        state.copy_(start)
        torch.cuda.synchronize()
        calls()
        c.sync()
        for a, b in zip(got, (par, tok, sc, state, tv, ti, tl, row, mean, d)):
            assert torch.equal(a, b)


def test_a_recording_keeps_its_scratch(ctx):
    """What is allocated after a recording is not written over by its replay."""
    V = 50257
    z = make_logits("fp32", 8, V, V, 97)
    scores = torch.zeros(2, 4, device=DEV)
    par, tok = torch.empty(2, 4, dtype=torch.int32, device=DEV), torch.empty(2, 4, dtype=torch.int32, device=DEV)
    sc, tv, ti = torch.empty(2, 4, device=DEV), torch.empty(8, 9, device=DEV), torch.empty(8, 9, dtype=torch.int32, device=DEV)
    with api.Context(16 << 20, stream=torch.cuda.Stream().cuda_stream) as c:
        def calls():
            c.beam_select("fp32", z, scores, None, par, tok, sc, None, 2, 4, V, V, 4)
            c.top_logits("fp32", z, tv, ti, None, 8, V, V, 9)

        torch.cuda.synchronize()
        c.record(calls)
        node = c.tensor(1 << 20)
        node.fill(np.full(1 << 20, 3.0, dtype=np.float32))
        c.replay(2)
        assert np.all(node.numpy() == 3.0)
        rp, rt, _, _ = ref_select(z, scores, None, 4, V, 4, -1)
        assert torch.equal(par, rp) and torch.equal(tok, rt)
        assert np.array_equal(ti.cpu().numpy(), ref_top(z, V, 9, 1.0)[1])


def test_two_contexts_at_once(ctx):
    """Two contexts on two streams, calls interleaved: each gets its own results."""
    V, B, K = 50257, 2, 4
    streams = [torch.cuda.Stream() for _ in range(2)]
    ctxs = [api.Context(8 << 20, stream=s.cuda_stream) for s in streams]
    zs = [make_logits("bf16", B * K, V, 50304, 101 + i) for i in range(2)]
    scores = torch.randn(B, K, generator=gen(103), device=DEV)
    outs = [[torch.empty(B, K, dtype=torch.int32, device=DEV), torch.empty(B, K, dtype=torch.int32, device=DEV),
             torch.empty(B, K, device=DEV)] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, z, o in zip(ctxs, zs, outs):
            c.beam_select("bf16", z, scores, None, o[0], o[1], o[2], None, B, K, V, 50304, K)
    for c, z, o in zip(ctxs, zs, outs):
        c.sync()
        rp, rt, _, _ = ref_select(z, scores, None, K, V, K, -1)
        assert torch.equal(o[0], rp) and torch.equal(o[1], rt)
        c.close()


# ---------------------------------------------------------------- the model's paths
def plain_gpt2(sh, flat, tok):
    """GPT-2's logits [B, T, V] in 64 bits from the flat parameter vector (a
    float64 torch tensor), in elementary operations."""
    at = [0]

    def take(*shape):
        n = math.prod(shape)
        x = flat[at[0]:at[0] + n].view(*shape)
        at[0] += n
        return x

    def ln(x, w, b):
        m = x.mean(-1, keepdim=True)
        v = ((x - m) ** 2).mean(-1, keepdim=True)
        return (x - m) / torch.sqrt(v + 1e-5) * w + b

    C, H = sh.C, sh.H
    B, T = tok.shape
    wte, wpe = take(sh.V, C), take(sh.maxT, C)
    x = wte[tok.long()] + wpe[:T]
    hide = torch.ones(T, T, dtype=torch.bool).triu(1)
    for _ in range(sh.L):
        l1w, l1b, qw, qb = take(C), take(C), take(3 * C, C), take(3 * C)
        pw, pb, l2w, l2b = take(C, C), take(C), take(C), take(C)
        fw, fb, gw, gb = take(4 * C, C), take(4 * C), take(C, 4 * C), take(C)
        q, k, v = ((ln(x, l1w, l1b) @ qw.T + qb).view(B, T, 3, H, C // H).permute(2, 0, 3, 1, 4))
        s = (q @ k.transpose(-1, -2) / math.sqrt(C // H)).masked_fill(hide, -INF)
        a = (torch.softmax(s, -1) @ v).transpose(1, 2).reshape(B, T, C)
        x = x + a @ pw.T + pb
        u = ln(x, l2w, l2b) @ fw.T + fb
        u = 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
        x = x + u @ gw.T + gb
    return ln(x, take(C), take(C)) @ wte.T


def host_values(oracle, p, dtype):
    return {"bf16": oracle.bf16_values, "fp16": oracle.f16_values}.get(dtype, lambda x: x.astype(np.float64))(p)


def device_params(c, sh, p, dtype):
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, dtype)
    c.set_model(cfg)
    master = torch.from_numpy(p).to(DEV)
    if dtype == "fp32":
        return cfg, master
    low = torch.empty(p.size, device=DEV, dtype=TYPES[dtype])
    (c.cast_bf16 if dtype == "bf16" else c.cast_f16)(master, low)
    return cfg, low


@pytest.mark.parametrize("name,B,T,dtype,tol", [("tiny_fp32", 3, 17, "fp32", 1e-4), ("char_bf16", 3, 33, "bf16", 2e-2),
                                                ("char_bf16", 3, 33, "fp16", 2.5e-3)])
@pytest.mark.parametrize("rest,alpha", [(True, 0.5), (False, 1.0)])
def test_teacher_and_student_step(oracle, name, B, T, dtype, tol, rest, alpha):
    """The teacher's lists from tt_gpt2_top_logits, then the student's step on
    them: lists, loss and every parameter's gradient against 64 bits on the
    same lists.  The bounds are the step's own (rel-L2 1e-4 in fp32, 2e-2 in
    bf16, an eighth of that in half)."""
    native_build.build()
    sh = synth.WORKLOADS[name].shape
    k, tau, M = 12, 2.0, B * T
    tok, tgt = synth.token_stream(B, T, sh.V, "uniform", seed=3)
    tgt[0, :5] = -1
    tok_d, tgt_d = torch.from_numpy(tok).to(DEV), torch.from_numpy(tgt).to(DEV)
    pt = synth.init_params(sh, seed=5, std=0.1, jitter=0.05)
    ps = synth.init_params(sh, seed=6, std=0.02, jitter=0.05)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, dtype)
    with api.Context(2 * api.arena_bytes(cfg, B, T) + (1 << 20)) as c:
        _, wt = device_params(c, sh, pt, dtype)
        vals, lse = torch.empty(M, k, device=DEV), torch.empty(M, device=DEV)
        idx = torch.empty(M, k, dtype=torch.int32, device=DEV)
        c.reset()
        c.top_logits_of(wt, tok_d, B, T, k, vals, idx, lse, tau)
        with pytest.raises(api.TTError, match="TT_ERR_STATE"):
            c.loss_device()
        c.sync()
        zt = plain_gpt2(sh, torch.from_numpy(host_values(oracle, pt, dtype)), torch.from_numpy(tok)).view(M, sh.V)
        near = {"fp32": 1e-4, "bf16": 8e-2, "fp16": 1e-2}[dtype] * float(zt.abs().max())
        assert float((zt.gather(1, idx.cpu().long()) - vals.cpu().double()).abs().max()) <= near
        assert float((zt.sort(1, descending=True).values[:, :k] - vals.cpu().double()).abs().max()) <= near

        _, ws = device_params(c, sh, ps, dtype)
        grads = torch.full((ps.size,), math.nan, device=DEV)
        scale = torch.tensor([1024.0], device=DEV) if dtype == "fp16" else None
        targets = tgt_d if alpha < 1 else None
        c.reset()
        loss = c.step_distill(ws, grads, tok_d, targets, vals, idx, lse if rest else None, k, alpha, tau, B, T,
                              loss_scale=scale)
        flat = torch.from_numpy(host_values(oracle, ps, dtype)).requires_grad_(True)
        z = plain_gpt2(sh, flat, torch.from_numpy(tok)).view(M, sh.V)
        ref = ref_distill(z, sh.V, vals.cpu(), idx.cpu(), lse.cpu() if rest else None,
                          torch.from_numpy(tgt).view(-1) if alpha < 1 else None, alpha, tau).mean()
        (g,) = torch.autograd.grad(ref, flat)
        ref = ref.detach()
        assert abs(loss - float(ref)) <= tol * abs(float(ref)), (loss, float(ref))
        got = grads.double().cpu() / (1024.0 if scale is not None else 1.0)
        for i, (tname, n, _) in enumerate(synth.param_table(sh)):
            a = sum(t[1] for t in synth.param_table(sh)[:i])
            x, y = got[a:a + n], g[a:a + n]
            assert float((x - y).norm()) <= tol * float(y.norm()) + 1e-9, tname
        # host token buffers, and accumulation: twice the gradient
        first = grads.clone()
        c.reset()
        assert c.step_distill(ws, grads, tok, tgt if alpha < 1 else None, vals, idx, lse if rest else None, k, alpha, tau,
                              B, T, accumulate=True, loss_scale=scale) == loss
        assert float((grads.double() - 2 * first.double()).norm()) <= 1e-6 * float(first.double().norm()) * 2
        # a loop of updates on it
        m, v = torch.zeros(ps.size, device=DEV), torch.zeros(ps.size, device=DEV)
        master = torch.from_numpy(ps).to(DEV)
        for step in range(1, 4):
            c.reset()
            c.step_distill(ws, grads, tok_d, targets, vals, idx, lse if rest else None, k, alpha, tau, B, T,
                           loss_scale=scale, sync=False)
            c.adamw(master, None if dtype == "fp32" else ws, grads, m, v, 1e-4, 0.9, 0.95, 1e-8, 0.1, step)
        c.sync()
        assert bool(torch.isfinite(master).all())


def test_step_distill_of_hard_labels_is_the_step(ctx, oracle):
    """One entry per position, the target, at tau 1: the distillation loss is
    the cross entropy."""
    sh = synth.WORKLOADS["tiny_fp32"].shape
    B, T = 4, 32
    p = synth.init_params(sh, jitter=0.05)
    tok, tgt = synth.token_stream(B, T, sh.V, "uniform")
    rl, rg, _ = oracle.gpt2_step(sh, p.astype(np.float64), tok, tgt)
    _, w = device_params(ctx, sh, p, "fp32")
    grads = torch.empty(p.size, device=DEV)
    idx = torch.from_numpy(tgt).to(DEV).view(-1, 1).contiguous()
    vals = torch.zeros(B * T, 1, device=DEV)
    ctx.reset()
    loss = ctx.step_distill(w, grads, tok, None, vals, idx, None, 1, 1.0, 1.0, B, T)
    assert abs(loss - rl) <= 1e-5 * abs(rl)
    assert np.linalg.norm(grads.cpu().numpy() - rg) <= 1e-4 * np.linalg.norm(rg)


def test_step_distill_refusals(ctx):
    sh = synth.WORKLOADS["tiny_fp32"].shape
    p = synth.init_params(sh)
    _, w = device_params(ctx, sh, p, "fp32")
    B, T, k = 2, 8, 4
    tok, tgt = synth.token_stream(B, T, sh.V, "uniform")
    vals, idx, lse = make_lists(B * T, sh.V, k, 1)
    grads = torch.empty(p.size, device=DEV)
    base = dict(params=w, grads=grads, tokens=tok, targets=tgt, t_vals=vals, t_idx=idx, t_lse=lse, k=k, alpha=0.5,
                tau=1.0, B=B, T=T)
    ctx.reset()
    for bad in [dict(params=None), dict(grads=None), dict(tokens=None), dict(targets=None), dict(t_vals=None),
                dict(t_idx=None), dict(k=0), dict(k=129), dict(alpha=2.0), dict(tau=0.0), dict(B=0), dict(T=33)]:
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.step_distill(**{**base, **bad})
    for bad in [dict(k=0), dict(k=200), dict(tau=-1.0), dict(vals=None), dict(T=33)]:
        a = dict(params=w, tokens=tok, B=B, T=T, k=k, vals=vals, idx=idx, lse=lse, tau=1.0)
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.top_logits_of(**{**a, **bad})
    t2 = tgt.copy()
    t2[1, 1] = sh.V
    ctx.reset()
    with pytest.raises(api.TTError, match="TT_ERR_ARG"):
        ctx.step_distill(**{**base, "targets": t2})
    ctx.reset()
    assert math.isfinite(ctx.step_distill(**base))


def test_model_lists_in_host_memory_are_refused(ctx):
    sh = synth.WORKLOADS["tiny_fp32"].shape
    p = synth.init_params(sh)
    _, w = device_params(ctx, sh, p, "fp32")
    B, T, k = 2, 8, 4
    tok, tgt = synth.token_stream(B, T, sh.V, "uniform")
    lists = dict(zip(("vals", "idx", "lse"), make_lists(B * T, sh.V, k, 1)))
    grads = torch.empty(p.size, device=DEV)
    ctx.reset()
    n0 = ctx.launches
    for name in lists:
        a = {**lists, name: lists[name].cpu()}
        with pytest.raises(api.TTError, match="device memory"):
            ctx.step_distill(w, grads, tok, tgt, a["vals"], a["idx"], a["lse"], k, 0.5, 1.0, B, T)
        with pytest.raises(api.TTError, match="device memory"):
            ctx.top_logits_of(w, tok, B, T, k, a["vals"], a["idx"], a["lse"])
    assert ctx.launches == n0


def ref_beam(oracle, sh, po, prompt, n_new, K, eos):
    """Plain beam search on the oracle's logits: sequences, scores, and the
    smallest gap between kept and dropped or between neighbours."""
    outs, scs, gap = [], [], INF
    for b in range(prompt.shape[0]):
        hyps = [(list(prompt[b]), 0.0, False)]
        for _ in range(n_new):
            z = oracle.gpt2_logits_last(sh, po, np.array([h[0] for h in hyps], dtype=np.int32))
            cand = []
            for j, (seq, s, over) in enumerate(hyps):
                if over:
                    cand.append((s, j * sh.V + eos, seq + [eos], True))
                    continue
                m = z[j].max()
                lp = z[j] - m - math.log(np.exp(z[j] - m).sum())
                for v in np.argsort(-lp, kind="stable")[:K + 1]:
                    cand.append((s + lp[v], j * sh.V + int(v), seq + [int(v)], int(v) == eos))
            cand.sort(key=lambda c: (-c[0], c[1]))
            top = [c[0] for c in cand[:K + 1]]
            gap = min([gap] + [a - c for a, c in zip(top, top[1:])])
            hyps = [(c[2], c[0], c[3]) for c in cand[:K]]
        outs.append([h[0] for h in hyps])
        scs.append([h[1] for h in hyps])
    return np.array(outs, dtype=np.int32), np.array(scs), gap


@pytest.mark.parametrize("name,B,Tp,n_new,K,use_eos,seed", [
    ("tiny_fp32", 2, 5, 10, 4, False, 11), ("tiny_fp32", 3, 3, 12, 3, True, 11), ("char_bf16", 1, 140, 6, 8, False, 11),
    ("tiny_fp32", 7, 4, 6, 5, True, 24)])
def test_generate_beam_matches_a_plain_search(oracle, name, B, Tp, n_new, K, use_eos, seed):
    """fp32 mode, weights at ten times the init scale (logits well apart): the
    same hypotheses in the same order, and scores within fp32's error of the
    model (1e-5 of the largest logit a step, as the greedy test's).  The seeds
    are ones whose candidates the oracle finds further apart than that."""
    native_build.build()
    sh = synth.WORKLOADS[name].shape
    p = synth.init_params(sh, std=0.2, jitter=0.05)
    prompt, _ = synth.token_stream(B, Tp, sh.V, "uniform", seed=seed)
    po = p.astype(np.float64)
    eos = -1
    if use_eos:  # a token that the search takes early on
        free, _, _ = ref_beam(oracle, sh, po, prompt, 3, K, -1)
        eos = int(free[0, 0, Tp + 1])
    want, ws, gap = ref_beam(oracle, sh, po, prompt, n_new, K, eos)
    zmax = float(np.abs(oracle.gpt2_logits_last(sh, po, prompt)).max())
    assert gap > 2e-5 * zmax * n_new, "the inputs leave a tie"
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, "fp32")
    need = api.generate_beam_arena_bytes(cfg, B, Tp, n_new, K)
    with api.Context(need) as c:
        _, w = device_params(c, sh, p, "fp32")
        out = np.full((B, K, Tp + n_new), -1, dtype=np.int32)
        sc = np.full((B, K), 9.0, dtype=np.float32)
        c.reset()
        c.generate_beam(w, prompt, B, Tp, n_new, K, out, sc, eos)
        assert c.high_water <= need
        assert np.array_equal(out, want)
        assert np.abs(sc - ws).max() <= 2e-5 * zmax * n_new
        out_d = torch.zeros(B, K, Tp + n_new, dtype=torch.int32, device=DEV)
        sc_d = torch.zeros(B, K, device=DEV)
        c.reset()
        c.generate_beam(w, torch.from_numpy(prompt).to(DEV), B, Tp, n_new, K, out_d, sc_d, eos)
        assert np.array_equal(out_d.cpu().numpy(), out) and np.array_equal(sc_d.cpu().numpy(), sc)


@pytest.mark.parametrize("name,B,Tp,n_new,dtype", [("tiny_fp32", 3, 5, 12, "fp32"), ("char_bf16", 4, 16, 24, "bf16"),
                                                   ("char_bf16", 20, 8, 9, "bf16")])
def test_one_beam_is_greedy(oracle, name, B, Tp, n_new, dtype):
    """K = 1 takes greedy's tokens."""
    native_build.build()
    sh = synth.WORKLOADS[name].shape
    p = synth.init_params(sh, std=0.2, jitter=0.05)
    prompt, _ = synth.token_stream(B, Tp, sh.V, "uniform", seed=7)
    with api.Context(256 << 20) as c:
        _, w = device_params(c, sh, p, dtype)
        want = np.zeros((B, Tp + n_new), dtype=np.int32)
        c.reset()
        c.generate(w, prompt, B, Tp, n_new, want)
        out, sc = np.zeros((B, 1, Tp + n_new), dtype=np.int32), np.zeros((B, 1), dtype=np.float32)
        c.reset()
        c.generate_beam(w, prompt, B, Tp, n_new, 1, out, sc)
        assert np.array_equal(out[:, 0], want)
        assert np.all(sc < 0) and np.all(np.isfinite(sc))


def test_generate_beam_bf16_scores_are_those_of_its_tokens(oracle):
    """bf16, more rows than the few-row linear layers take: hypotheses differ,
    are ordered, and each score is the oracle's log probability of its tokens
    within bf16's error of the logits (3e-2 of the largest a step, as greedy)."""
    native_build.build()
    sh = synth.WORKLOADS["char_bf16"].shape
    B, Tp, n_new, K = 4, 12, 10, 6
    p = synth.init_params(sh, std=0.02, jitter=0.05)
    prompt, _ = synth.token_stream(B, Tp, sh.V, "zipf", seed=5)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, "bf16")
    po = oracle.bf16_values(p)
    with api.Context(api.generate_beam_arena_bytes(cfg, B, Tp, n_new, K)) as c:
        _, w = device_params(c, sh, p, "bf16")
        out, sc = np.zeros((B, K, Tp + n_new), dtype=np.int32), np.zeros((B, K), dtype=np.float32)
        c.reset()
        c.generate_beam(w, prompt, B, Tp, n_new, K, out, sc)
    flat = out.reshape(B * K, -1)
    total, size = np.zeros(B * K), 0.0
    for t in range(Tp, Tp + n_new):
        z = oracle.gpt2_logits_last(sh, po, np.ascontiguousarray(flat[:, :t]))
        m = z.max(1)
        total += z[np.arange(B * K), flat[:, t]] - m - np.log(np.exp(z - m[:, None]).sum(1))
        size = max(size, float(np.abs(z).max()))
    assert np.abs(total.reshape(B, K) - sc).max() <= n_new * (3e-2 * size + 1e-3)
    assert np.all(np.diff(sc, axis=1) <= 0)
    for b in range(B):
        assert len({tuple(h) for h in out[b]}) == K
        assert np.array_equal(out[b, :, :Tp], np.repeat(prompt[b][None], K, 0))


def test_generate_beam_edges_and_errors(ctx):
    sh = synth.WORKLOADS["tiny_fp32"].shape
    p = synth.init_params(sh)
    cfg, w = device_params(ctx, sh, p, "fp32")
    prompt = np.arange(6, dtype=np.int32).reshape(2, 3)
    out, sc = np.full((2, 2, 3), -1, dtype=np.int32), np.full((2, 2), 5.0, dtype=np.float32)
    ctx.reset()
    ctx.generate_beam(w, prompt, 2, 3, 0, 2, out, sc)
    assert np.array_equal(out, np.repeat(prompt[:, None], 2, 1)) and np.all(sc == 0)
    one = np.zeros((2, 32, 4), dtype=np.int32)
    s1 = np.zeros((2, 32), dtype=np.float32)
    ctx.reset()
    ctx.generate_beam(w, prompt, 2, 3, 1, 32, one, s1)  # one step: the 32 likeliest tokens
    assert all(len(set(one[b, :, 3])) == 32 for b in range(2)) and np.all(np.diff(s1, axis=1) <= 0)
    big, bs = np.zeros((2, 40, sh.maxT + 1), dtype=np.int32), np.zeros((2, 40), dtype=np.float32)
    for args in [(2, 3, sh.maxT, 2), (0, 3, 1, 2), (2, 0, 1, 2), (2, 3, -1, 2), (2, 3, 1, 0), (2, 3, 1, 33)]:
        ctx.reset()
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.generate_beam(w, prompt, *args, big, bs)
        assert api.generate_beam_arena_bytes(cfg, *args) == 0
    for eos in (-2, sh.V):
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            ctx.generate_beam(w, prompt, 2, 3, 1, 2, big, bs, eos)
    bad = prompt.copy()
    bad[1, 2] = sh.V
    ctx.reset()
    with pytest.raises(api.TTError, match="TT_ERR_ARG"):
        ctx.generate_beam(w, bad, 2, 3, 2, 2, np.zeros((2, 2, 5), dtype=np.int32), np.zeros((2, 2), dtype=np.float32))
    small = api.Context(1 << 12)
    device_params(small, sh, p, "fp32")
    with pytest.raises(api.TTError, match="TT_ERR_ARENA_OOM"):
        small.generate_beam(w, prompt, 2, 3, 2, 2, big, bs)
    small.close()
    ctx.reset()
    ctx.generate_beam(w, prompt, 2, 3, 2, 2, np.zeros((2, 2, 5), dtype=np.int32), np.zeros((2, 2), dtype=np.float32))
