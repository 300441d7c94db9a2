"""The model's steps on answers (tt_gpt2_logprobs, tt_gpt2_step_policy,
tt_gpt2_step_preference) over sequences and over groups, against a GPT-2 in 64
bits that computes every answer as a sequence of its own.

The bounds are the step's own: loss and every parameter's gradient within 1e-4
(rel-L2) in fp32, 2e-2 in bf16, an eighth of that in half."""
import math

import pytest
import torch

from autograd_arena_allocated_gb300 import api, synth
from autograd_arena_allocated_gb300 import build as native_build
from test_gpu_head import DEV, device_params, host_values, plain_gpt2

pytestmark = pytest.mark.gpu
TOL = {"fp32": 1e-4, "bf16": 2e-2, "fp16": 2.5e-3}

# starts: prompt's end, then the answers' ends; the tiny model has 32 positions,
# the character model 256, which the groups' own lengths exceed
GROUPS = {
    "tiny_fp32": (70, [[12, 30, 32, 32, 50], [0, 20, 40, 60, 70], [31, 32, 32, 32, 33]]),
    "char_bf16": (330, [[100, 180, 330], [200, 256, 257]]),
}


def batch(name, grouped, seed):
    """tokens, labels, starts (or None), and per answer its rows and the positions that it sees"""
    sh = synth.WORKLOADS[name].shape
    T, starts = GROUPS[name]
    if not grouped:
        T = min(sh.maxT, 40)
        starts = [[0, T]] * 4
    B = len(starts)
    g = torch.Generator().manual_seed(seed)
    tok = torch.randint(0, sh.V, (B, T), generator=g, dtype=torch.int32)
    tgt = torch.full((B, T), -1, dtype=torch.int32)
    answers = []
    for b, s in enumerate(starts):
        for a, e in zip(s, s[1:]):
            first = a if grouped else a + 7  # sequences: the prompt is their first part
            if first < e:
                tgt[b, first:e - 1] = tok[b, first + 1:e]
                tgt[b, e - 1] = 1
            answers.append((b * T + first, b * T + max(e, first), list(range(s[0])) + list(range(a, e)), b))
        if grouped:
            tok[b, s[-1]:] = -7  # not used
    return tok, tgt, (torch.tensor(starts, dtype=torch.int32) if grouped else None), answers


def plain_logits(sh, flat, tok, answers):
    """[B * T, V]: every labelled row's logits, an answer at a time; zeros elsewhere"""
    B, T = tok.shape
    rows, vals = [], []
    for first, last, seen, b in answers:
        if first >= last:
            continue
        z = plain_gpt2(sh, flat, tok[b, seen][None])[0]
        rows.append(torch.arange(first, last))
        vals.append(z[-(last - first):])
    return torch.zeros(B * T, sh.V, dtype=torch.float64).index_put((torch.cat(rows),), torch.cat(vals))


def labelled(z, tgt, tau):
    y = tgt.view(-1)
    lp = torch.log_softmax(z / tau, 1).gather(1, y.clamp(min=0).long()[:, None])[:, 0]
    return torch.where(y >= 0, lp, 0.0)


def policy_loss(lp, on, old, ref, adv, w, lo, hi, beta):
    r, x = torch.exp(lp - old), ref - lp
    l = -torch.minimum(r * adv, r.clamp(1 - lo, 1 + hi) * adv) + beta * (torch.exp(x) - x - 1)
    return torch.where(on, w * l, 0.0).mean()


def pair_loss(lp, ref, on, spans, beta, gamma, smooth, mean):
    """the pairs' v and losses, and the answers' sums"""
    s, total = [], []
    for a, b in spans.tolist():
        n = max(int(on[a:b].sum()), 1) if mean else 1
        s.append(torch.where(on[a:b], lp[a:b] - ref[a:b], 0.0).sum() / n)
        total.append(torch.where(on[a:b], lp[a:b], 0.0).sum())
    v = beta * (torch.stack(s[0::2]) - torch.stack(s[1::2])) - gamma
    f = torch.nn.functional.logsigmoid
    return v, -(1 - smooth) * f(v) - smooth * f(-v), torch.stack(total)


def pair_slope(seq, ref, on, spans, beta, gamma, smooth, mean):
    """d loss / d v at the sums that the call reports: rounded activations move
    an answer's sum by the tokens' errors added up, and the slope with it, which
    is not the gradient's error (the sums are compared by themselves)"""
    lp = torch.zeros_like(ref)
    for (a, b), x in zip(spans.tolist(), seq.tolist()):
        n = int(on[a:b].sum())
        if n:
            lp[a:b] = torch.where(on[a:b], x / n, 0.0)
    v = pair_loss(lp, ref, on, spans, beta, gamma, smooth, mean)[0]
    return smooth * torch.sigmoid(v) - (1 - smooth) * torch.sigmoid(-v)


def check_grads(sh, got, want, tol):
    at = 0
    for name, n, _ in synth.param_table(sh):
        x, y = got[at:at + n], want[at:at + n]
        assert float((x - y).norm()) <= tol * float(y.norm()) + 1e-9, (name, float((x - y).norm() / y.norm()))
        at += n


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("name,dtype", [("tiny_fp32", "fp32"), ("char_bf16", "bf16"), ("char_bf16", "fp16"),
                                        ("tiny_fp32", "fp16")])
def test_steps_on_answers(oracle, name, dtype, grouped):
    native_build.build()
    sh = synth.WORKLOADS[name].shape
    tol, tau = TOL[dtype], 1.3
    tok, tgt, starts, answers = batch(name, grouped, 3)
    B, T = tok.shape
    M, K = B * T, 0 if starts is None else starts.shape[1] - 1
    p = synth.init_params(sh, seed=6, std=0.05, jitter=0.05)
    flat = torch.from_numpy(host_values(oracle, p, dtype)).requires_grad_(True)
    lp = labelled(plain_logits(sh, flat, tok, answers), tgt, tau)
    on = tgt.view(-1) >= 0
    g = torch.Generator().manual_seed(4)
    d = 0.3 * torch.randn(M, generator=g)
    lo, hi, beta = 0.2, 0.3, 0.1
    for edge in (math.log1p(-lo), math.log1p(hi)):  # no ratio next to a bound
        d = torch.where((d - edge).abs() < 0.06, edge + 0.07, d)
    f32 = lambda x: x.detach().float().to(DEV)  # noqa: E731
    old, ref = f32(lp - d), f32(lp + 0.4 * torch.randn(M, generator=g))
    adv = (torch.randn(M, generator=g) + 1.0).to(DEV)
    w = (0.5 + torch.rand(M, generator=g)).to(DEV)
    host = lambda x: x.cpu().double()  # noqa: E731
    tok_d, tgt_d, st_d = tok.to(DEV), tgt.to(DEV), None if starts is None else starts.to(DEV)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, dtype)
    with api.Context(api.answers_arena_bytes(cfg, B, T, K)) as c:
        _, ws = device_params(c, sh, p, dtype)
        scale = torch.tensor([1024.0], device=DEV) if dtype == "fp16" else None
        unscale = 1024.0 if scale is not None else 1.0

        # the log probabilities
        out, lse = torch.full((M,), 7.0, device=DEV), torch.full((M,), 7.0, device=DEV)
        c.reset()
        c.logprobs_of(ws, tok_d, tgt_d, B, T, out, lse, tau, st_d, K)
        with pytest.raises(api.TTError, match="TT_ERR_STATE"):
            c.loss_device()
        c.sync()
        near = {"fp32": 1e-4, "bf16": 8e-2, "fp16": 1e-2}[dtype]
        assert float((host(out) - lp.detach()).abs().max()) <= near * float(lp.detach().abs().max())
        assert not out.cpu()[~on].any() and not lse.cpu()[~on].any()

        # policy
        grads = torch.full((p.size,), math.nan, device=DEV)
        got_lp = torch.empty(M, device=DEV)
        args = dict(B=B, T=T, tau=tau, starts=st_d, K=K, loss_scale=scale)
        pol = (old, ref, adv, w, lo, hi, beta)
        c.reset()
        loss = c.step_policy(ws, grads, tok_d, tgt_d, *pol, logp=got_lp, **args)
        want = policy_loss(lp, on, host(old), host(ref), host(adv), host(w), lo, hi, beta)
        (want_g,) = torch.autograd.grad(want, flat, retain_graph=True)
        assert abs(loss - float(want.detach())) <= tol * abs(float(want.detach()))
        assert torch.equal(got_lp, out)
        check_grads(sh, host(grads) / unscale, want_g, tol)
        rows = c.row_losses(torch.empty(M))
        assert abs(float(rows.double().mean()) - loss) <= 1e-5 * abs(loss) and not rows[~on].any()
        # host tokens and targets, accumulation: the same loss, twice the gradient
        first = grads.clone()
        c.reset()
        assert c.step_policy(ws, grads, tok, tgt, *pol, accumulate=True, **args) == loss
        assert float((grads.double() - 2 * first.double()).norm()) <= 2e-6 * float(first.double().norm())
        # the same bits again
        c.reset()
        assert c.step_policy(ws, grads, tok_d, tgt_d, *pol, **args) == loss and torch.equal(grads, first)

        # pairs: the answers two by two (an odd last one is left out)
        pairs = len(answers) // 2
        spans = torch.tensor([[a[0], a[1]] for a in answers[:2 * pairs]], dtype=torch.int32)
        for opt in (dict(beta=0.2, gamma=0.1, smoothing=0.1, mean=False), dict(beta=3.0, gamma=0.0, smoothing=0.0, mean=True)):
            seq = torch.empty(2 * pairs, device=DEV)
            c.reset()
            loss = c.step_preference(ws, grads, tok_d, tgt_d, ref, spans.to(DEV), pairs, seq_logp=seq, **opt, **args)
            a = (opt["beta"], opt["gamma"], opt["smoothing"], opt["mean"])
            vv, each, total = pair_loss(lp, host(ref), on, spans, *a)
            assert abs(loss - float(each.detach().mean())) <= tol * float(each.detach().mean())
            assert float((host(seq) - total.detach()).abs().max()) <= near * float(total.detach().abs().max())
            slope = pair_slope(host(seq), host(ref), on, spans, *a)
            (want_g,) = torch.autograd.grad((slope * vv).mean(), flat, retain_graph=True)
            check_grads(sh, host(grads) / unscale, want_g, tol)
            got = c.row_losses(torch.empty(pairs))
            assert abs(float(got.double().mean()) - loss) <= 1e-5 * loss
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                c.row_losses(torch.empty(pairs + 1))

        # together: old and reference log probabilities from the model itself, then updates on them
        master = torch.from_numpy(p).to(DEV)
        m, v = torch.zeros(p.size, device=DEV), torch.zeros(p.size, device=DEV)
        c.reset()
        c.logprobs_of(ws, tok_d, tgt_d, B, T, out, None, tau, st_d, K)
        losses = []
        for step in range(1, 5):
            c.reset()
            losses.append(c.step_policy(ws, grads, tok_d, tgt_d, out, out, adv, None, lo, hi, beta, **args))
            if scale is not None:
                grads /= 1024.0
            c.adamw(master, None if dtype == "fp32" else ws, grads, m, v, 1e-4, 0.9, 0.95, 1e-8, 0.0, step)
            if dtype == "fp32":
                ws.copy_(master)
        c.sync()
        # on policy: ratios of 1 and no distance, so the first loss is the mean of -adv
        first = -float(torch.where(on, host(adv), 0.0).mean())
        assert abs(losses[0] - first) <= 1e-5 * abs(first)
        assert all(math.isfinite(x) for x in losses) and bool(torch.isfinite(master).all())


def test_one_answer_groups_are_the_sequences(oracle):
    """Groups of one answer without a prompt or padding are the plain batch, bit for bit in bf16."""
    sh = synth.WORKLOADS["char_bf16"].shape
    tok, tgt, _, _ = batch("char_bf16", False, 9)
    B, T = tok.shape
    p = synth.init_params(sh, seed=7, std=0.05, jitter=0.05)
    adv = torch.randn(B * T, generator=torch.Generator().manual_seed(1)).to(DEV)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, "bf16")
    with api.Context(api.answers_arena_bytes(cfg, B, T, 1)) as c:
        _, ws = device_params(c, sh, p, "bf16")
        out = []
        for st, K in ((None, 0), (torch.tensor([[0, T]] * B, dtype=torch.int32, device=DEV), 1),
                      (torch.tensor([[5, T]] * B, dtype=torch.int32, device=DEV), 1)):
            g = torch.empty(p.size, device=DEV)
            c.reset()
            loss = c.step_policy(ws, g, tok, tgt, None, None, adv, None, 0.2, 0.2, 0.0, B=B, T=T, starts=st, K=K)
            out.append((loss, g))
        for loss, g in out[1:]:
            assert loss == out[0][0] and torch.equal(g, out[0][1])


def test_positions_past_the_table_are_reported(oracle):
    sh = synth.WORKLOADS["tiny_fp32"].shape  # 32 positions
    p = synth.init_params(sh)
    T = 40
    tok = torch.zeros(1, T, dtype=torch.int32, device=DEV)
    tgt = torch.full((1, T), -1, dtype=torch.int32, device=DEV)
    tgt[0, 12] = 1
    adv = torch.ones(T, device=DEV)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, "fp32")
    with api.Context(api.answers_arena_bytes(cfg, 1, T, 2)) as c:
        _, ws = device_params(c, sh, p, "fp32")
        g = torch.empty(p.size, device=DEV)

        def go(s):
            c.reset()
            st = torch.tensor([s], dtype=torch.int32, device=DEV)
            return c.step_policy(ws, g, tok, tgt, None, None, adv, None, 0.2, 0.2, 0.0, B=1, T=T, starts=st, K=2)

        assert math.isfinite(go([12, 26, 40])) and math.isfinite(go([12, 32, 40]))
        for bad in ([12, 33, 40], [33, 33, 33], [0, 7, 40], [5, 3, 40], [0, 8, 41]):
            with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                go(bad)
        tok[0, 13] = sh.V
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            go([12, 26, 40])
        tok[0, 13] = 0
        tok[0, 39] = sh.V
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            go([12, 26, 40])
        assert math.isfinite(go([12, 26, 39]))  # padding now
        tgt[0, 12] = sh.V
        with pytest.raises(api.TTError, match="TT_ERR_ARG"):
            go([12, 26, 40])


def test_refusals(oracle):
    sh = synth.WORKLOADS["tiny_fp32"].shape
    p = synth.init_params(sh)
    B, T = 2, 16
    tok, tgt = torch.zeros(B, T, dtype=torch.int32), torch.ones(B, T, dtype=torch.int32)
    f = torch.zeros(B * T + 8, device=DEV)
    st = torch.tensor([[4, 8, 16]] * B, dtype=torch.int32, device=DEV)
    spans = torch.tensor([[0, 16], [16, 32]], dtype=torch.int32, device=DEV)
    cfg = api.make_config(sh.L, sh.C, sh.H, sh.V, sh.maxT, "fp32")
    assert api.answers_arena_bytes(cfg, 1, 33) == 0 and api.answers_arena_bytes(cfg, 1, 33, 1) > 0
    assert api.answers_arena_bytes(cfg, 0, 8, 1) == 0 and api.answers_arena_bytes(cfg, 1, 8, -1) == 0
    with api.Context(api.answers_arena_bytes(cfg, B, T, 2)) as c:
        g = torch.empty(p.size, device=DEV)
        with pytest.raises(api.TTError, match="TT_ERR_STATE"):
            c.step_policy(g, g, tok, tgt, f, f, f, f, 0.2, 0.2, 0.1, B=B, T=T)
        with pytest.raises(api.TTError, match="TT_ERR_STATE"):
            c.logprobs_of(g, tok, tgt, B, T, f)
        _, ws = device_params(c, sh, p, "fp32")
        odd, h = f.data_ptr() + 2, torch.zeros(B * T)
        n0 = c.launches

        def refused(fn, base, *bad):
            for b in bad:
                with pytest.raises(api.TTError, match="TT_ERR_ARG"):
                    fn(**{**base, **b})

        shapes = [dict(tokens=None), dict(targets=None), dict(params=None), dict(B=0), dict(T=0), dict(T=33), dict(B=2 ** 30),
                  dict(tau=0.0), dict(tau=math.nan), dict(starts=st, K=0), dict(starts=st, K=-1), dict(starts=st, K=2, B=0),
                  dict(starts=st.cpu(), K=2), dict(starts=odd, K=2)]
        pol = dict(params=ws, grads=g, tokens=tok, targets=tgt, old_logp=f, ref_logp=f, adv=f, weight=f, eps_low=0.2,
                   eps_high=0.2, beta=0.1, B=B, T=T)
        refused(c.step_policy, pol, *shapes, dict(grads=None), dict(adv=None), dict(ref_logp=None), dict(eps_low=1.0),
                dict(eps_high=-1.0), dict(beta=-1.0), dict(adv=h), dict(old_logp=h), dict(ref_logp=h), dict(weight=h),
                dict(logp=h), dict(adv=odd), dict(loss_scale=torch.ones(1)))
        pref = dict(params=ws, grads=g, tokens=tok, targets=tgt, ref_logp=f, spans=spans, pairs=1, beta=0.1, B=B, T=T)
        refused(c.step_preference, pref, *shapes, dict(grads=None), dict(spans=None), dict(pairs=0), dict(pairs=33),
                dict(beta=0.0), dict(gamma=math.inf), dict(smoothing=0.5), dict(spans=spans.cpu()), dict(ref_logp=h),
                dict(seq_logp=h), dict(spans=odd))
        lps = dict(params=ws, tokens=tok, targets=tgt, B=B, T=T, logp=f)
        refused(c.logprobs_of, lps, *shapes, dict(logp=None), dict(logp=h), dict(lse=h), dict(logp=odd))
        assert c.launches == n0
        c.reset()
        assert math.isfinite(c.step_preference(**pref))
        c.reset()
        assert math.isfinite(c.step_policy(**pol, starts=st, K=2))
        c.reset()
        c.logprobs_of(**lps, starts=st, K=2)
        c.sync()
    with api.Context(4096) as c:
        _, ws = device_params(c, sh, p, "fp32")
        for call in (lambda: c.step_policy(**pol), lambda: c.step_preference(**pref), lambda: c.logprobs_of(**lps)):
            with pytest.raises(api.TTError, match="TT_ERR_ARENA_OOM"):
                call()
