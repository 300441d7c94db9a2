"""Cases that measure the operators on the LM head's logits: the list of a
row's top logits, distillation from a teacher's list, the selection step of a
beam search and the reordering of its states.

`run` computes an operator in plain torch operations, or, with `own` set,
through the package's public calls.  Logits are [rows, ld] with V real columns;
the columns V..ld-1 are padding and hold values that no result may depend on.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a whole training batch of the 124M model (32 x 1024 positions) against a teacher's 64 best logits,
        # half of the loss from the hard labels
        dict(name="distill_124m_batch", op="distill", dtype="bf16", M=32768, V=50257, ld=50304, k=64, alpha=0.5,
             tau=2.0, rest=False, grad=True, scale=1.0),
        # the batch of the 8 x 1024 workload in half with a loss scale, the teacher's log-sum-exp known
        dict(name="distill_124m_half", op="distill", dtype="fp16", M=8192, V=50257, ld=50304, k=32, alpha=0.9,
             tau=3.0, rest=True, grad=True, scale=32768.0),
        # fp32 training of one odd batch on an unpadded vocabulary, teacher only
        dict(name="distill_fp32_unpadded", op="distill", dtype="fp32", M=999, V=50257, ld=50257, k=100, alpha=1.0,
             tau=1.0, rest=True, grad=True, scale=1.0),
        # the character model's batch (64 x 256): many short rows
        dict(name="distill_char", op="distill", dtype="bf16", M=16384, V=65, ld=128, k=8, alpha=0.7, tau=1.5,
             rest=False, grad=True, scale=1.0),
        # the validation loss of one short sequence: no gradient, latency counts
        dict(name="distill_eval_short", op="distill", dtype="bf16", M=64, V=50257, ld=50304, k=64, alpha=0.5,
             tau=2.0, rest=True, grad=False, scale=1.0),
        # the teacher's side of a training batch
        dict(name="top_124m_batch", op="top", dtype="bf16", M=32768, V=50257, ld=50304, k=64, tau=2.0, lse=True),
        # the ten most likely tokens of a prompt's positions, unpadded fp32 logits
        dict(name="top_fp32_prompt", op="top", dtype="fp32", M=300, V=50257, ld=50257, k=10, tau=1.0, lse=True),
        # one sequence searched with four beams: a step's latency
        dict(name="select_1x4", op="select", dtype="bf16", B=1, K=4, V=50257, ld=50304, n=4, eos=-1),
        # a served batch, eight beams, twice as many candidates, some hypotheses finished
        dict(name="select_32x8", op="select", dtype="fp32", B=32, K=8, V=50257, ld=50304, n=16, eos=50256),
        # the 124M model's cache after a step of that search: 500 positions of 12 layers
        dict(name="reorder_124m", op="reorder", dtype="bf16", N=12, B=8, K=4, T=1024, C=768, t0=0, t1=500, sources=2,
             kept=1),
        # the tiny model's cache: latency
        dict(name="reorder_tiny", op="reorder", dtype="fp32", N=2, B=1, K=2, T=32, C=64, t0=0, t1=20, sources=1,
             kept=1),
        # the 350M model's cache in fp32, five beams, only the generated positions move
        dict(name="reorder_350m_tail", op="reorder", dtype="fp32", N=24, B=3, K=5, T=1024, C=1024, t0=65, t1=1000,
             sources=3, kept=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["distill", "distill", "top", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "reorder":
        K = rng.choice([2, 3, 4, 5, 8, 11, 16])
        T, C, N, B = _log(rng, 16, 1024), 64 * rng.randint(1, 16), rng.randint(1, 24), _log(rng, 1, 16)
        while N * B * K * T * 2 * C * BYTES[dtype] > 6e9:
            N, B = max(1, N // 2), max(1, B // 2)
        t1 = rng.randint(1, T)
        sources = rng.randint(1, K)
        kept = rng.randint(0, sources - 1)
        return dict(op=op, dtype=dtype, N=N, B=B, K=K, T=T, C=C, t0=rng.choice([0, rng.randint(0, t1 - 1)]), t1=t1,
                    sources=sources, kept=kept)
    V = _log(rng, 65, 150000)
    ld = rng.choice([(V + 127) // 128 * 128, (V + 127) // 128 * 128, V, V + rng.randint(1, 9)])
    if op == "select":
        K = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        B = max(1, min(_log(rng, 1, 64), int(4e8 / (K * ld * BYTES[dtype]))))
        n = rng.choice([K, K, 2 * K, rng.randint(1, 2 * K)])
        return dict(op=op, dtype=dtype, B=B, K=K, V=V, ld=ld, n=n, eos=rng.choice([-1, V - 1, rng.randint(0, V - 1)]))
    M = max(1, min(_log(rng, 1, 32768), int(3.2e9 / (ld * BYTES[dtype]))))
    k = rng.choice([1, 5, 10, 16, 32, 50, 64, rng.randint(1, min(64, V))])
    if op == "top":
        return dict(op=op, dtype=dtype, M=M, V=V, ld=ld, k=k, tau=rng.choice([1.0, 2.0, 0.7]),
                    lse=rng.choice([True, True, False]))
    return dict(op=op, dtype=dtype, M=M, V=V, ld=ld, k=k, alpha=rng.choice([1.0, 0.5, 0.9, round(rng.random(), 2)]),
                tau=rng.choice([1.0, 2.0, 4.0, round(rng.uniform(0.5, 5.0), 2)]), rest=rng.choice([True, False]),
                grad=rng.choice([True, True, True, False]), scale=32768.0 if dtype == "fp16" else 1.0)


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "distill":
        M, V, ld, k = case["M"], case["V"], case["ld"], case["k"]
        lists = M * (8 * k + 4 * case["rest"] + 4 * (case["alpha"] < 1))
        return {"bytes": M * V * es + lists + 4 * M + (M * ld * es if case["grad"] else 0),
                "flops": M * V * (4.0 + 4.0 * (case["alpha"] < 1 and case["tau"] != 1)) * (1 + case["grad"])}
    if case["op"] == "top":
        M, V, k = case["M"], case["V"], case["k"]
        return {"bytes": M * V * es + M * (8 * k + 4 * case["lse"]), "flops": M * V * (1.0 + 3.0 * case["lse"])}
    if case["op"] == "select":
        R, V = case["B"] * case["K"], case["V"]
        return {"bytes": R * V * es + 16 * case["B"] * case["n"], "flops": R * V * 4.0}
    moved = case["K"] - case["kept"]
    part = (case["t1"] - case["t0"]) * 2 * case["C"] * es * case["N"] * case["B"]
    read = len({p for j, p in enumerate(_pattern(case["K"], case["sources"], case["kept"])) if p != j})
    return {"bytes": part * (moved + read) + 4 * case["B"] * case["K"], "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _pattern(K, sources, kept):
    """Parents of K slots: `kept` slots stay as they are, the others copy one of the first `sources` slots, never
    themselves."""
    p = list(range(kept))
    for j in range(kept, K):
        q = (j + 1) % sources
        p.append(q if q != j else (q + 1) % sources if sources > 1 else (j + 1) % K)
    return p


def _columns(V, rows, k, g):
    """k different columns for each row, in any order."""
    at = torch.sort(torch.randint(0, V - k + 1, (rows, k), generator=g, device=DEV), dim=1).values
    at = at + torch.arange(k, device=DEV)
    return at.gather(1, torch.argsort(torch.rand(rows, k, generator=g, device=DEV), dim=1))


def _logits(case, rows, g):
    """Logits as a language model gives them (a wide bell, a few columns well above it), any values in the padding."""
    V, ld = case["V"], case["ld"]
    z = torch.empty(rows, ld, dtype=DTYPES[case["dtype"]], device=DEV)
    step = max(1, (1 << 27) // ld)
    for r in range(0, rows, step):
        z[r:r + step] = torch.randn(min(step, rows - r), ld, generator=g, device=DEV) * 2.0 - 1.0
    hot = _columns(V, rows, 12, g)
    lift = torch.randn(rows, 12, generator=g, device=DEV) * 1.5 + 7.0
    z.scatter_(1, hot, lift.to(z.dtype))
    return z


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "reorder":
        N, B, K, T, C = (case[n] for n in "NBKTC")
        s["state"] = torch.randn(N, B, K, T, 2 * C, generator=g, device=DEV).to(dt)
        perm = torch.argsort(torch.rand(B, K, generator=g, device=DEV), dim=1)
        pat = torch.tensor(_pattern(K, case["sources"], case["kept"]), device=DEV)
        parents = torch.empty(B, K, dtype=torch.int64, device=DEV)
        parents.scatter_(1, perm, perm[:, pat])
        s["parents"] = parents.to(torch.int32)
        return s
    if case["op"] == "select":
        B, K, n = case["B"], case["K"], case["n"]
        s["logits"] = _logits(case, B * K, g)
        s["scores"] = -20.0 + 3.0 * torch.randn(B, K, generator=g, device=DEV)
        s["done"] = (torch.rand(B, K, generator=g, device=DEV) < 0.2).to(torch.int32) if case["eos"] >= 0 else None
        s["out"] = dict(parent=torch.empty(B, n, dtype=torch.int32, device=DEV),
                        token=torch.empty(B, n, dtype=torch.int32, device=DEV),
                        score=torch.empty(B, n, device=DEV),
                        done=torch.empty(B, n, dtype=torch.int32, device=DEV))
        return s
    M, V, ld, k, tau = case["M"], case["V"], case["ld"], case["k"], case["tau"]
    s["logits"] = _logits(case, M, g)
    if case["op"] == "top":
        s["out"] = dict(vals=torch.empty(M, k, device=DEV), idx=torch.empty(M, k, dtype=torch.int32, device=DEV))
        if case["lse"]:
            s["out"]["lse"] = torch.empty(M, device=DEV)
        return s
    # the teacher's list: k different columns, its logits in descending order; one entry of sixteen rows unused
    idx = _columns(V, M, k, g)
    vals = torch.sort(torch.randn(M, k, generator=g, device=DEV) * 1.5 + 7.0, dim=1, descending=True).values
    near = vals + 0.7 * torch.randn(M, k, generator=g, device=DEV)  # the student has learnt some of it
    s["logits"].scatter_(1, idx, near.to(dt))
    if k > 1:
        idx[::16, k - 1] = -1
    s["t_vals"], s["t_idx"] = vals, idx.to(torch.int32)
    if case["rest"]:
        s["t_lse"] = torch.logsumexp(vals / tau, 1) + 0.02 + 0.3 * torch.rand(M, generator=g, device=DEV)
    if case["alpha"] < 1:
        y = torch.randint(0, V, (M,), generator=g, device=DEV)
        first = idx[:, 0]
        s["targets"] = torch.where((torch.rand(M, generator=g, device=DEV) < 0.5) & (first >= 0), first, y).to(torch.int32)
        s["targets"][5::97] = -1  # positions without a label
    s["out"] = dict(row_loss=torch.empty(M, device=DEV), mean_loss=torch.empty(1, device=DEV))
    if case["grad"]:
        s["out"]["dlogits"] = torch.empty(M, ld, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_top(s):
    c = s["case"]
    z = s["logits"][:, :c["V"]].float()
    # one whole number that orders by value, then by lowest column: the float's bits made monotone, then ~column
    bits = (z + 0.0).view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    col = torch.arange(c["V"], device=DEV)
    best = torch.topk(bits * (1 << 32) + ((1 << 32) - 1 - col), c["k"], dim=1, sorted=True).values
    idx = (1 << 32) - 1 - (best & 0xFFFFFFFF)
    out = dict(vals=z.gather(1, idx), idx=idx.to(torch.int32))
    if c["lse"]:
        u = z / c["tau"]
        m = u.amax(1, keepdim=True)
        out["lse"] = (m + (u - m).exp().sum(1, keepdim=True).log())[:, 0]
    return out


def _plain_distill(s):
    c = s["case"]
    V, tau, a = c["V"], c["tau"], c["alpha"]
    z = s["logits"][:, :V].float()
    used = s["t_idx"] >= 0
    idx = s["t_idx"].long().clamp(min=0)
    u = z / tau
    m = u.amax(1, keepdim=True)
    e = (u - m).exp()
    S = e.sum(1, keepdim=True)
    log_q = u.gather(1, idx) - m - S.log()
    t = torch.where(used, s["t_vals"] / tau, torch.full_like(s["t_vals"], -math.inf))
    if c["rest"]:
        log_p = t - s["t_lse"][:, None]
    else:
        tm = t.amax(1, keepdim=True)
        log_p = t - tm - (t - tm).exp().sum(1, keepdim=True).log()
    p = log_p.exp()
    W = p.sum(1, keepdim=True)
    loss = (p * (torch.where(used, log_p, torch.zeros_like(log_p)) - log_q)).sum(1)
    # unused entries point at column V of a wider row
    at = torch.where(used, idx, torch.full_like(idx, V))
    coef = W
    if c["rest"]:
        rest = torch.cat([e, torch.zeros_like(S)], 1).scatter(1, at, 0.0)[:, :V].sum(1, keepdim=True)
        p_r = (1.0 - W).clamp(min=0)
        has = rest > 0
        loss = loss + torch.where(has & (p_r > 0), p_r * (p_r.log() - rest.log() + S.log()), torch.zeros_like(S))[:, 0]
        W = torch.where(has, W + p_r, W)
        coef = torch.where(has, W - p_r * S / rest, W)
    loss = a * tau * tau * loss
    y = s.get("targets")
    if y is not None:
        lab = (y >= 0)[:, None]
        m1 = z.amax(1, keepdim=True)
        e1 = (z - m1).exp()
        S1 = e1.sum(1, keepdim=True)
        zy = z.gather(1, y.long().clamp(min=0)[:, None])
        loss = loss + (1 - a) * torch.where(lab, m1 + S1.log() - zy, torch.zeros_like(S1))[:, 0]
    out = dict(row_loss=loss, mean_loss=loss.mean(dtype=torch.float64).float()[None])
    if c["grad"]:
        d = (a * tau) * (coef / S) * e
        listed_ = (a * tau) * (W * log_q.exp() - p)
        d = torch.cat([d, torch.zeros_like(S)], 1).scatter(1, at, listed_)[:, :V]
        if y is not None:
            d += torch.where(lab, (1 - a) / S1, torch.zeros_like(S1)) * e1
            d.scatter_add_(1, y.long().clamp(min=0)[:, None], torch.where(lab, a - 1.0, 0.0).to(d.dtype))
        full = torch.zeros_like(s["logits"])
        full[:, :V] = (d * (c["scale"] / c["M"])).to(full.dtype)
        out["dlogits"] = full
    return out


def _plain_select(s):
    c = s["case"]
    B, K, V, n = c["B"], c["K"], c["V"], c["n"]
    z = s["logits"][:, :V].double()  # sums of many steps' scores: near candidates are told apart in 64 bits
    m = z.amax(1, keepdim=True)
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    cand = s["scores"].double()[:, :, None] + (z - lse).view(B, K, V)
    if s["done"] is not None:
        over = s["done"][:, :, None] != 0
        only = torch.arange(V, device=DEV) == c["eos"]
        cand = torch.where(over, torch.where(only, s["scores"].double()[:, :, None], -math.inf), cand)
    cand = cand.reshape(B, K * V)
    best, at = torch.sort(cand, dim=1, descending=True, stable=True)  # ties: the lowest beam, then column
    best, at = best[:, :n], at[:, :n]
    parent, token = at // V, at % V
    done = token == c["eos"]
    if s["done"] is not None:
        done = done | (s["done"].gather(1, parent) != 0)
    return dict(parent=parent.int(), token=token.int(), score=best.float(), done=done.int())


def _plain_reorder(s):
    c = s["case"]
    part = s["state"][:, :, :, c["t0"]:c["t1"]]
    b = torch.arange(c["B"], device=DEV)[:, None]
    part.copy_(part[:, b, s["parents"].long()])
    return dict(state=s["state"])


# ------------------------------------------------------------------ the package's calls
_kept = {}


def _context():
    if "ctx" not in _kept:
        from autograd_arena_allocated_gb300 import api
        _kept["ctx"] = api.Context(64 << 20)
    return _kept["ctx"]


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"distill": _plain_distill, "top": _plain_top, "select": _plain_select, "reorder": _plain_reorder}[op](state)
    ctx = _context()
    if op == "distill":
        o = state["out"]
        ctx.distill(c["dtype"], state["logits"], state["t_vals"], state["t_idx"], state.get("t_lse"),
                    state.get("targets"), o.get("dlogits"), o["row_loss"], o["mean_loss"], c["M"], c["V"], c["ld"],
                    c["k"], c["alpha"], c["tau"], c["scale"] / c["M"])
        return o
    if op == "top":
        o = state["out"]
        ctx.top_logits(c["dtype"], state["logits"], o["vals"], o["idx"], o.get("lse"), c["M"], c["V"], c["ld"], c["k"],
                       c["tau"])
        return o
    if op == "select":
        o = state["out"]
        ctx.beam_select(c["dtype"], state["logits"], state["scores"], state["done"], o["parent"], o["token"],
                        o["score"], o["done"], c["B"], c["K"], c["V"], c["ld"], c["n"], c["eos"])
        return o
    pos = 2 * c["C"] * BYTES[c["dtype"]]
    ctx.beam_reorder(state["state"], state["parents"], c["N"], c["B"], c["K"], c["T"] * pos, c["t0"] * pos,
                     (c["t1"] - c["t0"]) * pos)
    return dict(state=state["state"])


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_distill(c, s):
    M, V, a, tau = c["M"], c["V"], c["alpha"], c["tau"]
    losses, grads = [], []
    step = max(1, (1 << 26) // V)
    for r in range(0, M, step):
        z = s["logits"][r:r + step, :V].double()
        rows = torch.arange(z.shape[0], device=DEV)[:, None]
        i, t = s["t_idx"][r:r + step].long(), s["t_vals"][r:r + step].double() / tau
        w = torch.exp(t - (s["t_lse"][r:r + step].double()[:, None] if c["rest"] else t.amax(1, keepdim=True)))
        w = torch.where(i >= 0, w, 0.0)
        if not c["rest"]:
            w = w / w.sum(1, keepdim=True)
        # the teacher's distribution and the list's place, spread over the columns
        p = torch.zeros_like(z).index_put_((rows.expand_as(i), i.clamp(min=0)), w, accumulate=True)
        on = torch.zeros_like(z).index_put_((rows.expand_as(i), i.clamp(min=0)), (i >= 0).double(), accumulate=True) > 0
        logq = torch.log_softmax(z / tau, 1)
        del z
        kl = torch.xlogy(p, p).sum(1) - (p * logq).sum(1)
        q = logq.exp()
        del logq
        d = p.sum(1, keepdim=True) * q - p
        if c["rest"]:
            pr = (1 - p.sum(1)).clamp(min=0)
            qr = torch.where(on, 0.0, q).sum(1)
            ok = qr > 0
            kl = kl + torch.where(ok, torch.xlogy(pr, pr) - torch.xlogy(pr, qr), 0.0)
            d += torch.where(ok, pr, 0.0)[:, None] * q
            d -= torch.where(ok, pr / qr, 0.0)[:, None] * torch.where(on, 0.0, q)
        del p, on, q
        loss = a * tau ** 2 * kl
        d *= a * tau
        if a < 1:
            y = s["targets"][r:r + step].long()
            lp = torch.log_softmax(s["logits"][r:r + step, :V].double(), 1)
            hard = (y >= 0).double()
            loss = loss - (1 - a) * hard * lp.gather(1, y.clamp(min=0)[:, None])[:, 0]
            one = lp.exp_()
            one[rows[:, 0], y.clamp(min=0)] -= 1.0
            d += (1 - a) * hard[:, None] * one
        losses.append(loss)
        if c["grad"]:
            full = torch.zeros(d.shape[0], c["ld"], dtype=torch.float64, device=DEV)
            full[:, :V] = d * (c["scale"] / M)
            grads.append(full)
    row = torch.cat(losses)
    out = dict(row_loss=row, mean_loss=row.mean()[None])
    if c["grad"]:
        out["dlogits"] = torch.cat(grads)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "distill":
        return _exact_distill(case, s)
    if case["op"] == "top":
        lse = []
        step = max(1, (1 << 26) // case["V"])
        first = []
        for r in range(0, case["M"], step):
            z = s["logits"][r:r + step, :case["V"]].double()
            first.append(torch.sort(z, 1, descending=True).values[:, :case["k"]])
            lse.append(torch.logsumexp(z / case["tau"], 1))
        out = dict(vals=torch.cat(first), idx=None)
        if case["lse"]:
            out["lse"] = torch.cat(lse)
        return out
    if case["op"] == "select":
        logp = torch.log_softmax(s["logits"][:, :case["V"]].double(), 1).view(case["B"], case["K"], case["V"])
        got = []
        for b in range(case["B"]):
            every = []
            for k in range(case["K"]):
                score = s["scores"][b, k].double()
                if s["done"] is not None and int(s["done"][b, k]):
                    every.append(score[None])
                    every.append(torch.full((case["V"] - 1,), -math.inf, dtype=torch.float64, device=DEV))
                else:
                    every.append(score + logp[b, k])
            got.append(torch.topk(torch.cat(every), case["n"]).values)
        return dict(parent=None, token=None, score=torch.stack(got), done=None)
    state, parents = s["state"], s["parents"].cpu()
    old = state.clone()
    for b in range(case["B"]):
        for k in range(case["K"]):
            state[:, b, k, case["t0"]:case["t1"]] = old[:, b, int(parents[b, k]), case["t0"]:case["t1"]]
    return dict(state=state.double())
