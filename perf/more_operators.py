"""Cases that measure the operators of training on groups of answers: the log
probabilities of given tokens, the clipped policy loss, the loss of preferred
and rejected answers, and attention over answers that share their prompt.

`run` computes an operator in plain torch operations, or, with `own` set,
through the package's public calls.  Logits are [rows, ld] with V real columns;
the columns V..ld-1 are padding and hold values that no result may depend on.
A batch of B sequences of T positions has the label of a position where its
next token belongs to the sequence's answer, and -1 in the prompt and behind
the end.  A group is one row of T positions: a prompt, K answers that follow it
independently of each other, and padding.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the reference model's side of a training batch of the 124M model (32 answers of up to 1024 positions)
        dict(name="logprobs_124m_batch", op="logprobs", dtype="bf16", B=32, T=1024, V=50257, ld=50304, tau=1.0, lens=1),
        # three short prompts in fp32 on an unpadded vocabulary, at a sampling temperature: latency counts
        dict(name="logprobs_fp32_short", op="logprobs", dtype="fp32", B=3, T=100, V=50257, ld=50257, tau=0.7, lens=2),
        # a policy step over that batch, with the term that holds the policy near the reference model
        dict(name="policy_124m_batch", op="policy", dtype="bf16", B=32, T=1024, V=50257, ld=50304, tau=1.0, lo=0.2, hi=0.2,
             beta=0.05, ref=True, weighted=True, grad=True, scale=1.0, lens=3),
        # the 8 x 1024 workload in half with a loss scale, a wider bound above, no reference model
        dict(name="policy_124m_half", op="policy", dtype="fp16", B=8, T=1024, V=50257, ld=50304, tau=0.9, lo=0.2, hi=0.28,
             beta=0.0, ref=False, weighted=False, grad=True, scale=32768.0, lens=4),
        # the character model's batch (64 x 256): many short rows
        dict(name="policy_char", op="policy", dtype="bf16", B=64, T=256, V=65, ld=128, tau=1.0, lo=0.1, hi=0.3, beta=0.1,
             ref=True, weighted=True, grad=True, scale=1.0, lens=5),
        # sixteen pairs of answers of the 124M model against a reference model
        dict(name="preference_124m_pairs", op="preference", dtype="bf16", B=32, T=1024, V=50257, ld=50304, tau=1.0,
             beta=0.1, gamma=0.0, smooth=0.1, mean=False, ref=True, grad=True, scale=1.0, lens=6),
        # three odd pairs in fp32 on an unpadded vocabulary, without a reference model, by the mean token
        dict(name="preference_fp32_odd", op="preference", dtype="fp32", B=6, T=111, V=50257, ld=50257, tau=1.0,
             beta=2.0, gamma=0.5, smooth=0.0, mean=True, ref=False, grad=True, scale=1.0, lens=7),
        # the validation loss of one pair of the tiny model: latency
        dict(name="preference_tiny_eval", op="preference", dtype="fp32", B=2, T=32, V=256, ld=256, tau=1.0, beta=0.1,
             gamma=0.0, smooth=0.0, mean=False, ref=True, grad=False, scale=1.0, lens=8),
        # the 124M model: eight prompts with four answers each
        dict(name="group_124m_fwd", op="group", dtype="bf16", B=8, K=4, T=2048, C=768, H=12, prefix=0.5, pad=200,
             bwd=False, lens=9),
        dict(name="group_124m_bwd", op="group", dtype="bf16", B=8, K=4, T=2048, C=768, H=12, prefix=0.5, pad=200,
             bwd=True, lens=9),
        # the 350M model in half, eight answers each, odd lengths
        dict(name="group_350m_half_bwd", op="group", dtype="fp16", B=2, K=8, T=3001, C=1024, H=16, prefix=0.3, pad=77,
             bwd=True, lens=10),
        # the tiny model (fp32, heads of 16): latency
        dict(name="group_tiny_fwd", op="group", dtype="fp32", B=4, K=2, T=40, C=64, H=4, prefix=0.4, pad=5, bwd=False,
             lens=11),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "policy", "preference", "group", "group"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    lens = rng.randint(100, 10 ** 6)
    if op == "group":
        hd = rng.choice([64, 64, 64, 64, 32, 16])
        C = 64 * rng.randint(1, 16)
        H = C // hd
        B, T = _log(rng, 1, 16), _log(rng, 1, 8192)
        cost = 3e10 if dtype != "fp32" and hd == 64 else 4e9  # positions squared x channels, as the listed ones have
        while B * T * T * C > cost:
            B, T = max(1, B // 2), max(1, T * 3 // 4)
        return dict(op=op, dtype=dtype, B=B, K=rng.choice([1, 2, 3, 4, 8, 16]), T=T, C=C, H=H,
                    prefix=rng.choice([0.0, 0.3, 0.5, 0.8, round(rng.random(), 2)]), pad=rng.choice([0, 5, 70]),
                    bwd=rng.choice([True, False]), lens=lens)
    V = _log(rng, 65, 150000)
    ld = rng.choice([(V + 127) // 128 * 128, (V + 127) // 128 * 128, V, V + rng.randint(1, 9)])
    B, T = _log(rng, 1, 64), _log(rng, 1, 1024)
    if op == "preference":
        B = 2 * max(1, B // 2)
    while B * T * ld * BYTES[dtype] > 3.2e9:
        T = max(1, T // 2)
    grad, scale = rng.choice([True, True, True, False]), 32768.0 if dtype == "fp16" else 1.0
    tau = rng.choice([1.0, 1.0, 0.7, round(rng.uniform(0.5, 2.0), 2)])
    if op == "logprobs":
        return dict(op=op, dtype=dtype, B=B, T=T, V=V, ld=ld, tau=tau, lens=lens)
    if op == "policy":
        ref = rng.choice([True, False])
        return dict(op=op, dtype=dtype, B=B, T=T, V=V, ld=ld, tau=tau, lo=rng.choice([0.1, 0.2]),
                    hi=rng.choice([0.2, 0.28, 0.4]), beta=rng.choice([0.01, 0.05, 0.2]) if ref else 0.0, ref=ref,
                    weighted=rng.choice([True, False]), grad=grad, scale=scale, lens=lens)
    mean = rng.choice([True, False])
    return dict(op=op, dtype=dtype, B=B, T=T, V=V, ld=ld, tau=tau,
                beta=rng.choice([1.0, 2.5]) if mean else rng.choice([0.02, 0.1, 0.3]), gamma=rng.choice([0.0, 0.5]),
                smooth=rng.choice([0.0, 0.1]), mean=mean, ref=rng.choice([True, False]), grad=grad, scale=scale, lens=lens)


def _answers(case):
    """First and last + 1 labelled row of each sequence."""
    r = random.Random(case["lens"])
    T, out = case["T"], []
    for b in range(case["B"]):
        first = r.randint(0, T // 2)
        last = T if b == 0 else r.randint(min(T, first + 1 + T // 4), T)
        out.append((b * T + first, b * T + last))
    return out


def _left_out(row, T):
    """A few tokens inside the answers carry no label."""
    return (row % 89 == 7) & (row % T != T // 2)


def _starts(case):
    """Per group the end of the prompt, then the end of each answer (an answer may be empty)."""
    r = random.Random(case["lens"])
    T, K, out = case["T"], case["K"], []
    for b in range(case["B"]):
        end = T if b == 0 else max(1, T - r.randint(0, min(case["pad"], T - 1)))
        first = min(end, int(end * case["prefix"] * r.uniform(0.9, 1.0)))
        out.append([first] + sorted(r.randint(first, end) for _ in range(K - 1)) + [end])
    return out


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "group":
        pairs = rows = 0
        for s in _starts(case):
            pairs += s[0] * (s[0] + 1) // 2
            for a, b in zip(s, s[1:]):
                pairs += (b - a) * s[0] + (b - a) * (b - a + 1) // 2
            rows += s[-1]
        M, C = case["B"] * case["T"], case["C"]
        lse = 4 * M * case["H"]
        if case["bwd"]:
            return {"bytes": (3 + 2) * rows * C * es + lse + 3 * M * C * es, "flops": 10.0 * pairs * C}
        return {"bytes": 3 * rows * C * es + M * C * es + lse, "flops": 4.0 * pairs * C}
    M, V, ld = case["B"] * case["T"], case["V"], case["ld"]
    rows = sum(not _left_out(r, case["T"]) for a, b in _answers(case) for r in range(a, b))
    if case["op"] == "logprobs":
        return {"bytes": rows * V * es + 8 * M, "flops": rows * V * 4.0}
    out = M * ld * es if case["grad"] else 0
    if case["op"] == "policy":
        return {"bytes": rows * V * es + out + M * (4 + 4 + 4 + 4 * case["ref"] + 4 * case["weighted"] + 8),
                "flops": rows * V * 4.0 * (1 + case["grad"])}
    return {"bytes": rows * V * es + out + M * (4 + 4 * case["ref"]) + 8 * case["B"], "flops": rows * V * 4.0 * (1 + case["grad"])}


# ------------------------------------------------------------------ inputs
def _logits(case, rows, labels, g):
    """Logits as a language model gives them (a wide bell, the label well above it as a rule), any values in the padding."""
    V, ld = case["V"], case["ld"]
    z = torch.empty(rows, ld, dtype=DTYPES[case["dtype"]], device=DEV)
    step = max(1, (1 << 27) // ld)
    for r in range(0, rows, step):
        z[r:r + step] = torch.randn(min(step, rows - r), ld, generator=g, device=DEV) * 2.0 - 1.0
    y = labels.clamp(min=0).long()[:, None]
    lift = torch.randn(rows, 1, generator=g, device=DEV) * 2.0 + 0.6 * math.log(V)
    keep = z.gather(1, y).float()
    z.scatter_(1, y, torch.where((labels >= 0)[:, None], lift, keep).to(z.dtype))
    return z


def _logp_now(case, z, labels):
    """The labels' log probabilities to a few digits, for inputs that lie near them."""
    V, tau = case["V"], case["tau"]
    step = max(1, (1 << 28) // V)
    lse = torch.cat([torch.logsumexp(z[r:r + step, :V].float() / tau, 1) for r in range(0, z.shape[0], step)])
    return z.gather(1, labels.clamp(min=0).long()[:, None])[:, 0].float() / tau - lse


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "group":
        B, T, C, H = case["B"], case["T"], case["C"], case["H"]
        s["starts"] = torch.tensor(_starts(case), dtype=torch.int32, device=DEV)
        s["qkv"] = torch.randn(B * T, 3 * C, generator=g, device=DEV).to(dt)
        if not case["bwd"]:
            s["out"] = dict(y=torch.empty(B * T, C, dtype=dt, device=DEV), lse=torch.empty(B, H, T, device=DEV))
            return s
        fwd = _plain_group_fwd(s)
        s["y"], s["lse"] = fwd["y"], fwd["lse"]
        s["dy"] = torch.randn(B * T, C, generator=g, device=DEV).to(dt)
        s["out"] = dict(dqkv=torch.empty(B * T, 3 * C, dtype=dt, device=DEV))
        return s
    B, T, V, ld = case["B"], case["T"], case["V"], case["ld"]
    M = B * T
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    row = torch.arange(M, device=DEV)[:, None]
    spans = torch.tensor(_answers(case), device=DEV)
    on = ((row >= spans[:, 0]) & (row < spans[:, 1])).any(1)
    on &= ~_left_out(row[:, 0], T)
    labels = torch.where(on, labels, -1)
    s["targets"] = labels.to(torch.int32)
    s["logits"] = _logits(case, M, labels, g)
    noise = lambda sd: sd * torch.randn(M, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "logprobs":
        s["out"] = dict(logp=torch.empty(M, device=DEV), lse=torch.empty(M, device=DEV))
        return s
    now = _logp_now(case, s["logits"], labels)
    if case["ref"]:
        s["ref"] = torch.where(on, now + noise(0.3), 0.0)
    if case["op"] == "policy":
        # log ratios of a policy some updates on, none of them next to where the ratio is clipped
        d = noise(0.2)
        for edge in (math.log1p(-case["lo"]), math.log1p(case["hi"])):
            near = (d - edge).abs() < 2e-3
            d = torch.where(near, d + 5e-3, d)
        s["old"] = torch.where(on, now - d, 0.0)
        s["adv"] = torch.where(on, noise(1.0) + 0.4, 0.0)
        if case["weighted"]:
            s["weight"] = 0.5 + torch.rand(M, generator=g, device=DEV)
        s["out"] = dict(row_loss=torch.empty(M, device=DEV), mean_loss=torch.empty(1, device=DEV),
                        logp=torch.empty(M, device=DEV))
    else:
        s["spans"] = spans.to(torch.int32)
        s["out"] = dict(pair_loss=torch.empty(B // 2, device=DEV), mean_loss=torch.empty(1, device=DEV),
                        seq_logp=torch.empty(B, device=DEV))
    if case["grad"]:
        s["out"]["dlogits"] = torch.empty(M, ld, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _allowed(case, starts):
    """[B, T, T]: whether position i sees position j, and which positions belong to the group."""
    T = case["T"]
    at = torch.arange(T, device=DEV, dtype=torch.int32)
    seg = torch.searchsorted(starts, at.expand(starts.shape[0], T).contiguous(), right=True)  # 0: the prompt, 1..: the answers
    real = at[None] < starts[:, -1:]
    same = (seg[:, :, None] == seg[:, None, :]) | (seg[:, None, :] == 0)
    return same & (at[:, None] >= at[None, :]) & real[:, :, None] & real[:, None, :], real


def _heads(case, x, parts):
    B, T, H = case["B"], case["T"], case["H"]
    return x.float().view(B, T, parts, H, case["C"] // H).permute(2, 0, 3, 1, 4)


def _plain_group_fwd(s):
    c = s["case"]
    B, T, C, H = c["B"], c["T"], c["C"], c["H"]
    q, k, v = _heads(c, s["qkv"], 3)
    ok, real = _allowed(c, s["starts"])
    a = (q @ k.transpose(-1, -2)) / math.sqrt(C // H)
    a.masked_fill_(~ok[:, None], -math.inf)
    m = a.amax(-1, keepdim=True).clamp(min=-1e30)
    p = a.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    y = (p @ v) / l
    y = torch.where(real[:, None, :, None], y, 0.0)
    lse = torch.where(real[:, None], (m + l.log())[..., 0], 0.0)
    return dict(y=y.transpose(1, 2).reshape(B * T, C).to(s["qkv"].dtype), lse=lse)


def _plain_group_bwd(s):
    c = s["case"]
    B, T, C, H = c["B"], c["T"], c["C"], c["H"]
    scale = 1.0 / math.sqrt(C // H)
    q, k, v = _heads(c, s["qkv"], 3)
    y, dy = _heads(c, s["y"], 1)[0], _heads(c, s["dy"], 1)[0]
    ok, real = _allowed(c, s["starts"])
    p = (q @ k.transpose(-1, -2)) * scale
    p = p.sub_(s["lse"][..., None]).exp_().masked_fill_(~ok[:, None], 0.0)
    dy = torch.where(real[:, None, :, None], dy, 0.0)
    dv = p.transpose(-1, -2) @ dy
    ds = dy @ v.transpose(-1, -2)
    ds = ds.sub_((dy * y).sum(-1, keepdim=True)).mul_(p)
    dq, dk = (ds @ k) * scale, (ds.transpose(-1, -2) @ q) * scale
    out = torch.stack([dq, dk, dv])
    return dict(dqkv=out.permute(1, 3, 0, 2, 4).reshape(B * T, 3 * C).to(s["qkv"].dtype))


def _plain_logp(s, rows):
    """Of the labelled rows: exponentials, their sum, the log-sum-exp and the label's log probability."""
    c = s["case"]
    u = s["logits"][rows, :c["V"]].float() / c["tau"]
    y = s["targets"][rows].long()[:, None]
    uy = u.gather(1, y)[:, 0]
    m = u.amax(1, keepdim=True)
    e = u.sub_(m).exp_()
    S = e.sum(1, keepdim=True)
    lse = (m + S.log())[:, 0]
    return e, S, lse, uy - lse, y


def _spread(s, rows, x):
    return torch.zeros(s["targets"].shape[0], device=DEV).index_copy_(0, rows, x)


def _plain_grad(s, rows, e, S, y, coef):
    """coef (onehot - softmax) / tau in the labelled rows, zeros elsewhere."""
    c = s["case"]
    k = (coef / c["tau"])[:, None]
    d = e.mul_(-k / S).scatter_add_(1, y, k)
    full = torch.zeros_like(s["logits"])
    full[rows, :c["V"]] = d.to(full.dtype)
    return full


def _plain_logprobs(s):
    rows = (s["targets"] >= 0).nonzero()[:, 0]
    _, _, lse, logp, _ = _plain_logp(s, rows)
    return dict(logp=_spread(s, rows, logp), lse=_spread(s, rows, lse))


def _plain_policy(s):
    c = s["case"]
    rows = (s["targets"] >= 0).nonzero()[:, 0]
    e, S, _, logp, y = _plain_logp(s, rows)
    A = s["adv"][rows]
    d = logp - s["old"][rows]
    ratio = d.exp()
    inside = torch.where(A >= 0, d.double() <= math.log1p(c["hi"]), d.double() >= math.log1p(-c["lo"]))
    loss = -torch.where(inside, ratio, torch.where(A >= 0, 1 + c["hi"], 1 - c["lo"])) * A
    coef = -torch.where(inside, ratio, 0.0) * A
    if c["ref"]:
        t = s["ref"][rows] - logp
        loss = loss + c["beta"] * (torch.expm1(t) - t)
        coef = coef - c["beta"] * torch.expm1(t)
    if c["weighted"]:
        w = s["weight"][rows]
        loss, coef = loss * w, coef * w
    row = _spread(s, rows, loss)
    out = dict(row_loss=row, mean_loss=row.mean(dtype=torch.float64).float()[None], logp=_spread(s, rows, logp))
    if c["grad"]:
        out["dlogits"] = _plain_grad(s, rows, e, S, y, coef * (c["scale"] / row.shape[0]))
    return out


def _plain_preference(s):
    c = s["case"]
    P = c["B"] // 2
    rows = (s["targets"] >= 0).nonzero()[:, 0]
    e, S, _, logp, y = _plain_logp(s, rows)
    inside = (rows[:, None] >= s["spans"][:, 0]) & (rows[:, None] < s["spans"][:, 1])
    seq = inside.long().argmax(1)
    zero = torch.zeros(2 * P, dtype=torch.float64, device=DEV)  # sums of a whole answer
    total = zero.index_add(0, seq, logp.double())
    score = zero.index_add(0, seq, (logp - s["ref"][rows]).double()) if c["ref"] else total
    n = zero.index_add(0, seq, torch.ones_like(logp, dtype=torch.float64)).clamp(min=1) if c["mean"] else torch.ones_like(zero)
    score = c["beta"] * score / n
    u = (score[0::2] - score[1::2] - c["gamma"]).float()
    up, down = u.sigmoid(), (-u).sigmoid()
    softplus = lambda x: x.clamp(min=0) + (-x.abs()).exp().log1p()  # noqa: E731
    loss = (1 - c["smooth"]) * softplus(-u) + c["smooth"] * softplus(u)
    out = dict(pair_loss=loss, mean_loss=loss.mean(dtype=torch.float64).float()[None], seq_logp=total.float())
    if c["grad"]:
        du = (c["smooth"] * up - (1 - c["smooth"]) * down) * (c["beta"] * c["scale"] / P)
        coef = torch.stack([du, -du], 1).reshape(-1) / n.float()
        out["dlogits"] = _plain_grad(s, rows, e, S, y, coef[seq])
    return out


# ------------------------------------------------------------------ the package's calls
_kept = {}


def _context():
    if "ctx" not in _kept:
        from autograd_arena_allocated_gb300 import api
        _kept["ctx"] = api.Context(64 << 20)
    return _kept["ctx"]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "group":
            return (_plain_group_bwd if c["bwd"] else _plain_group_fwd)(s)
        return {"logprobs": _plain_logprobs, "policy": _plain_policy, "preference": _plain_preference}[op](s)
    ctx, o = _context(), s["out"]
    if op == "group":
        if c["bwd"]:
            ctx.group_attention_bwd(c["dtype"], s["qkv"], s["starts"], s["y"], s["lse"], s["dy"], o["dqkv"], c["B"], c["T"],
                                    c["C"], c["H"], c["K"])
        else:
            ctx.group_attention_fwd(c["dtype"], s["qkv"], s["starts"], o["y"], o["lse"], c["B"], c["T"], c["C"], c["H"],
                                    c["K"])
        return o
    M = c["B"] * c["T"]
    if op == "logprobs":
        ctx.logprobs(c["dtype"], s["logits"], s["targets"], o["logp"], o["lse"], M, c["V"], c["ld"], c["tau"])
    elif op == "policy":
        ctx.policy(c["dtype"], s["logits"], s["targets"], s["old"], s.get("ref"), s["adv"], s.get("weight"),
                   o.get("dlogits"), o["logp"], o["row_loss"], o["mean_loss"], M, c["V"], c["ld"], c["lo"], c["hi"],
                   c["beta"], c["tau"], c["scale"] / M)
    else:
        P = c["B"] // 2
        ctx.preference(c["dtype"], s["logits"], s["targets"], s.get("ref"), s["spans"], o.get("dlogits"), o["seq_logp"],
                       o["pair_loss"], o["mean_loss"], M, c["V"], c["ld"], P, c["beta"], c["gamma"], c["smooth"],
                       c["mean"], c["tau"], c["scale"] / P)
    return o


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(case, s, coef):
    """logp and lse of every row, and, where coef(logp) gives the loss's derivative by it, the logits' gradient."""
    V, tau = case["V"], case["tau"]
    y = s["targets"].long()
    step = max(1, (1 << 26) // V)
    lse, logp = [], []
    for r in range(0, y.shape[0], step):
        u = s["logits"][r:r + step, :V].double() / tau
        lse.append(torch.logsumexp(u, 1))
        logp.append(u.gather(1, y[r:r + step].clamp(min=0)[:, None])[:, 0] - lse[-1])
    on = y >= 0
    lse, logp = torch.where(on, torch.cat(lse), 0.0), torch.where(on, torch.cat(logp), 0.0)
    if coef is None:
        return lse, logp, None
    k = torch.where(on, coef(logp), 0.0)
    grad = torch.zeros(y.shape[0], case["ld"], dtype=torch.float64, device=DEV)
    for r in range(0, y.shape[0], step):
        here = slice(r, r + step)
        hot = torch.nn.functional.one_hot(y[here].clamp(min=0), V)
        soft = torch.softmax(s["logits"][here, :V].double() / tau, 1)
        grad[here, :V] = (hot - soft) * (k[here] / tau)[:, None]
    return lse, logp, grad


def _exact_policy(case, s):
    M, on = s["targets"].shape[0], s["targets"] >= 0
    A, old = s["adv"].double(), s["old"].double()
    w = s["weight"].double() if case["weighted"] else torch.ones(M, dtype=torch.float64, device=DEV)

    def value(logp):
        ratio = torch.exp(logp - old)
        loss = -torch.minimum(ratio * A, ratio.clamp(1 - case["lo"], 1 + case["hi"]) * A)
        if case["ref"]:
            x = s["ref"].double() - logp
            loss = loss + case["beta"] * (torch.exp(x) - x - 1)
        return torch.where(on, loss * w, 0.0)

    def coef(logp):
        logp = logp.detach().requires_grad_(True)
        value(logp).sum().backward()
        return logp.grad * (case["scale"] / M)

    _, logp, grad = _exact_rows(case, s, coef if case["grad"] else None)
    row = value(logp)
    out = dict(row_loss=row, mean_loss=row.mean()[None], logp=logp)
    if case["grad"]:
        out["dlogits"] = grad
    return out


def _exact_preference(case, s):
    P = case["B"] // 2
    spans = s["spans"].tolist()
    ref = s["ref"].double() if case["ref"] else torch.zeros(s["targets"].shape[0], dtype=torch.float64, device=DEV)
    labelled = s["targets"] >= 0

    def value(logp):
        score, total = [], []
        for a, b in spans:
            on = labelled[a:b].double()
            total.append((logp[a:b] * on).sum())
            n = on.sum().clamp(min=1) if case["mean"] else 1.0
            score.append(case["beta"] * ((logp[a:b] - ref[a:b]) * on).sum() / n)
        score = torch.stack(score).view(P, 2)
        u = score[:, 0] - score[:, 1] - case["gamma"]
        logsig = torch.nn.functional.logsigmoid
        return -(1 - case["smooth"]) * logsig(u) - case["smooth"] * logsig(-u), torch.stack(total)

    def coef(logp):
        logp = logp.detach().requires_grad_(True)
        value(logp)[0].sum().backward()
        return logp.grad * (case["scale"] / P)

    _, logp, grad = _exact_rows(case, s, coef if case["grad"] else None)
    loss, total = value(logp)
    out = dict(pair_loss=loss, mean_loss=loss.mean()[None], seq_logp=total)
    if case["grad"]:
        out["dlogits"] = grad
    return out


def _exact_group(case, s):
    """Group by group and answer by answer: an answer's queries against the prompt's keys and its own."""
    B, T, C, H = case["B"], case["T"], case["C"], case["H"]
    D = C // H
    ys = torch.zeros(B, T, C, dtype=torch.float64, device=DEV)
    lses = torch.zeros(B, H, T, dtype=torch.float64, device=DEV)
    grads = torch.zeros(B, T, 3 * C, dtype=torch.float64, device=DEV)
    for b, cuts in enumerate(s["starts"].tolist()):
        rows = s["qkv"].view(B, T, 3, H, D)[b].double().permute(1, 2, 0, 3)  # [3, H, T, D]
        for a, e in zip([0] + cuts[:-1], cuts):
            if a == e:
                continue
            seen = list(range(cuts[0])) + list(range(a, e)) if a > 0 or cuts[0] == 0 else list(range(e))
            seen = torch.tensor(seen, device=DEV)
            q, k, v = rows[0][:, a:e], rows[1][:, seen], rows[2][:, seen]
            score = torch.einsum("hid,hjd->hij", q, k) / math.sqrt(D)
            score = score.masked_fill(seen[None, None, :] > torch.arange(a, e, device=DEV)[None, :, None], -math.inf)
            if not case["bwd"]:
                lses[b, :, a:e] = torch.logsumexp(score, -1)
                ys[b, a:e] = torch.einsum("hij,hjd->ihd", torch.softmax(score, -1), v).reshape(e - a, C)
                continue
            p = torch.exp(score - s["lse"][b, :, a:e, None].double())
            y, dy = (s[n].view(B, T, H, D)[b, a:e].double().transpose(0, 1) for n in ("y", "dy"))
            dsc = p * (torch.einsum("hid,hjd->hij", dy, v) - (y * dy).sum(-1, keepdim=True)) / math.sqrt(D)
            place = grads[b].view(T, 3, H, D)
            place[a:e, 0] += torch.einsum("hij,hjd->ihd", dsc, k)
            place[:, 1].index_add_(0, seen, torch.einsum("hij,hid->jhd", dsc, q))
            place[:, 2].index_add_(0, seen, torch.einsum("hij,hid->jhd", p, dy))
    if case["bwd"]:
        return dict(dqkv=grads.view(B * T, 3 * C))
    return dict(y=ys.view(B * T, C), lse=lses)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "group":
        return _exact_group(case, s)
    if case["op"] == "logprobs":
        lse, logp, _ = _exact_rows(case, s, None)
        return dict(logp=logp, lse=lse)
    return (_exact_policy if case["op"] == "policy" else _exact_preference)(case, s)
