"""The post-training loss operators: measured cases, their plain forms, and their values in 64 bits.

Operators over a language model's logits and token log-probabilities:

* ``logp``    token log-probabilities (and entropies) from logits,
* ``vjp``     their backward pass,
* ``pref``    the paired preference loss with its gradient,
* ``policy``  the clipped policy loss with a KL term, with its gradient,
* ``head``    the policy loss taken from the logits, with the logits' gradient.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one sampled token of a serving loop, scored as it is accepted: latency counts
        {"name": "logp_one_token", "kind": "logp", "dtype": "bf16", "rows": 1, "vocab": 32768, "pad": 0,
         "temperature": 1.0, "entropy": False, "ignored": 0.0, "banned": 0.0},
        # a decode batch at a sampling temperature with entropies, fp16, a constrained vocabulary (-inf logits)
        {"name": "logp_decode_batch", "kind": "logp", "dtype": "f16", "rows": 96, "vocab": 131072, "pad": 0,
         "temperature": 0.7, "entropy": True, "ignored": 0.0, "banned": 0.3},
        # reference scoring of packed training sequences, prompts ignored
        {"name": "logp_scoring", "kind": "logp", "dtype": "bf16", "rows": 8192, "vocab": 65536, "pad": 0,
         "temperature": 1.0, "entropy": False, "ignored": 0.25, "banned": 0.0},
        # an odd vocabulary in 32 bits, rows padded to another stride, entropies monitored
        {"name": "logp_odd_f32", "kind": "logp", "dtype": "f32", "rows": 1111, "vocab": 50021, "pad": 27,
         "temperature": 1.0, "entropy": True, "ignored": 0.1, "banned": 0.0},
        # the backward pass of a preference step over packed sequences
        {"name": "vjp_bf16", "kind": "vjp", "dtype": "bf16", "rows": 4096, "vocab": 65536, "pad": 0,
         "temperature": 1.0, "entropy": False, "ignored": 0.25, "banned": 0.0},
        # the backward pass with an entropy bonus, 32 bits, odd sizes
        {"name": "vjp_odd_f32_entropy", "kind": "vjp", "dtype": "f32", "rows": 515, "vocab": 99991, "pad": 0,
         "temperature": 1.3, "entropy": True, "ignored": 0.0, "banned": 0.1},
        # a few short pairs: latency counts
        {"name": "pref_small", "kind": "pref", "pairs": 4, "tokens": 777, "masked": 0.3, "beta": 0.1,
         "smoothing": 0.0, "squared": False, "mean": False},
        # a large batch of ragged pairs with masked prompts and label smoothing
        {"name": "pref_large", "kind": "pref", "pairs": 1000, "tokens": 4000037, "masked": 0.3, "beta": 0.05,
         "smoothing": 0.1, "squared": False, "mean": False},
        # a small update: 16 sampled answers
        {"name": "policy_small", "kind": "policy", "seqs": 16, "tokens": 2999, "masked": 0.2, "lo": 0.2, "hi": 0.2,
         "kl": 0.0, "seq_mean": False},
        # a large update: ragged answers, wider upper clip, KL against a reference, each sequence weighted alike
        {"name": "policy_large", "kind": "policy", "seqs": 8192, "tokens": 8000011, "masked": 0.2, "lo": 0.2, "hi": 0.28,
         "kl": 0.04, "seq_mean": True},
        # one micro-batch of an update from logits, a small odd vocabulary, fp16
        {"name": "head_small_f16", "kind": "head", "dtype": "f16", "rows": 37, "vocab": 32003, "pad": 0, "seqs": 3,
         "temperature": 1.0, "ignored": 0.2, "banned": 0.0, "lo": 0.2, "hi": 0.2, "kl": 0.1, "seq_mean": True},
        # a full update from logits
        {"name": "head_large_bf16", "kind": "head", "dtype": "bf16", "rows": 4096, "vocab": 131072, "pad": 0, "seqs": 16,
         "temperature": 1.0, "ignored": 0.2, "banned": 0.0, "lo": 0.2, "hi": 0.28, "kl": 0.04, "seq_mean": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["logp", "vjp", "pref", "policy", "head"])
    if kind == "pref":
        pairs = _log_int(rng, 1, 2000)
        return {"kind": kind, "pairs": pairs, "tokens": _log_int(rng, 8 * pairs, 4000000),
                "masked": rng.choice([0.0, 0.3]), "beta": rng.choice([0.05, 0.1, 0.5]),
                "smoothing": rng.choice([0.0, 0.1]), "squared": rng.random() < 0.3, "mean": rng.random() < 0.3}
    if kind == "policy":
        seqs = _log_int(rng, 1, 8192)
        return {"kind": kind, "seqs": seqs, "tokens": _log_int(rng, 4 * seqs, 8000000),
                "masked": rng.choice([0.0, 0.2]), "lo": 0.2, "hi": rng.choice([0.2, 0.28]),
                "kl": rng.choice([0.0, 0.04]), "seq_mean": rng.random() < 0.5}
    vocab = _log_int(rng, 1000, 131072)
    rows = _log_int(rng, 1 if kind == "logp" else 16, min(4096, (3 << 26) // vocab))
    case = {"kind": kind, "dtype": rng.choice(["f32", "f16", "bf16"]), "rows": rows, "vocab": vocab,
            "pad": rng.choice([0, 0, 5, 64]), "temperature": rng.choice([1.0, 0.7]),
            "ignored": rng.choice([0.0, 0.2]) if rows > 8 else 0.0, "banned": rng.choice([0.0, 0.2])}
    if kind == "head":
        case.update(seqs=_log_int(rng, 1, max(1, rows // 8)), lo=0.2, hi=rng.choice([0.2, 0.28]),
                    kl=rng.choice([0.0, 0.04]), seq_mean=rng.random() < 0.5)
    else:
        case["entropy"] = rng.random() < 0.5
    return case


def work(case):
    if case["kind"] in ("pref", "policy"):
        n, live = case["tokens"], 1.0 - case["masked"]
        arrays = 2 if case["kind"] == "pref" or not case["kl"] else 3  # log-probabilities read
        return {"bytes": n * (4.0 * arrays * live + 4 + (1 if case["masked"] else 0)), "flops": n * live * 10.0}
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    n, live = float(case["rows"]) * case["vocab"], 1.0 - case["ignored"]
    if case["kind"] == "logp":
        return {"bytes": n * size * live + 16.0 * case["rows"], "flops": 4 * n * live}
    return {"bytes": n * size * (1 + live) + 16.0 * case["rows"], "flops": (4 if case["kind"] == "vjp" else 8) * n * live}


# ---- inputs ----

def _offsets(gen, seqs, tokens):
    """Bounds of packed sequences of uneven lengths (some may be empty)."""
    cuts = torch.randint(0, tokens + 1, (seqs - 1,), generator=gen, device="cuda").sort().values
    ends = torch.tensor([0, tokens], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _prompt(off, tokens, part):
    """Truth values: a token lies in the first `part` of its sequence (its prompt)."""
    at = torch.arange(tokens, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(off[1:].contiguous(), at, right=True)
    start, length = off[seq], off[seq + 1] - off[seq]
    return (at - start) < (length.double() * part).int(), seq


def _logits(case, gen):
    """Noise with the target's logit near the rest's log-sum, so that its probability is spread over (0, 1)."""
    rows, vocab = case["rows"], case["vocab"]
    store = torch.empty(rows, vocab + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    logits = store[:, :vocab]
    scale = 2.0 * case["temperature"]
    part = max(1, (1 << 28) // vocab)
    for r in range(0, rows, part):
        x = torch.randn(min(part, rows - r), vocab, generator=gen, device="cuda")
        if case["banned"]:
            x = x.masked_fill(torch.rand(x.shape, generator=gen, device="cuda") < case["banned"], -math.inf)
        logits[r:r + part] = x * scale
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    lift = math.log(vocab * (1 - case["banned"])) + 2.0 + 1.5 * torch.randn(rows, generator=gen, device="cuda")
    logits[torch.arange(rows, device="cuda"), target] = (lift * case["temperature"]).to(logits.dtype)
    return logits, target.to(torch.int32)


def _true_logp(case, logits, target):
    """Log-sums and the targets' log-probabilities in 64 bits, by blocks of rows."""
    part = max(1, (1 << 27) // case["vocab"])
    sums, ents = [], []
    for r in range(0, case["rows"], part):
        x = logits[r:r + part].double() / case["temperature"]
        m = x.max(1, keepdim=True).values
        e = torch.exp(x - m)
        s = e.sum(1)
        lse = m[:, 0] + torch.log(s)
        sums.append(lse)
        ents.append(lse - (e * x.clamp_min(-1e30)).sum(1) / s)
    lse = torch.cat(sums)
    at = target.long().clamp_min(0)
    x = logits[torch.arange(case["rows"], device="cuda"), at].double() / case["temperature"]
    return x - lse, lse, torch.cat(ents)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    state = {"case": case}
    kind = case["kind"]
    if kind in ("pref", "policy"):
        n = case["tokens"]
        seqs = 2 * case["pairs"] if kind == "pref" else case["seqs"]
        off = _offsets(gen, seqs, n)
        logp = -torch.log1p(torch.exp(1.5 * randn(n) - 0.5))
        state.update(off=off, logp=logp, mask=None, ref=logp + 0.15 * randn(n))
        if kind == "policy":
            state.update(old=logp + 0.12 * randn(n), adv=randn(seqs))
            if not case["kl"]:
                state["ref"] = None
        if case["masked"]:
            masked, _ = _prompt(off, n, case["masked"])
            state["mask"] = ~masked
            state["logp"] = logp.masked_fill(masked, -math.inf)  # prompts are not scored
        return state
    logits, target = _logits(case, gen)
    rows = case["rows"]
    if kind == "head":
        true = _true_logp(case, logits, target)[0].float()
        state.update(old=true + 0.12 * randn(rows), ref=true + 0.15 * randn(rows) if case["kl"] else None)
        off = _offsets(gen, case["seqs"], rows)
        state.update(off=off, adv=randn(case["seqs"]))
    else:
        off = _offsets(gen, 1 + rows // 512, rows)
    if case["ignored"]:
        target = target.masked_fill(_prompt(off, rows, case["ignored"])[0], -1)
    if kind == "vjp":
        _, lse, ent = _true_logp(case, logits, target)
        live = target >= 0
        state.update(lse=torch.where(live, lse, 0).float(), g=randn(rows) / rows, ent=None, gent=None)
        if case["entropy"]:
            state.update(ent=torch.where(live, ent, 0).float(), gent=-0.01 * torch.rand(rows, generator=gen, device="cuda") / rows)
    state.update(logits=logits, target=target)
    return state


# ---- one pass ----

def run(state):
    case, kind = state["case"], state["case"]["kind"]
    if own:
        from lower_convex_hull_amd import iso

        if kind == "logp":
            return iso.token_logp(state["logits"], state["target"], temperature=case["temperature"], entropy=case["entropy"])
        if kind == "vjp":
            return iso.token_logp_vjp(state["g"], state["logits"], state["target"], state["lse"], temperature=case["temperature"],
                                      entropy=state["ent"], g_entropy=state["gent"])
        if kind == "pref":
            smoothing = 0.0 if case["squared"] else case["smoothing"]  # the squared loss has none
            return iso.pref_loss(state["logp"], state["ref"], state["off"], mask=state["mask"], beta=case["beta"],
                                 label_smoothing=smoothing, squared=case["squared"], mean=case["mean"])
        if kind == "policy":
            return iso.policy_loss(state["logp"], state["old"], state["adv"], ref_logp=state["ref"], mask=state["mask"],
                                   seq_off=state["off"], clip_lo=case["lo"], clip_hi=case["hi"], kl_coef=case["kl"],
                                   seq_mean=case["seq_mean"])
        return iso.policy_loss_logits(state["logits"], state["target"], state["old"], state["adv"], ref_logp=state["ref"],
                                      seq_off=state["off"], temperature=case["temperature"], clip_lo=case["lo"],
                                      clip_hi=case["hi"], kl_coef=case["kl"], seq_mean=case["seq_mean"])
    if kind == "logp":
        x, live, logp, lse = _plain_logp(state["logits"], state["target"], case["temperature"])
        if not case["entropy"]:
            return logp.float(), lse.float()
        p = torch.exp(x - lse[:, None].float())
        ent = lse - torch.where(p > 0, p * x, 0).sum(1, dtype=torch.float64)
        return logp.float(), lse.float(), torch.where(live, ent, 0).float()
    if kind == "vjp":
        return _plain_vjp(state["logits"], state["target"], state["lse"], state["g"], state["ent"], state["gent"], case["temperature"])
    if kind == "pref":
        return _plain_pref(state)
    if kind == "policy":
        mask = state["mask"] if state["mask"] is not None else torch.ones_like(state["logp"], dtype=torch.bool)
        return _plain_policy(state["logp"].double(), mask, state)
    _, live, logp, lse = _plain_logp(state["logits"], state["target"], case["temperature"])
    loss, counts, g = _plain_policy(logp, live, state)
    return loss, counts, logp.float(), _plain_vjp(state["logits"], state["target"], lse, g, None, None, case["temperature"])


def _plain_logp(logits, target, temperature):
    live = target >= 0
    x = logits.float() / temperature
    m = x.max(1, keepdim=True).values
    lse = m[:, 0].double() + torch.log(torch.exp(x - m).sum(1, dtype=torch.float64))
    at = target.long().clamp_min(0)[:, None]
    logp = x.gather(1, at)[:, 0].double() - lse
    return x, live, torch.where(live, logp, 0), torch.where(live, lse, 0)


def _plain_vjp(logits, target, lse, g, ent, gent, temperature):
    live = target >= 0
    x = logits.float() / temperature
    g = torch.where(live, g, 0)
    z = x - lse[:, None].float()
    p = torch.exp(z)
    grad = p * -g[:, None]
    if ent is not None:
        grad -= torch.where(p > 0, torch.where(live, gent, 0)[:, None] * p * (z + ent[:, None]), 0)
    at = target.long().clamp_min(0)[:, None]
    grad.scatter_add_(1, at, g[:, None])
    return torch.where(live[:, None], grad / temperature, 0).to(logits.dtype)


def _by_sequence(values, off):
    """Sums over the packed sequences."""
    c = torch.cat([values.new_zeros(1), values.cumsum(0)])
    off = off.long()
    return c[off[1:]] - c[off[:-1]]


def _sequence_of(off, n):
    at = torch.arange(n, device=off.device, dtype=off.dtype)
    return torch.searchsorted(off[1:].contiguous(), at, right=True)


def _plain_pref(state):
    case, off, mask = state["case"], state["off"], state["mask"]
    n, pairs, beta = case["tokens"], case["pairs"], case["beta"]
    ratio = state["logp"].double() - state["ref"].double()
    live = torch.ones(n, dtype=torch.bool, device=off.device) if mask is None else mask
    s = _by_sequence(torch.where(live, ratio, 0), off)
    share = torch.ones_like(s)
    if case["mean"]:
        share = 1.0 / _by_sequence(live.double(), off).clamp_min(1)
        s = s * share
    delta = s[0::2] - s[1::2]
    if case["squared"]:
        loss = (delta - 0.5 / beta) ** 2
        slope = 2 * (delta - 0.5 / beta)
    else:
        e, h = case["smoothing"], beta * delta
        soft = lambda v: torch.clamp_min(v, 0) + torch.log1p(torch.exp(-v.abs()))  # noqa: E731
        loss = (1 - e) * soft(-h) + e * soft(h)
        slope = beta * (e / (1 + torch.exp(-h)) - (1 - e) / (1 + torch.exp(h)))
    coef = torch.stack([slope, -slope], 1).reshape(-1) * share / pairs
    grad = torch.where(live, coef[_sequence_of(off, n)], 0)
    return loss.sum().div(pairs).float(), loss.float(), (beta * s).float(), grad.float()


def _plain_policy(logp, live, state):
    case, off = state["case"], state["off"]
    n, seqs = logp.numel(), case["seqs"]
    seq = _sequence_of(off, n)
    adv = state["adv"].double()[seq]
    d = torch.where(live, logp - state["old"].double(), 0)
    over = live & (((adv > 0) & (d > math.log1p(case["hi"]))) | ((adv < 0) & (d < math.log1p(-case["lo"]))))
    ratio = torch.exp(d)
    edge = torch.where(adv > 0, 1 + case["hi"], 1 - case["lo"])
    pg = -torch.where(over, edge, ratio) * adv
    slope = torch.where(over, 0, -ratio * adv)
    kl = torch.zeros_like(pg)
    if state["ref"] is not None:
        u = torch.where(live, state["ref"].double() - logp, 0)
        kl = torch.exp(u) - u - 1
        slope = slope + case["kl"] * (1 - torch.exp(u))
    if case["seq_mean"]:
        w = (1.0 / (seqs * _by_sequence(live.double(), off).clamp_min(1)))[seq]
    else:
        w = 1.0 / live.sum().clamp_min(1).double()
    w = torch.where(live, w, 0)
    pg, kl = (w * pg).sum(), (w * kl).sum()
    loss = torch.stack([pg + case["kl"] * kl, pg, kl]).float()
    counts = torch.stack([live.sum(), over.sum()]).to(torch.int32)
    return loss, counts, (w * slope).float()


# ---- the definitions in 64 bits ----

def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "logp":
        parts = [_exact_logp(case, x, t) for x, t in _row_blocks(case, state["logits"], state["target"])]
        return tuple(torch.cat(v) for v in zip(*parts))
    if kind == "vjp":
        return _exact_vjp(case, state)
    if kind == "pref":
        logp = state["logp"].double()
        if state["mask"] is not None:
            logp = logp.masked_fill(~state["mask"], 0)
        logp.requires_grad_(True)
        return _exact_pref(case, state, logp)
    if kind == "policy":
        logp = state["logp"].double()
        live = state["mask"] if state["mask"] is not None else logp > -math.inf
        logp = logp.masked_fill(~live, 0).requires_grad_(True)
        loss, counts = _exact_policy(case, state, logp, live)
        return loss.detach(), counts, torch.autograd.grad(loss[0], logp)[0]
    live = state["target"] >= 0
    parts = [_exact_logp({**case, "entropy": False}, x, t)[0] for x, t in _row_blocks(case, state["logits"], state["target"])]
    logp = torch.cat(parts).requires_grad_(True)
    loss, counts = _exact_policy(case, state, logp, live)
    g = torch.autograd.grad(loss[0], logp)[0]
    grads = []
    at = 0
    for x, t in _row_blocks(case, state["logits"], state["target"]):
        z = x.double().requires_grad_(True)
        y = torch.log_softmax(z / case["temperature"], 1).gather(1, t.long().clamp_min(0)[:, None])[:, 0]
        up = torch.where(t >= 0, g[at:at + len(t)], 0)
        grads.append(torch.autograd.grad(y, z, up)[0])
        at += len(t)
    return loss.detach(), counts, logp.detach(), torch.cat(grads)


def _row_blocks(case, logits, target):
    part = max(1, (1 << 26) // case["vocab"])
    return [(logits[r:r + part], target[r:r + part]) for r in range(0, case["rows"], part)]


def _exact_logp(case, x, t):
    live = t >= 0
    z = x.double() / case["temperature"]
    lse = torch.logsumexp(z, 1)
    logs = z - lse[:, None]
    rows = torch.arange(len(t), device=t.device)
    found = [torch.where(live, logs[rows, t.long().clamp_min(0)], 0), torch.where(live, lse, 0)]
    if case["entropy"]:
        found.append(torch.where(live, torch.special.entr(torch.exp(logs)).sum(1), 0))
    return tuple(found)


def _exact_vjp(case, state):
    """The gradient at the log-sums and entropies that the call is given."""
    grads, at = [], 0
    for x, t in _row_blocks(case, state["logits"], state["target"]):
        pick = slice(at, at + len(t))
        z = x.double() / case["temperature"] - state["lse"][pick].double()[:, None]
        p = z.exp()
        hot = torch.zeros_like(p)
        hot[torch.arange(len(t), device=t.device), t.long().clamp_min(0)] = 1
        one = state["g"][pick].double()[:, None] * (hot - p)
        if state["ent"] is not None:
            inner = torch.special.entr(p) - p * state["ent"][pick].double()[:, None]  # -p (z + H)
            one = one + state["gent"][pick].double()[:, None] * inner
        grads.append((one / case["temperature"]).masked_fill((t < 0)[:, None], 0))
        at += len(t)
    return torch.cat(grads)


def _lengths(off):
    return (off[1:] - off[:-1]).long()


def _exact_pref(case, state, logp):
    off, mask = state["off"], state["mask"]
    owner = torch.repeat_interleave(torch.arange(2 * case["pairs"], device="cuda"), _lengths(off))
    live = torch.ones_like(logp) if mask is None else mask.double()
    zero = torch.zeros(2 * case["pairs"], dtype=torch.float64, device="cuda")
    s = zero.index_add(0, owner, live * (logp - state["ref"].double()))
    if case["mean"]:
        s = s / zero.index_add(0, owner, live).clamp_min(1)
    margin = s.view(-1, 2)[:, 0] - s.view(-1, 2)[:, 1]
    if case["squared"]:
        each = (margin - 1 / (2 * case["beta"])).square()
    else:
        log_sigmoid = torch.nn.functional.logsigmoid
        h = case["beta"] * margin
        each = -(1 - case["smoothing"]) * log_sigmoid(h) - case["smoothing"] * log_sigmoid(-h)
    loss = each.mean()
    grad = torch.autograd.grad(loss, logp)[0]
    return loss.detach(), each.detach(), (case["beta"] * s).detach(), grad


def _exact_policy(case, state, logp, live):
    off = state["off"]
    owner = torch.repeat_interleave(torch.arange(case["seqs"], device="cuda"), _lengths(off))
    adv = state["adv"].double()[owner]
    ratio = (logp - state["old"].double()).exp()
    bounded = ratio.clamp(1 - case["lo"], 1 + case["hi"])
    pg = -torch.minimum(ratio * adv, bounded * adv)
    over = live & (bounded * adv < ratio * adv)
    kl = torch.zeros_like(pg)
    if state["ref"] is not None:
        u = state["ref"].double() - logp
        kl = torch.expm1(u) - u
    if case["seq_mean"]:
        n = torch.zeros(case["seqs"], dtype=torch.float64, device="cuda").index_add(0, owner, live.double())
        w = 1 / (case["seqs"] * n.clamp_min(1))[owner]
    else:
        w = 1 / live.sum().clamp_min(1).double()
    w = w * live.double()
    pg, kl = (w * pg).sum(), (w * kl).sum()
    return torch.stack([pg + case["kl"] * kl, pg, kl]), torch.stack([live.sum(), over.sum()]).to(torch.int32)
