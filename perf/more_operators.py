"""The decoding-step operators: measured cases, their plain forms, and the computed values in 64 bits.

Operators that make a model's answers and keep their states apart while they are made:

* ``select``   beam search's selection over beams and vocabulary, from logits,
* ``reorder``  contiguous states of beams brought into the order of their parents, in place,
* ``fork``     a step of a paged cache: sequences forked, grown, begun and freed,
* ``compact``  a paged cache's live pages moved together.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NONE = -(1 << 63)  # below every key
LOW = (1 << 32) - 1


def listed():
    return [
        # one request's four beams, one step of its decoding loop: latency counts
        {"name": "select_one_request", "kind": "select", "dtype": "bf16", "batch": 1, "beams": 4, "take": 4, "vocab": 32768,
         "pad": 0, "temperature": 1.0, "banned": 0.0, "ended": 0.0, "weighted": False, "first": False},
        # a decode batch of eight beams each, twice as many candidates asked for as beams
        {"name": "select_decode_batch", "kind": "select", "dtype": "bf16", "batch": 64, "beams": 8, "take": 16, "vocab": 131072,
         "pad": 0, "temperature": 1.0, "banned": 0.0, "ended": 0.0, "weighted": False, "first": False},
        # an odd vocabulary in 32 bits, rows padded to another stride, ended beams ranked by length
        {"name": "select_odd_f32", "kind": "select", "dtype": "f32", "batch": 33, "beams": 5, "take": 10, "vocab": 50021,
         "pad": 27, "temperature": 1.0, "banned": 0.0, "ended": 0.25, "weighted": True, "first": False},
        # wide beams under a grammar that forbids much of the vocabulary (-inf logits), fp16
        {"name": "select_wide_f16", "kind": "select", "dtype": "f16", "batch": 7, "beams": 32, "take": 64, "vocab": 100003,
         "pad": 5, "temperature": 0.7, "banned": 0.6, "ended": 0.1, "weighted": False, "first": False},
        # the small states of one request's beams: tokens so far, lengths, sums
        {"name": "reorder_histories", "kind": "reorder", "form": "history", "dtype": "f32", "batch": 1, "beams": 4, "layers": 1,
         "heads": 1, "tokens": 129, "room": 129, "dim": 1},
        # keys and values of 16 layers, heads outside tokens, of which 377 of 512 are filled
        {"name": "reorder_cache", "kind": "reorder", "form": "cache", "dtype": "bf16", "batch": 8, "beams": 8, "layers": 16,
         "heads": 8, "tokens": 377, "room": 512, "dim": 128},
        # recurrent states of odd sizes, 32 bits, five beams
        {"name": "reorder_recurrent", "kind": "reorder", "form": "recurrent", "dtype": "f32", "batch": 13, "beams": 5, "layers": 12,
         "heads": 9, "tokens": 1, "room": 1, "dim": 515},
        # four beams of one request, a step: latency counts
        {"name": "fork_one_request", "kind": "fork", "pattern": "beams", "dtype": "bf16", "groups": 1, "per": 4, "answers": 1,
         "tokens": 200, "page": 16, "layers": 8, "heads": 2, "dim": 64, "heads_first": False},
        # eight beams for each of 32 requests, pages of heads outside tokens
        {"name": "fork_beam_batch", "kind": "fork", "pattern": "beams", "dtype": "bf16", "groups": 32, "per": 8, "answers": 1,
         "tokens": 1500, "page": 16, "layers": 4, "heads": 8, "dim": 128, "heads_first": True},
        # continuous serving: most sequences grow by a token, some end and others begin with their prompt; a latent cache
        {"name": "fork_serving", "kind": "fork", "pattern": "serving", "dtype": "bf16", "groups": 1024, "per": 1, "answers": 1,
         "tokens": 2048, "page": 32, "layers": 1, "heads": 1, "dim": 256, "heads_first": False},
        # a small pool after a few requests have ended
        {"name": "compact_small", "kind": "compact", "dtype": "bf16", "groups": 5, "per": 2, "tokens": 190, "page": 16, "layers": 4,
         "heads": 2, "dim": 64, "heads_first": False, "live": 0.4},
        # a large pool, half of its pages free and strewn
        {"name": "compact_large", "kind": "compact", "dtype": "bf16", "groups": 96, "per": 4, "tokens": 1300, "page": 16, "layers": 3,
         "heads": 6, "dim": 128, "heads_first": True, "live": 0.5},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["select", "reorder", "fork", "compact"])
    case = {"kind": kind, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if kind == "select":
        beams = _log_int(rng, 1, 32)
        vocab = _log_int(rng, 1000, 200000)
        case.update(batch=_log_int(rng, 1, min(256, max(1, (1 << 25) // (vocab * beams)))), beams=beams,
                    take=beams * rng.choice([1, 1, 2]), vocab=vocab, pad=rng.choice([0, 0, 3, 64]),
                    temperature=rng.choice([1.0, 0.7]), banned=rng.choice([0.0, 0.0, 0.5]), ended=rng.choice([0.0, 0.2]),
                    weighted=rng.random() < 0.3, first=rng.random() < 0.15)
        return case
    if kind == "reorder":
        form = rng.choice(["history", "cache", "recurrent"])
        case.update(form=form, batch=_log_int(rng, 1, 16), beams=_log_int(rng, 2, 16), layers=rng.choice([1, 2, 6, 12]))
        if form == "recurrent":
            case.update(heads=rng.randint(1, 12), tokens=1, room=1, dim=_log_int(rng, 16, 700))
        else:
            room = _log_int(rng, 16, 512)
            case.update(heads=rng.randint(1, 8), tokens=rng.randint(1, room), room=room, dim=rng.choice([64, 80, 128]))
        return case
    groups, per = _log_int(rng, 1, 32), _log_int(rng, 1, 8)
    case.update(groups=groups, per=per, tokens=_log_int(rng, 2, 1000), page=rng.choice([1, 8, 16, 32]), layers=rng.choice([1, 2, 4]),
                heads=rng.randint(1, 8), dim=rng.choice([64, 80, 128]), heads_first=rng.random() < 0.5)
    if kind == "compact":
        case["live"] = rng.uniform(0.2, 0.95)
    else:
        case["pattern"] = rng.choice(["beams", "beams", "answers", "serving"])
        case["answers"] = rng.randint(2, 8) if case["pattern"] == "answers" else 1
    return case


def _page_count(case):
    """Pages of the pool: what the sequences hold at most, and a quarter more."""
    most = -(-case["tokens"] // case["page"])
    held = case["groups"] * (most + case["per"] * (most // 4 + 2)) if case["per"] > 1 else case["groups"] * most
    extra = case["groups"] * case["per"] * (case.get("answers", 1) + 1)
    return held + held // 4 + extra + 8


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
    kind = case["kind"]
    if kind == "select":
        live = case["beams"] * (1.0 - case["ended"]) if not case["first"] else 1.0
        n = case["batch"] * live * case["vocab"]
        return {"bytes": n * size + case["batch"] * (case["take"] * 16.0 + case["beams"] * 4), "flops": 4 * n}
    if kind == "reorder":
        # parents are uniform over a group's beams: rows that move, and rows that others come from
        k, rows = case["beams"], case["batch"] * case["beams"]
        moved, read = 1 - 1 / k, 1 - (1 - 1 / k) ** (k - 1)
        if case["form"] == "history":
            row = case["tokens"] * 8 + 8 + 4
        else:
            row = 2 * case["layers"] * case["heads"] * case["tokens"] * case["dim"] * size
        return {"bytes": rows * row * (moved + read) + rows * 4.0, "flops": 0}
    token = 2 * case["layers"] * case["heads"] * case["dim"] * size
    pages, seqs = _page_count(case), case["groups"] * case["per"]
    most = -(-case["tokens"] // case["page"])
    if kind == "compact":
        moves = pages * case["live"] * (1 - case["live"])
        return {"bytes": 2 * moves * case["page"] * token + 8 * seqs * most + 12 * pages, "flops": 0}
    partly = (case["page"] - 1) / case["page"]  # sequences that end inside a page, half filled on average
    children = seqs * case["answers"]
    copies = {"beams": children * (1 - 1 / case["per"]) ** case["per"], "answers": children - seqs, "serving": 0}[case["pattern"]]
    return {"bytes": 2 * copies * partly * case["page"] / 2 * token + 4 * (seqs + children) * (most + 2) + 8 * pages, "flops": 0}


# ---- inputs ----

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = {"select": _prepare_select, "reorder": _prepare_reorder, "fork": _prepare_fork, "compact": _prepare_compact}
    return {"case": case, **make[case["kind"]](case, gen)}


def _prepare_select(case, gen):
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
    rows = batch * beams
    store = torch.empty(rows, vocab + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    logits = store[:, :vocab]
    x = randn(rows, vocab) * 2.0
    # a few tokens of each row stand out, as a trained model's do
    likely = torch.randint(0, vocab, (rows, 6), generator=gen, device="cuda")
    x.scatter_(1, likely, math.log(vocab) + 2.0 + 1.5 * randn(rows, 6))
    if case["banned"]:
        x.masked_fill_(rand(rows, vocab) < case["banned"], -math.inf)
    logits.copy_(x * case["temperature"])
    score = -20 * rand(batch, 1) - 4 * rand(batch, beams)
    if case["first"]:  # the first step: all beams are alike, one counts
        score[:, 1:] = -math.inf
    ended = rand(batch, beams) < case["ended"] if case["ended"] else None
    weight = None
    if case["weighted"]:  # lengths to the power 0.6, ended beams have stayed shorter
        weight = 1.0 / torch.randint(8, 24, (batch, beams), generator=gen, device="cuda").float() ** 0.6
    return {"logits": logits, "score": score, "ended": ended, "weight": weight}


def _prepare_reorder(case, gen):
    batch, beams = case["batch"], case["beams"]
    rows = batch * beams
    parent = torch.randint(0, beams, (batch, beams), generator=gen, device="cuda")
    parent += torch.arange(batch, device="cuda")[:, None] * beams
    dtype = DTYPES[case["dtype"]]
    if case["form"] == "history":
        states = [torch.randint(0, 1 << 40, (rows, case["tokens"]), generator=gen, device="cuda"),
                  torch.randint(0, 1 << 40, (rows,), generator=gen, device="cuda"),
                  torch.randn(rows, generator=gen, device="cuda")]
        return {"states": states, "dim": 0, "parent": parent.to(torch.int32)}
    shape = (2 * case["layers"], rows, case["heads"], case["room"], case["dim"])
    store = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)
    return {"states": [store[:, :, :, :case["tokens"]]], "dim": 1, "parent": parent.to(torch.int32)}


def _pool(case, gen):
    token = (case["heads"], case["page"], case["dim"]) if case["heads_first"] else (case["page"], case["heads"], case["dim"])
    pool = torch.empty((2 * case["layers"], _page_count(case)) + token, dtype=DTYPES[case["dtype"]], device="cuda")
    return pool.normal_(generator=gen), 3 if case["heads_first"] else 2


def _sequences(case, gen):
    """Tables, lengths and reference counts: the sequences of a group share about three quarters of their pages."""
    groups, per, page = case["groups"], case["per"], case["page"]
    seqs, pages, most = groups * per, _page_count(case), -(-case["tokens"] // case["page"])
    last = torch.randint((case["tokens"] + 3) // 4, case["tokens"] + 1, (groups, 1), generator=gen, device="cuda")
    length = last.expand(groups, per).reshape(-1).contiguous()
    held = (length + page - 1) // page
    common = torch.where(held > 1, held - held // 4 - 1, 0) if per > 1 else torch.zeros_like(held)
    alone = held - common
    shared = common.view(groups, per)[:, 0]
    begin_own = shared.sum() + alone.cumsum(0) - alone
    begin_shared = (shared.cumsum(0) - shared).repeat_interleave(per)
    col = torch.arange(most + 2, device="cuda")
    place = torch.where(col < common[:, None], begin_shared[:, None] + col, begin_own[:, None] + col - common[:, None])
    valid = col < held[:, None]
    strewn = torch.randperm(pages, generator=gen, device="cuda")
    table = torch.where(valid, strewn[torch.where(valid, place, 0)], -1)
    refs = torch.zeros(pages + 1, dtype=torch.int64, device="cuda")
    refs.index_add_(0, table.reshape(-1) % (pages + 1), valid.reshape(-1).long())
    return table.to(torch.int32), length.to(torch.int32), refs[:pages].to(torch.int32), seqs


def _prepare_fork(case, gen):
    table, length, refs, seqs = _sequences(case, gen)
    pool, token_dim = _pool(case, gen)
    every = torch.arange(seqs, device="cuda")
    grow = torch.ones(seqs, dtype=torch.int64, device="cuda")
    if case["pattern"] == "beams":  # each beam goes on from one of its group; a tenth have ended
        parent = torch.randint(0, case["per"], (seqs,), generator=gen, device="cuda") + every // case["per"] * case["per"]
        grow -= (torch.rand(seqs, generator=gen, device="cuda") < 0.1).long()
    elif case["pattern"] == "answers":  # each sequence is a prompt, `answers` begin with it
        parent = every.repeat_interleave(case["answers"])
        grow = grow.repeat_interleave(case["answers"])
    else:  # a twentieth end; as many prompts begin in their places, no longer than what they take over
        ended = torch.rand(seqs, generator=gen, device="cuda") < 0.05
        prompt = (torch.rand(seqs, generator=gen, device="cuda") * length).long()
        parent, grow = torch.where(ended, -1, every), torch.where(ended, prompt, grow)
    return {"table": table, "length": length, "refs": refs, "parent": parent.to(torch.int32), "grow": grow.to(torch.int32),
            "pool": pool, "token_dim": token_dim}


def _prepare_compact(case, gen):
    table, _, _, _ = _sequences(case, gen)
    pool, _ = _pool(case, gen)
    pages = pool.shape[1]
    # which pages live is drawn afresh; freed pages leave the tables, and some are held from outside them too
    live = torch.rand(pages, generator=gen, device="cuda") < case["live"]
    table = torch.where((table >= 0) & live[table.long().clamp_min(0)], table, -1)
    refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.reshape(-1).long() % (pages + 1), (table >= 0).reshape(-1).int())
    refs = torch.where(live, refs[:pages].clamp_min(1), 0).to(torch.int32)
    return {"table": table, "refs": refs, "pool": pool}


# ---- one pass ----

def run(state):
    case, kind = state["case"], state["case"]["kind"]
    if own:
        from lower_convex_hull_amd import iso

        if kind == "select":
            return iso.beam_select(state["logits"], state["score"], take=case["take"], weight=state["weight"],
                                   ended=state["ended"], end_token=2, temperature=case["temperature"])
        if kind == "reorder":
            return iso.beam_reorder(state["states"], state["parent"], dim=state["dim"])
        if kind == "fork":
            out = iso.pages_fork(state["table"], state["length"], state["refs"], state["parent"], page_size=case["page"],
                                 grow=state["grow"], pools=state["pool"], page_dim=1, token_dim=state["token_dim"])
        else:
            out = iso.pages_compact(state["table"], state["refs"], pools=state["pool"], page_dim=1)
        return (*out, state["pool"])
    plain = {"select": _plain_select, "reorder": _plain_reorder, "fork": _plain_fork, "compact": _plain_compact}
    return plain[kind](state)


def _ordered(x):
    """Whole numbers in the order of the f32 values; -0 is 0."""
    b = (x + 0.0).view(torch.int32).long()
    return torch.where(b < 0, b ^ 0x7fffffff, b)


def _best(key, count):
    """The places of the largest keys in order (equal keys: the lowest place first), -1 past the keys that count; (rows, count)."""
    rows, n = key.shape
    place = torch.arange(n, device=key.device)
    top = torch.where(key == NONE, NONE, key * (1 << 32) + (LOW - place)).topk(min(count, n), dim=1).values
    found = torch.full((rows, count), -1, dtype=torch.int64, device=key.device)
    found[:, :min(count, n)] = torch.where(top == NONE, -1, LOW - (top & LOW))
    return found


def _plain_select(state):
    case = state["case"]
    batch, beams, take, temperature = case["batch"], case["beams"], case["take"], case["temperature"]
    x = state["logits"].float()
    m = x.max(1, keepdim=True).values
    total = torch.exp((x - m) / temperature).sum(1, dtype=torch.float64)
    lse = m[:, 0].double() / temperature + torch.log(total)
    token = _best(torch.where(x > -math.inf, _ordered(x), NONE), take)
    logp = x.gather(1, token.clamp_min(0)).double() / temperature - lse[:, None]
    score = state["score"].reshape(-1, 1).double()
    valid = (token >= 0) & torch.isfinite(score) & torch.isfinite(lse[:, None])
    if state["ended"] is not None:
        ended = state["ended"].reshape(-1, 1)
        only = torch.arange(take, device=x.device) == 0
        token, logp = torch.where(ended, 2, token), torch.where(ended, 0.0, logp)
        valid = torch.where(ended, only & torch.isfinite(score), valid)
    s = score + logp
    key = s if state["weight"] is None else s * state["weight"].reshape(-1, 1).double()
    key = key.float()
    key = torch.where(valid & (key > -math.inf), _ordered(key), NONE).reshape(batch, beams * take)
    at = _best(key, take)
    pick = lambda v: v.reshape(batch, beams * take).gather(1, at.clamp_min(0))  # noqa: E731
    beam = at // take + torch.arange(batch, device=x.device)[:, None] * beams
    return (torch.where(at >= 0, pick(s), -math.inf).float(), torch.where(at >= 0, pick(logp), -math.inf).float(),
            torch.where(at >= 0, beam, -1).to(torch.int32), torch.where(at >= 0, pick(token), -1).to(torch.int32))


def _plain_reorder(state):
    at, dim = state["parent"].reshape(-1).long(), state["dim"]
    return [s.copy_(s.index_select(dim, at)) for s in state["states"]]


def _plain_fork(state):
    table, length, page = state["table"].long(), state["length"].long(), state["case"]["page"]
    parent, grow = state["parent"].long(), state["grow"].long()
    children, cols, pages = parent.numel(), table.shape[1], state["refs"].numel()
    col, each = torch.arange(cols, device=table.device), torch.arange(children, device=table.device)
    up = lambda n: (n + page - 1) // page  # noqa: E731
    old = torch.where(parent >= 0, length[parent.clamp_min(0)], 0)
    new = old + grow
    held, want = up(old), up(new)
    rows = table[parent.clamp_min(0)]
    had, kept = col < up(length)[:, None], col < held[:, None]
    refs = state["refs"].long()
    refs = refs.index_add(0, table.clamp_min(0).reshape(-1), -had.long().reshape(-1))
    refs = refs.index_add(0, rows.clamp_min(0).reshape(-1), kept.long().reshape(-1))
    # a child that grows inside a page has it for itself: the first such child keeps it if nobody else holds it, others copy
    writes = (grow > 0) & (old % page > 0)
    edge = torch.where(writes, rows.gather(1, (old // page).clamp_max(cols - 1)[:, None])[:, 0], 0)
    writers = torch.zeros_like(refs).index_add(0, edge, writes.long())
    first = torch.full_like(refs, children).scatter_reduce(0, edge, torch.where(writes, each, children), "amin")
    copies = writes & ~((refs[edge] == writers[edge]) & (first[edge] == each))
    refs = refs.index_add(0, edge, -copies.long())
    need = want - held + copies
    start = need.cumsum(0) - need
    taken, free = need.sum(), (refs <= 0).sum()
    order = torch.argsort((refs > 0).to(torch.uint8), stable=True)  # the lowest free pages first
    fresh = order[((start + copies - held)[:, None] + col).clamp(0, pages - 1)]
    out = torch.where(kept, rows, torch.where(col < want[:, None], fresh, -1))
    out = torch.where(copies[:, None] & (col == (old // page)[:, None]), order[start.clamp_max(pages - 1)][:, None], out)
    refs = refs.scatter(0, order, torch.where(torch.arange(pages, device=table.device) < taken, 1, refs[order]))
    who = copies.nonzero()[:, 0]
    source, target, dim = edge[who], order[start[who]], state["token_dim"]
    pool = state["pool"]
    shape = [1] * pool.dim()
    shape[dim] = page
    filled = torch.arange(page, device=table.device).view(shape) < (old[who] % page).view(1, -1, *[1] * (pool.dim() - 2))
    pool[:, target] = torch.where(filled, pool[:, source], pool[:, target])
    status = torch.stack([(taken - free).clamp_min(0), (want > cols).sum(), copies.sum(), taken, free - taken])
    return out.to(torch.int32), new.to(torch.int32), refs.to(torch.int32), status.to(torch.int32), pool


def _plain_compact(state):
    table, refs, pool = state["table"].long(), state["refs"], state["pool"]
    live = refs > 0
    count = live.sum()
    below = torch.arange(refs.numel(), device=table.device) < count
    holes, movers = (~live & below).nonzero()[:, 0], (live & ~below).nonzero()[:, 0]
    moved = torch.where(live, torch.arange(refs.numel(), device=table.device), -1)
    moved[movers] = holes
    pool[:, holes] = pool[:, movers]
    out = torch.where(table >= 0, moved[table.clamp_min(0)], -1)
    packed = torch.zeros_like(refs)
    packed[moved[live]] = refs[live]
    status = torch.stack([count, torch.tensor(movers.numel(), device=table.device)])
    return out.to(torch.int32), packed, moved.to(torch.int32), status.to(torch.int32), pool


# ---- the definitions in 64 bits ----

def exact(case, seed):
    """The selected candidates' scores and log-probabilities; everything else is whole numbers and copies."""
    if case["kind"] != "select":
        return None
    state = prepare(case, seed)
    batch, beams, take, vocab = case["batch"], case["beams"], case["take"], case["vocab"]
    each = [_exact_item(state, b, case) for b in range(batch)]
    return torch.stack([e[0] for e in each]), torch.stack([e[1] for e in each]), None, None


def _exact_item(state, b, case):
    beams, take = case["beams"], case["take"]
    z = state["logits"][b * beams:(b + 1) * beams].double() / case["temperature"]
    logp = torch.log_softmax(z, 1)
    score = state["score"][b].double()
    if state["ended"] is not None:
        stop = state["ended"][b]
        logp[stop] = -math.inf
        logp[stop, 2] = 0.0
    total = logp + score[:, None]
    rank = total if state["weight"] is None else total * state["weight"][b].double()[:, None]
    rank = rank.reshape(-1)
    top = rank.topk(min(take, rank.numel())).indices
    fill = torch.full((take,), -math.inf, dtype=torch.float64, device=z.device)
    some = rank[top] > -math.inf
    scores, logs = fill.clone(), fill.clone()
    scores[:top.numel()] = torch.where(some, total.reshape(-1)[top], -math.inf)
    logs[:top.numel()] = torch.where(some, logp.reshape(-1)[top], -math.inf)
    return scores, logs
