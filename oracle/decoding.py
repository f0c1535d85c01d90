"""Plain numpy forms of the decoding steps (definitions in iso.h), candidate by
candidate and page by page.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of f32, relative


def row_logp(x, temperature=1.0):
    """(logp, err) of a row of f64 logits: None where the row has no candidates.
    err: what the log-sum may be off by in units of U when its terms are f32 and
    their sum f64: sum p (3 |z - zmax| + 5), a term's exponent rounded three times
    (difference, constant, product), its exp by two half steps, and up to eight
    terms summed in f32 first, three roundings in pairs."""
    with np.errstate(invalid="ignore", over="ignore"):
        z = x / temperature
        m = z.max()
        if not np.isfinite(m) or np.isnan(z).any():
            return None, 0.0
        e = np.exp(z - m)
        s = e.sum()
        d = np.where(e > 0, z - m, 0.0)
        return (z - m) - np.log(s), float((e / s * (3 * np.abs(d) + 5)).sum())


def beam_select(x, score, take, weight=None, ended=None, end_token=-1, temperature=1.0):
    """For each batch item the list of all candidates that can be among the first
    `take`, in order: dicts with rank (f64), score, logp, parent, token, err."""
    batch, beams = score.shape
    out = []
    for b in range(batch):
        found = []
        for k in range(beams):
            r, s = b * beams + k, float(score[b, k])
            w = 1.0 if weight is None else float(weight[b, k])
            if not np.isfinite(s) or not (w > 0 and np.isfinite(w)):
                continue
            if ended is not None and ended[b, k]:
                found.append(dict(rank=s * w, score=s, logp=0.0, parent=r, token=end_token, err=0.0, beam=k, place=0, w=w))
                continue
            logp, err = row_logp(x[r], temperature)
            if logp is None:
                continue
            # the higher logit first, then the lower token
            best = np.argsort(-x[r], kind="stable")[:take]
            for i, v in enumerate(best):
                if x[r][v] > -np.inf:
                    t = s + logp[v]
                    found.append(dict(rank=t * w, score=t, logp=logp[v], parent=r, token=int(v), err=err, beam=k, place=i, w=w))
        with np.errstate(over="ignore"):
            key = lambda c: (-float(np.float32(c["rank"])) + 0.0, c["beam"], c["place"])  # noqa: E731
            out.append(sorted((c for c in found if np.float32(c["rank"]) > -np.inf), key=key))
    return out


def beam_reorder(state, parent, dim=0):
    """A copy of `state` with the rows along `dim` from their parents."""
    batch, beams = parent.shape
    rows = np.arange(batch * beams)
    p = parent.reshape(-1)
    at = np.where((p >= 0) & (p // beams == rows // beams), p, rows)
    return np.take(state, at, axis=dim)


def pages_fork(table, length, refs, parent, page_size, grow, pools=(), page_dim=0, token_dim=1):
    """(table, length, refs, status, pools) after the step, child by child."""
    seqs, most = table.shape
    pages, children = len(refs), len(parent)
    up = lambda n: -(-n // page_size)  # noqa: E731
    pools = [p.copy() for p in pools]
    had = [min(max(int(n), 0), most * page_size) for n in length]
    page = lambda q: 0 <= q < pages  # noqa: E731
    kids = []
    for i in range(children):
        p = int(parent[i]) if 0 <= parent[i] < seqs else -1
        before = had[p] if p >= 0 else 0
        kids.append((p, before, before + max(0, int(grow[i]))))
    old = np.maximum(refs, 0).astype(np.int64)
    new = old.copy()
    for s in range(seqs):
        for j in range(up(had[s])):
            if page(table[s, j]):
                new[table[s, j]] -= 1
    for p, before, _ in kids:
        for j in range(up(before)):
            if page(table[p, j]):
                new[table[p, j]] += 1
    edge = []
    for p, before, after in kids:
        q = int(table[p, before // page_size]) if after > before and before % page_size else -1
        edge.append(q if page(q) else -1)
    for q in set(edge) - {-1}:
        new[q] = max(new[q], edge.count(q))  # however few holders are counted, these hold it
    copies = []
    for i, q in enumerate(edge):
        alone = q >= 0 and new[q] == edge.count(q) and edge.index(q) == i
        copies.append(q >= 0 and not alone)
    need = sum(up(after) - up(before) + c for (_, before, after), c in zip(kids, copies))
    free = [q for q in range(pages) if new[q] <= 0]
    late = sum(up(after) > most or after > 2 ** 31 - 1 for _, _, after in kids)
    if late:
        need = sum((up(after) - up(before) + c) if up(after) <= most and after <= 2 ** 31 - 1 else 0
                   for (_, before, after), c in zip(kids, copies))
    if late or need > len(free):
        none = np.full((children, most), -1, np.int32)
        return (none, np.zeros(children, np.int32), old.astype(np.int32),
                np.array([min(max(need - len(free), 0), 2 ** 31 - 1), late, 0, 0, 0], np.int32), pools)
    out = np.full((children, most), -1, np.int32)
    give = iter(free)
    for i, (p, before, after) in enumerate(kids):
        for j in range(up(before)):
            out[i, j] = table[p, j] if page(table[p, j]) else -1
        if copies[i]:
            q = next(give)
            out[i, up(before) - 1] = q
            new[edge[i]] -= 1
            new[q] = 1
            for pool in pools:
                _move(pool, page_dim, token_dim, edge[i], q, before % page_size)
        for j in range(up(before), up(after)):
            out[i, j] = next(give)
            new[out[i, j]] = 1
    status = np.array([0, 0, sum(copies), need, len(free) - need], np.int32)
    return out, np.array([k[2] for k in kids], np.int32), np.maximum(new, 0).astype(np.int32), status, pools


def _move(pool, page_dim, token_dim, a, b, tokens):
    src, dst = [slice(None)] * pool.ndim, [slice(None)] * pool.ndim
    src[page_dim], dst[page_dim] = a, b
    if tokens is not None:
        src[token_dim] = dst[token_dim] = slice(0, tokens)
    pool[tuple(dst)] = pool[tuple(src)]


def pages_compact(table, refs, pools=(), page_dim=0):
    """(table, refs, moved, status, pools) with the live pages moved together."""
    pages = len(refs)
    pools = [p.copy() for p in pools]
    live = [q for q in range(pages) if refs[q] > 0]
    n = len(live)
    moved = np.full(pages, -1, np.int32)
    new = np.zeros(pages, np.int32)
    holes = iter([q for q in range(n) if refs[q] <= 0])
    moves = 0
    for q in live:
        moved[q] = q
        if q >= n:
            moved[q] = next(holes)
            moves += 1
            for pool in pools:
                _move(pool, page_dim, None, q, moved[q], None)
        new[moved[q]] = refs[q]
    out = np.array([moved[q] if 0 <= q < pages else -1 for q in table.reshape(-1)], np.int32).reshape(table.shape)
    return out, new, moved, np.array([n, moves], np.int32), pools
