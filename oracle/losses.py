"""Plain f64 numpy forms of the post-training losses (formulas in iso.h), row by
row and sequence by sequence.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of f32, relative


def token_logp(x, target, temperature=1.0):
    """(logp, lse, entropy, err) of f64 logits x (rows, vocab).  err: for each
    row the weighted size sum p (3 |z - zmax| + 2) + 2 rises of what a sum of f32
    exponentials may be off, in units of U: a term's exponent is rounded three
    times (difference, constant, product) and its exp by two half steps; the sums
    are f64, but scaled by an f32 factor, off by two half steps, when a maximum
    rises: after a chunk of 1024 logits or more of a row, at the row's ends and in
    the joins of lanes, waves and pieces.  16 at most are counted: a longer row has
    more chunks, but its maximum seldom rises after the first ones."""
    rises = min(16, x.shape[1] // 1024 + 4)
    rows, vocab = x.shape
    out = np.zeros((4, rows))
    for r in range(rows):
        t = int(target[r])
        if t < 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            z = x[r] / temperature
            m = z.max()
            if not np.isfinite(m):
                out[:, r] = np.nan
                continue
            d = z - m
            e = np.exp(d)
            s = e.sum()
            lse = m + np.log(s)
            p = e / s
            zd = np.where(p > 0, d, 0.0)
            out[0, r] = d[t] - np.log(s) if t < vocab else np.nan
            out[1, r] = lse
            out[2, r] = np.log(s) - (p * zd).sum()
            out[3, r] = (p * (3 * np.abs(zd) + 2)).sum() + 2 * rises
    return tuple(out)


def token_logp_vjp(x, target, lse, g, entropy=None, g_entropy=None, temperature=1.0):
    """(grad, err): the logits' gradient and, elementwise, what f32 arithmetic
    may be off by (U times the sizes of the terms, with the exponent's roundings)."""
    rows, vocab = x.shape
    grad = np.zeros((rows, vocab))
    err = np.zeros((rows, vocab))
    for r in range(rows):
        t = int(target[r])
        if t < 0:
            continue
        if t >= vocab or not np.isfinite(lse[r]):
            grad[r] = np.nan
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            z = x[r] / temperature - lse[r]
            p = np.exp(z)
        zz = np.where(p > 0, z, 0.0)
        v = -g[r] * p
        size = np.abs(g[r]) * p
        if g_entropy is not None:
            v = v - g_entropy[r] * p * (zz + entropy[r])
            size = size + np.abs(g_entropy[r]) * p * (np.abs(zz) + np.abs(entropy[r]))
        v[t] += g[r]
        grad[r] = v / temperature
        err[r] = U * (size * (3 * np.abs(zz) + 8) + np.abs(v)) / temperature
    return grad, err


def _span(off, q, tokens, seqs):
    if off is None:
        n = tokens // seqs
        return q * n, (q + 1) * n
    return int(off[q]), int(off[q + 1])


def pref_loss(logp, ref, mask, off, pairs, beta, smooth=0.0, squared=False, mean=False, grad_scale=1.0):
    """(loss, pair losses, rewards, grad) in f64 of f64 inputs."""
    n = len(logp)
    live = np.ones(n, bool) if mask is None else mask.astype(bool)
    s, count = np.zeros(2 * pairs), np.zeros(2 * pairs)
    for q in range(2 * pairs):
        a, b = _span(off, q, n, 2 * pairs)
        k = live[a:b]
        v = logp[a:b][k] - (0.0 if ref is None else ref[a:b][k])
        s[q], count[q] = v.sum(), max(1, k.sum())
    if mean:
        s = s / count
    each, reward, grad = np.zeros(pairs), beta * s, np.zeros(n)
    for i in range(pairs):
        d = s[2 * i] - s[2 * i + 1]
        if squared:
            each[i] = (d - 1 / (2 * beta)) ** 2
            slope = 2 * (d - 1 / (2 * beta))
        else:
            h = beta * d
            each[i] = (1 - smooth) * np.logaddexp(0, -h) + smooth * np.logaddexp(0, h)
            up = np.exp(-np.logaddexp(0, -h))  # sigma(h)
            slope = beta * (smooth * up - (1 - smooth) * np.exp(-np.logaddexp(0, h)))
        for q, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            a, b = _span(off, q, n, 2 * pairs)
            grad[a:b] = np.where(live[a:b], grad_scale * sign * slope / pairs / (count[q] if mean else 1.0), 0.0)
    return (each.mean() if pairs else 0.0), each, reward, grad


def policy_loss(logp, old, ref, adv, mask, off, seqs, lo=0.2, hi=0.2, kl_coef=0.0, seq_mean=False, token_adv=False,
                norm=0.0, grad_scale=1.0):
    """(loss (3,), counts (2,), grad, size) in f64: size is, token by token, how
    much the gradient moves for a change of logp (its derivative's size)."""
    n = len(logp)
    live = np.ones(n, bool) if mask is None else mask.astype(bool)
    grad, size = np.zeros(n), np.zeros(n)
    total = np.zeros(2)
    over = 0
    for q in range(seqs):
        a, b = _span(off, q, n, seqs)
        at = a + np.flatnonzero(live[a:b])
        if seq_mean:
            w = 1 / ((norm or seqs) * max(1, len(at)))
        else:
            w = 1 / (norm or max(1, live.sum()))
        adv_q = adv[at] if token_adv else np.full(len(at), adv[q])
        with np.errstate(over="ignore", invalid="ignore"):
            d = logp[at] - old[at]
            r = np.exp(d)
            r = np.where((adv_q == 0) & np.isfinite(d), 1.0, r)  # r A is 0, also where r is beyond f64
            clipped = np.clip(r, 1 - lo, 1 + hi)
            pg = -np.where(r * adv_q <= clipped * adv_q, r * adv_q, clipped * adv_q)
            pg = np.where(np.isnan(r * adv_q), np.nan, pg)
            held = np.where(adv_q > 0, r > 1 + hi, np.where(adv_q < 0, r < 1 - lo, False))
            slope = np.where(held, 0.0, -r * adv_q)
            kl = np.zeros(len(at))
            move = np.abs(slope)
            if ref is not None:
                u = ref[at] - logp[at]
                kl = np.where(u == np.inf, np.inf, np.expm1(u) - u)  # its limit
                if kl_coef:  # else the loss has no KL term, whatever u is
                    slope = slope - kl_coef * np.expm1(u)
                    move = move + abs(kl_coef) * np.exp(u)
        total += w * pg.sum(), w * kl.sum()
        over += int(held.sum())
        grad[at] = grad_scale * w * slope
        size[at] = abs(grad_scale) * w * move
    loss = np.array([total[0] + kl_coef * total[1] if kl_coef else total[0], total[0], total[1]])
    return loss, np.array([int(live.sum()), over]), grad, size
