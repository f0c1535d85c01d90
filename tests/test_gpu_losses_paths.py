"""The losses where their kernels take another path: sizes at the borders between
workgroup shapes, rows and gradients that no shift aligns both of, spans that
many sequences begin in, differences far from 0, small and large calls.

Tolerances are those of test_gpu_losses: an output's own rounding, what the
oracle counts for f32 sums of exponentials, and 1e-12 of the sizes for f64 sums.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import losses
from tests.test_gpu_losses import U, check_logp, check_vjp, dtype_of, floor_of, half, make, near, put, say, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# bytes of a row (f32: vocab * 4) around 8, 16, 32, 40, 64, 96, 128 and 160 KB, and whole and broken chunks beyond
VOCABS = [2048, 2049, 4096, 4099, 8191, 8192, 10240, 10241, 16384, 24577, 32768, 32771, 40960, 40961, 65536, 98307]


def head_case(torch, logits, target, x, seqs, off, seed, seq_mean, out=None, token_adv=False, norm=0.0):
    rng = np.random.default_rng(seed)
    rows, vocab = logits.shape
    tgt = target.numpy()
    lp, lse, _, err = losses.token_logp(x, tgt)
    adv = rng.normal(size=rows if token_adv else seqs).astype(np.float32)
    old = (lp + rng.choice([-0.6, -0.1, 0.0, 0.1, 0.6], rows)).astype(np.float32)
    ref = (lp + rng.normal(0, 0.3, rows)).astype(np.float32)
    got = iso.policy_loss_logits(logits, target.cuda(), put(torch, old), put(torch, adv), ref_logp=put(torch, ref),
                                 seq_off=put(torch, off), kl_coef=0.05, seq_mean=seq_mean, token_adv=token_adv,
                                 norm=norm, out=out)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    w = losses.policy_loss(lp, f(old), f(ref), f(adv), tgt >= 0, off, seqs, kl_coef=0.05, seq_mean=seq_mean,
                           token_adv=token_adv, norm=norm)
    assert np.array_equal(got[1].cpu().numpy(), w[1])
    moved = U * (err + 2)  # what logp may be off by
    assert np.all(np.abs(got[2].double().cpu().numpy() - lp) <= U * np.abs(lp) + moved)
    tol = ((np.abs(w[2]) + w[3]) * moved).sum() * 2 + 1e-12
    for k in range(3):
        assert abs(float(got[0][k]) - w[0][k]) <= U * abs(w[0][k]) + tol * (1 if k < 2 else 20), k
    want, werr = losses.token_logp_vjp(x, tgt, lse, w[2])
    shape, _ = losses.token_logp_vjp(x, tgt, lse, np.ones(rows))
    tol = werr + np.abs(shape) * ((w[3] + np.abs(w[2])) * moved + np.abs(w[2]) * 2 * U)[:, None]
    tol += half(torch, logits.dtype) * np.abs(want) + floor_of(torch, logits.dtype)
    bad = np.abs(got[3].double().cpu().numpy() - want) - tol
    assert bad.max() <= 0, bad.max()
    return got


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_rows_at_the_borders(torch, name, vocab):
    """Forward, backward and the loss from logits, at bases and strides that shift a row's first aligned element."""
    say(f"[losses] border {name} {vocab}")
    dtype = dtype_of(torch, name)
    logits, target, x, _ = make(torch, dtype, 3, vocab, vocab, pad=vocab % 7, shift=vocab % 4)
    target[0], target[1], target[2] = 0, vocab - 1, vocab // 2  # a row's ends, which single threads take
    tg = target.cuda()
    got = iso.token_logp(logits, tg, entropy=True)
    check_logp(torch, got, x, target, 1.0)
    g = torch.tensor([0.7, -1.3, 0.2], device="cuda")
    gent = torch.tensor([0.1, -0.2, 0.3], device="cuda")
    # a gradient at another alignment than the logits'
    store = torch.full((3, vocab + 11), 5.0, dtype=dtype, device="cuda")
    grad = iso.token_logp_vjp(g, logits, tg, got[1], entropy=got[2], g_entropy=gent, out=store[:, 1:vocab + 1])
    check_vjp(torch, grad, x, target, got[1], g, got[2], gent, 1.0, dtype)
    assert bool((store[:, 0] == 5).all()) and bool((store[:, vocab + 1:] == 5).all())
    store.fill_(5.0)
    off = np.array([0, 1, 3], np.int32)
    a = head_case(torch, logits, target, x, 2, off, vocab, True, out=store[:, 3:vocab + 3])
    assert bool((store[:, :3] == 5).all()) and bool((store[:, vocab + 3:] == 5).all())
    b = head_case(torch, logits, target, x, 2, off, vocab, True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("seq_mean,token_adv,norm", [(True, False, 0.0), (False, False, 0.0), (False, True, 0.0), (True, True, 3.5)])
@pytest.mark.parametrize("rows,seqs", [(1, 1), (255, 200), (256, 256), (257, 256), (300, 500), (4097, 11), (8192, 30), (8193, 2000), (9000, 3000)])
def test_rows_and_their_terms(torch, rows, seqs, seq_mean, token_adv, norm):
    """Rows' weights and advantages found by the row, by one workgroup, by many; sequences that are empty or ignored."""
    say(f"[losses] terms {rows}/{seqs} {seq_mean} {token_adv}")
    logits, target, x, _ = make(torch, torch.bfloat16, rows, 37, rows + seqs)
    rng = np.random.default_rng(rows)
    off = np.concatenate([[0], np.sort(rng.integers(0, rows + 1, seqs - 1)), [rows]]).astype(np.int32)
    target[torch.from_numpy(rng.random(rows) < 0.3)] = -1
    q = seqs // 2
    target[off[q]:off[q + 1]] = -1
    head_case(torch, logits, target, x, seqs, off, rows, seq_mean, token_adv=token_adv, norm=norm)
    if rows % 5 == 0:
        head_case(torch, logits, target, x, 5, (np.arange(6) * (rows // 5)).astype(np.int32), rows, seq_mean, token_adv=token_adv)


@pytest.mark.parametrize("name,rows,vocab", [("f32", 700, 50021), ("bf16", 1100, 65536), ("f16", 9000, 9001)])
def test_more_logits_than_the_cache_holds(torch, name, rows, vocab):
    """More than 128 MB: every row agrees with the calls on its own block of rows, and some with the oracle."""
    say(f"[losses] large {name} {rows}x{vocab}")
    dtype = dtype_of(torch, name)
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    logits = (torch.randn(rows, vocab, generator=gen, device="cuda") * 2).to(dtype)
    target = torch.randint(0, vocab, (rows,), generator=gen, device="cuda").to(torch.int32)
    target[rows // 3] = -1
    g = torch.randn(rows, generator=gen, device="cuda")
    lp, lse, ent = iso.token_logp(logits, target, entropy=True)
    grad = iso.token_logp_vjp(g, logits, target, lse, entropy=ent, g_entropy=g)
    pick = torch.tensor([0, 1, rows // 3, rows // 2, rows - 2, rows - 1], device="cuda")
    x, t = logits[pick], target[pick]
    xn = x.double().cpu().numpy()
    check_logp(torch, (lp[pick], lse[pick], ent[pick]), xn, t.cpu(), 1.0)
    check_vjp(torch, grad[pick], xn, t.cpu(), lse[pick], g[pick], ent[pick], g[pick], 1.0, dtype)
    part = slice(rows // 4, rows // 4 + 100)  # a small call's gradient is the same elements' arithmetic
    small = iso.token_logp_vjp(g[part], logits[part], target[part], lse[part], entropy=ent[part], g_entropy=g[part])
    assert torch.equal(small, grad[part])


@pytest.mark.parametrize("vocab", [1000, 16385, 131072])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_confident_tokens(torch, rows, vocab):
    """A target that takes nearly all: logp = -log(1 + r) keeps its relative accuracy.  The largest term is exactly 1 and
    the sums are f64, so each other term's own roundings (its exponent's three, its exp's two half steps) and the output's
    are all that is left."""
    gen = torch.Generator().manual_seed(rows + vocab)
    x = torch.randn(rows, vocab, generator=gen)
    target = torch.randint(0, vocab, (rows,), generator=gen, dtype=torch.int32)
    lift = math.log(vocab) + torch.linspace(2.0, 14.0, rows)
    x[torch.arange(rows), target.long()] = lift
    old = torch.zeros(rows, device="cuda")
    got = iso.token_logp(x.cuda(), target.cuda())[0]
    head = iso.policy_loss_logits(x.cuda(), target.cuda(), old, torch.ones(1, device="cuda"))[2]
    for r in range(rows):
        z = x[r].double().numpy()
        z = z - z.max()
        e = np.exp(z)
        e[target[r]] = 0.0
        want = -np.log1p(e.sum())
        tol = U * (abs(want) + (e * (3 * np.abs(z) + 2)).sum())
        for name, v in (("logp", got), ("head", head)):
            assert abs(float(v[r]) - want) <= tol, (name, r, float(v[r]), want, tol)


def piles(rng, seqs, tokens, places):
    """Offsets that fall on few places: many sequences are empty, hundreds begin at one token."""
    at = np.sort(rng.integers(0, tokens + 1, places))
    return np.concatenate([[0], np.sort(rng.choice(at, seqs - 1)), [tokens]]).astype(np.int32)


@pytest.mark.parametrize("tokens", [3000, 8192, 8193, 30011])
@pytest.mark.parametrize("kind", ["piles", "ones", "one-long", "all-in-the-last"])
def test_sequences_in_a_span(torch, kind, tokens):
    """More sequences in a span than a wave has lanes, most of them empty; one token each; one that takes nearly all."""
    say(f"[losses] spans {kind} {tokens}")
    rng = np.random.default_rng(tokens)
    if kind == "piles":
        seqs = 2000
        off = piles(rng, seqs, tokens, 9)
    elif kind == "ones":
        seqs = tokens - tokens % 2
        off = np.concatenate([np.arange(seqs), [tokens]]).astype(np.int32)
    elif kind == "one-long":
        seqs = 300
        off = np.concatenate([np.arange(150), tokens - np.arange(150, -1, -1)]).astype(np.int32)
    else:
        seqs = 700
        off = np.zeros(seqs + 1, np.int32)
        off[-1] = tokens
    logp = -rng.exponential(1.0, tokens).astype(np.float32)
    old = (logp + rng.normal(0, 0.25, tokens)).astype(np.float32)
    ref = (logp + rng.normal(0, 0.2, tokens)).astype(np.float32)
    mask = rng.random(tokens) < 0.8
    logp[~mask] = np.nan
    adv = rng.normal(size=seqs).astype(np.float32)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    size = 1.0 + np.abs(np.where(mask, logp, 0)).sum() * 2
    for m, mean in ((mask, True), (None, False)):
        lp = logp if m is not None else np.where(mask, logp, -1.0).astype(np.float32)
        loss, each, reward, grad = iso.pref_loss(put(torch, lp), put(torch, ref), put(torch, off), mask=put(torch, m), mean=mean)
        w = losses.pref_loss(f(lp), f(ref), m, off, seqs // 2, 0.1, mean=mean)
        near(loss, w[0], size)
        near(each, w[1], size)
        near(reward, w[2], size)
        near(grad, w[3], size)
        for seq_mean in (True, False):
            loss, counts, grad = iso.policy_loss(put(torch, lp), put(torch, old), put(torch, adv), ref_logp=put(torch, ref),
                                                 mask=put(torch, m), seq_off=put(torch, off), kl_coef=0.1, seq_mean=seq_mean)
            w = losses.policy_loss(f(lp), f(old), f(ref), f(adv), m, off, seqs, kl_coef=0.1, seq_mean=seq_mean)
            assert np.array_equal(counts.cpu().numpy(), w[1])
            near(loss, w[0], 100.0 * (1 + seqs))
            near(grad, w[2], w[3] + 1e-3)


@pytest.mark.parametrize("tokens", [64, 20000])
def test_differences_far_from_zero(torch, tokens):
    """Ratios from 1e-45 to beyond f32 and f64, and differences near 0, where exp(u) - 1 - u is small."""
    rng = np.random.default_rng(tokens)
    steps = np.array([0.0, 1e-7, -1e-6, 1e-4, -1e-3, 0.02, -0.3, 0.34, 0.35, -0.36, 1.0, -2.5, 20.0, -40.0, 80.0, -100.0, 690.0,
                      -699.0, 705.0, -710.0, 800.0, -5000.0, 1e30, -1e30])
    d, u = rng.choice(steps[:16], tokens), rng.choice(steps[:16], tokens)
    old = np.full(tokens, -1.0, np.float32)
    logp = (old + d).astype(np.float32)
    ref = (logp + u).astype(np.float32)
    adv = rng.normal(size=tokens).astype(np.float32)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    args = dict(kl_coef=0.5, token_adv=True)
    loss, counts, grad = iso.policy_loss(put(torch, logp), put(torch, old), put(torch, adv), ref_logp=put(torch, ref), **args)
    w = losses.policy_loss(f(logp), f(old), f(ref), f(adv), None, None, 1, **args)
    assert np.array_equal(counts.cpu().numpy(), w[1])
    near(grad, w[2], w[3] + 1e-3)
    near(loss, w[0], np.abs(w[0]).max() + 100.0)
    # beyond f32: infinities and zeros as they are in f32
    d = rng.choice(steps[16:], tokens)
    logp = d.astype(np.float32)
    zero = np.zeros(tokens, np.float32)
    one = np.full(tokens, -1.0, np.float32)  # A < 0: a large ratio is not clipped, a small one is
    _, counts, grad = iso.policy_loss(put(torch, logp), put(torch, zero), put(torch, one), token_adv=True, clip_lo=1.0)
    got = grad.cpu().numpy()
    assert np.all(got[d > 0] == np.inf) and np.all(got[d < 0] == 0.0) and int(counts[1]) == 0
    _, _, grad = iso.policy_loss(put(torch, zero), put(torch, zero), put(torch, zero), ref_logp=put(torch, logp), token_adv=True,
                                 kl_coef=1.0, norm=1.0)
    got = grad.cpu().numpy()
    assert np.all(got[d > 0] == -np.inf) and np.all(got[d < 0] == 1.0)


def test_offsets_are_held_in_large_calls(torch):
    """Broken offsets over many spans and rows: nothing outside the arrays is touched."""
    n = 40000
    store = torch.zeros(3 * n, device="cuda")
    lp = store[n:2 * n]
    lp.fill_(-1.0)
    rng = np.random.default_rng(5)
    for k in range(6):
        off = rng.integers(-2 * n, 3 * n, 301) if k < 3 else np.sort(rng.integers(-n, 2 * n, 301))[::1 if k < 5 else -1]
        o = put(torch, off.astype(np.int32))
        iso.pref_loss(lp, None, o)
        for seq_mean in (True, False):
            iso.policy_loss(lp, lp.clone(), torch.ones(300, device="cuda"), seq_off=o, seq_mean=seq_mean,
                            mask=torch.ones(n, dtype=torch.bool, device="cuda"))
            for rows in (200, 6000):
                x = torch.zeros(rows, 9, device="cuda")
                iso.policy_loss_logits(x, torch.zeros(rows, dtype=torch.int32, device="cuda"), lp[:rows].clone(),
                                       torch.ones(300, device="cuda"), seq_off=o, seq_mean=seq_mean)
        torch.cuda.synchronize()
    assert bool((store[:n] == 0).all()) and bool((store[2 * n:] == 0).all()) and bool((lp == -1).all())


def test_gradients_against_differences(torch):
    """Central differences of the losses' own outputs, with steps that f32 shows: a
    loss is rounded to 2^-24 of itself, so a difference over 2h is off by
    2^-24 |loss| / h, and by h^2 times the third derivative (below 2 here)."""
    rng = np.random.default_rng(9)
    n, h = 6, 2.0 ** -7
    logp = -rng.random(n).astype(np.float32)
    ref, old = (logp + rng.normal(0, 0.1, n)).astype(np.float32), (logp + rng.normal(0, 0.05, n)).astype(np.float32)
    adv = np.array([1.0, -0.5], np.float32)
    calls = {"pref": lambda a: iso.pref_loss(put(torch, a), put(torch, ref), put(torch, np.array([0, 2, 6], np.int32)), beta=0.5),
             "policy": lambda a: iso.policy_loss(put(torch, a), put(torch, old), put(torch, adv), ref_logp=put(torch, ref),
                                                 seq_off=put(torch, np.array([0, 4, 6], np.int32)), kl_coef=0.3, clip_lo=0.5,
                                                 clip_hi=0.5)}
    for name, call in calls.items():
        out = call(logp)
        grad = out[-1].cpu().numpy()
        value = lambda a: float(call(a)[0].reshape(-1)[0])  # noqa: E731
        tol = 2.0 ** -24 * (1.0 + abs(value(logp))) / h + 2 * h * h
        for k in range(n):
            up, down = logp.copy(), logp.copy()
            up[k] += h
            down[k] -= h
            diff = (value(up) - value(down)) / (float(up[k]) - float(down[k]))
            assert abs(diff - grad[k]) <= tol, (name, k, diff, grad[k])


def test_many_replays_of_larger_calls(torch):
    """The calls of several launches, captured and replayed with other work between."""
    n, seqs = 50000, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    s = {k: torch.empty(n, device="cuda") for k in ("lp", "old", "ref")}
    mask = torch.empty(n, dtype=torch.bool, device="cuda")
    off = put(torch, np.concatenate([[0], np.sort(np.random.default_rng(1).integers(0, n, seqs - 1)), [n]]).astype(np.int32))
    x = torch.empty(5000, 130, dtype=torch.float16, device="cuda")
    t = torch.zeros(5000, dtype=torch.int32, device="cuda")
    off2 = put(torch, np.linspace(0, 5000, seqs + 1).astype(np.int32))
    adv = torch.ones(seqs, device="cuda")

    def fill():
        for v in s.values():
            v.copy_(-torch.rand(n, generator=gen, device="cuda"))
        mask.copy_(torch.rand(n, generator=gen, device="cuda") < 0.6)
        x.copy_(torch.randn(5000, 130, generator=gen, device="cuda"))
        t.copy_(torch.randint(-1, 130, (5000,), generator=gen, device="cuda"))
        adv.copy_(torch.randn(seqs, generator=gen, device="cuda"))

    def calls():
        return [*iso.pref_loss(s["lp"], s["ref"], off, mask=mask), *iso.policy_loss(s["lp"], s["old"], adv, ref_logp=s["ref"],
                mask=mask, seq_off=off, kl_coef=0.1, seq_mean=True), *iso.policy_loss(s["lp"], s["old"], adv, mask=mask, seq_off=off),
                *iso.policy_loss_logits(x, t, s["old"][:5000], adv, seq_off=off2, seq_mean=True)]

    fill()
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for k in range(5):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        want = calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k
        assert math.isfinite(float(got[0]))
