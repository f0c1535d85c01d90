"""Token log-probabilities and the losses over them against the plain f64 forms
(oracle/losses.py), through the binding.

Tolerances.  Outputs are rounded once: half a step of their type relative to
the value (f32 2^-24, bf16 2^-8 / 2 steps as torch.finfo(t).eps / 2).  Before
that, sums of exponentials carry the f32 error that losses.token_logp's err
counts (in units of U = 2^-24); the losses themselves are f64 (1e-12 relative
to the sizes summed covers their rounding).
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import losses

pytestmark = pytest.mark.gpu

U = losses.U
TYPES = ("f32", "f16", "bf16")


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


def dtype_of(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def say(*a):
    print(*a, flush=True)


def half(torch, dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(torch, dtype):
    """Half the distance of the type's smallest values (its subnormals), or f32's
    smallest normal value where the exponential flushes below it."""
    return 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126


def make(torch, dtype, rows, vocab, seed, pad=0, shift=0, scale=2.5):
    """Logits in a wider store (row stride vocab + pad, base `shift` elements in), targets, f64 copy."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=gen) * scale).to(dtype)
    store = torch.full((rows * (vocab + pad) + shift + 8,), 7.0, dtype=dtype)
    view = torch.as_strided(store, (rows, vocab), (vocab + pad, 1), shift)
    view.copy_(x)
    dev = store.cuda()
    target = torch.randint(0, vocab, (rows,), generator=gen, dtype=torch.int32)
    return torch.as_strided(dev, (rows, vocab), (vocab + pad, 1), shift), target, x.double().numpy(), dev


def check_logp(torch, got, x, target, temperature, entropy=True):
    lp, lse, ent, err = losses.token_logp(x, target.numpy(), temperature)
    for name, g, w in (("logp", got[0], lp), ("lse", got[1], lse)):
        g = g.double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(w)), name
        ok = np.isfinite(w)
        assert np.array_equal(g[~ok & ~np.isnan(w)], w[~ok & ~np.isnan(w)]), name
        bad = np.abs(g[ok] - w[ok]) - U * (np.abs(w) + err)[ok]
        assert np.all(bad <= 0), (name, bad.max())
    if entropy:
        g = got[2].double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(ent))
        # the entropy's sum of p |z| carries the same roundings, times the distances summed
        ignored = target.numpy() < 0
        assert np.all(g[ignored] == 0)
        for r in np.flatnonzero(np.isfinite(ent) & ~ignored):
            d = np.where(np.isfinite(x[r]), (x[r] - x[r].max()) / temperature, 0.0)
            p = np.exp(np.where(np.isfinite(x[r]), d, -np.inf))
            p = p / p.sum()
            tol = U * (abs(ent[r]) + err[r] + (p * np.abs(d) * (3 * np.abs(d) + 4)).sum() + err[r] * (p * np.abs(d)).sum())
            assert abs(g[r] - ent[r]) <= tol, ("entropy", r, g[r], ent[r], tol)


def check_vjp(torch, grad, x, target, lse, g, ent, gent, temperature, dtype):
    n = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, err = losses.token_logp_vjp(x, target.numpy(), n(lse), n(g), n(ent), n(gent), temperature)
    got = grad.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    tol = err + half(torch, dtype) * np.abs(want) + floor_of(torch, dtype)
    bad = (np.abs(got - want) - tol)[ok]
    assert bad.size == 0 or bad.max() <= 0, bad.max()


SIZES = [(1, 1), (3, 2), (2, 7), (5, 63), (4, 64), (3, 65), (7, 255), (2, 256), (3, 257), (33, 1000), (2, 2047), (2, 4097),
         (300, 515), (5, 16385), (2, 50021), (1, 131072), (3, 131075), (1, 300007)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_token_logp_and_vjp(torch, name, rows, vocab):
    dtype = dtype_of(torch, name)
    say(f"[losses] logp {name} {rows}x{vocab}")
    temperature = 1.0 if vocab % 2 else 0.7
    logits, target, x, _ = make(torch, dtype, rows, vocab, rows * 1000 + vocab, pad=vocab % 5, shift=vocab % 3)
    if rows > 2:
        target[1] = -1
    tg = target.cuda()
    got = iso.token_logp(logits, tg, temperature=temperature, entropy=True)
    check_logp(torch, got, x, target, temperature)
    short = iso.token_logp(logits, tg, temperature=temperature)
    check_logp(torch, short, x, target, temperature, entropy=False)
    gen = torch.Generator().manual_seed(vocab)
    g, gent = torch.randn(rows, generator=gen).cuda(), torch.randn(rows, generator=gen).cuda()
    grad = iso.token_logp_vjp(g, logits, tg, got[1], temperature=temperature)
    check_vjp(torch, grad, x, target, got[1], g, None, None, temperature, dtype)
    grad = iso.token_logp_vjp(g, logits, tg, got[1], temperature=temperature, entropy=got[2], g_entropy=gent)
    check_vjp(torch, grad, x, target, got[1], g, got[2], gent, temperature, dtype)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("vocab", [9, 1000, 70001])
def test_masked_and_broken_rows(torch, name, vocab):
    """Masked entries (-infinity, the type's lowest value), rows of nothing but
    -infinity, NaN and +infinity, targets outside the vocabulary, ignored rows
    of NaN."""
    dtype = dtype_of(torch, name)
    logits, target, x, dev = make(torch, dtype, 10, vocab, vocab)
    target.clamp_(min=1)
    low = torch.finfo(dtype).min
    logits[0, ::2] = -math.inf
    logits[1, : vocab - 1] = low
    logits[2] = -math.inf
    logits[3, vocab // 2] = math.nan
    logits[4, 0] = math.inf
    target[5] = vocab
    logits[6] = math.nan
    target[6] = -1
    logits[7, : vocab - 2] = -math.inf  # one thread's worth of values at the end
    target[7] = vocab - 1
    logits[8] = low
    logits[9, 1:] = -math.inf
    target[9] = 0
    x = logits.double().cpu().numpy()
    tg = target.cuda()
    got = iso.token_logp(logits, tg, entropy=True)
    check_logp(torch, got, x, target, 1.0)
    g = torch.linspace(-1, 1, 10).cuda()
    gent = torch.linspace(0.5, -0.5, 10).cuda()
    grad = iso.token_logp_vjp(g, logits, tg, got[1], entropy=got[2], g_entropy=gent)
    check_vjp(torch, grad, x, target, got[1], g, got[2], gent, 1.0, dtype)
    assert float(grad[6].float().abs().sum()) == 0.0


@pytest.mark.parametrize("name", TYPES)
def test_in_place_and_padding_untouched(torch, name):
    dtype = dtype_of(torch, name)
    logits, target, x, dev = make(torch, dtype, 6, 1003, 5, pad=13, shift=1)
    target[3] = -1
    tg = target.cuda()
    _, lse = iso.token_logp(logits, tg)
    g = torch.linspace(-1, 1, 6).cuda()
    want = iso.token_logp_vjp(g, logits, tg, lse)
    out = torch.full((6, 1500), 9.0, dtype=dtype, device="cuda")
    iso.token_logp_vjp(g, logits, tg, lse, out=out[:, 3:1006])
    assert torch.equal(out[:, 3:1006], want) and bool((out[:, :3] == 9).all()) and bool((out[:, 1006:] == 9).all())
    back = iso.token_logp_vjp(g, logits, tg, lse, out=logits)
    assert back.data_ptr() == logits.data_ptr() and torch.equal(logits, want)
    store = dev.clone()
    torch.as_strided(store, (6, 1003), (1016, 1), 1).fill_(7.0)
    assert bool((store == 7).all())


def test_rows_past_32_bits(torch):
    """Row starts beyond 2^31 elements."""
    rows, vocab, ld = 5, 1001, (1 << 29) + 77
    store = torch.empty(ld * (rows - 1) + vocab, dtype=torch.bfloat16, device="cuda")
    logits = torch.as_strided(store, (rows, vocab), (ld, 1), 0)
    src, target, x, _ = make(torch, torch.bfloat16, rows, vocab, 3)
    logits.copy_(src)
    tg = target.cuda()
    got = iso.token_logp(logits, tg, entropy=True)
    check_logp(torch, got, x, target, 1.0)
    g = torch.ones(rows, device="cuda")
    grad = iso.token_logp_vjp(g, logits, tg, got[1], out=logits)
    check_vjp(torch, grad, x, target, got[1], g, None, None, 1.0, torch.bfloat16)


# ---- sequences ----

def offsets(rng, seqs, tokens):
    return np.concatenate([[0], np.sort(rng.integers(0, tokens + 1, seqs - 1)), [tokens]]).astype(np.int32)


def put(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def near(got, want, sizes, eps=U):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok & ~np.isnan(want)], want[~ok & ~np.isnan(want)])
    bad = (np.abs(got - want) - eps * np.abs(want) - 1e-12 * np.asarray(sizes) - 2.0 ** -149)[ok]
    assert bad.size == 0 or bad.max() <= 0, bad.max()


SHAPES = [(2, 0), (2, 1), (2, 5), (4, 64), (6, 777), (14, 4096), (200, 300), (40, 20011), (2, 70001), (4000, 90001),
          (3000, 2900)]


@pytest.mark.parametrize("variant", ["plain", "smooth-mean", "squared", "squared-mean", "padded", "no-ref"])
@pytest.mark.parametrize("seqs,tokens", SHAPES)
def test_pref_loss(torch, variant, seqs, tokens):
    say(f"[losses] pref {variant} {seqs}x{tokens}")
    rng = np.random.default_rng(seqs + tokens)
    if variant == "padded":
        tokens = tokens // seqs * seqs
    off = None if variant == "padded" else offsets(rng, seqs, tokens)
    logp = -rng.exponential(1.0, tokens).astype(np.float32)
    ref = None if variant == "no-ref" else (logp + rng.normal(0, 0.2, tokens)).astype(np.float32)
    mask = rng.random(tokens) < 0.7 if variant != "plain" else None
    if mask is not None:
        logp[~mask] = rng.choice([np.nan, -np.inf, 3.0], (~mask).sum()).astype(np.float32)
    kw = dict(beta=0.07, label_smoothing=0.1 if variant == "smooth-mean" else 0.0, squared="squared" in variant,
              mean="mean" in variant, grad_scale=3.0)
    shape = (seqs, tokens // seqs) if variant == "padded" else (tokens,)
    to = lambda a: None if a is None else put(torch, a).reshape(shape)  # noqa: E731
    loss, each, reward, grad = iso.pref_loss(to(logp), to(ref), put(torch, off), mask=to(mask), **kw)
    f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    w = losses.pref_loss(f(logp), f(ref), mask, off, seqs // 2, 0.07, kw["label_smoothing"], kw["squared"], kw["mean"], 3.0)
    size = 1.0 + np.abs(np.where(mask, logp, 0) if mask is not None else logp).sum() * 2
    slope = 1.0 + (size if kw["squared"] else 0.0)
    near(loss, w[0], size * slope)
    near(each, w[1], size * slope * (1 + 1 / 0.07))
    near(reward, w[2], size)
    near(grad.reshape(-1), w[3], size)
    only = iso.pref_loss(to(logp), to(ref), put(torch, off), mask=to(mask), grad=False, **kw)
    assert only[3] is None and torch.equal(only[0], loss) and torch.equal(only[1], each)


@pytest.mark.parametrize("variant", ["plain", "seq-mean-kl", "token-adv", "padded", "norm", "clip-edges"])
@pytest.mark.parametrize("seqs,tokens", SHAPES + [(1, 1), (1, 40000), (5000, 120007)])
def test_policy_loss(torch, variant, seqs, tokens):
    say(f"[losses] policy {variant} {seqs}x{tokens}")
    rng = np.random.default_rng(seqs * 3 + tokens)
    if variant == "padded":
        tokens = tokens // seqs * seqs
    off = None if variant == "padded" else offsets(rng, seqs, tokens)
    logp = -rng.exponential(1.0, tokens).astype(np.float32)
    old = (logp + rng.normal(0, 0.25, tokens)).astype(np.float32)
    ref = (logp + rng.normal(0, 0.2, tokens)).astype(np.float32) if variant in ("seq-mean-kl", "padded", "norm") else None
    token_adv = variant in ("token-adv", "clip-edges")
    adv = rng.normal(size=tokens if token_adv else seqs).astype(np.float32)
    if variant == "clip-edges" and tokens:
        adv[rng.random(tokens) < 0.2] = 0.0
    mask = rng.random(tokens) < 0.7 if variant != "plain" else None
    if mask is not None:
        for a in (logp, old, ref):
            if a is not None:
                a[~mask] = rng.choice([np.nan, np.inf, -np.inf], (~mask).sum()).astype(np.float32)
        if token_adv:
            adv[~mask] = np.nan
    kw = dict(clip_lo=1.0 if variant == "clip-edges" else 0.2, clip_hi=math.inf if variant == "clip-edges" else 0.28,
              kl_coef=0.05 if ref is not None else 0.0, seq_mean=variant in ("seq-mean-kl", "norm"), token_adv=token_adv,
              norm=7.5 if variant == "norm" else 0.0, grad_scale=2.0)
    shape = (seqs, tokens // seqs) if variant == "padded" else (tokens,)
    to = lambda a: None if a is None else put(torch, a).reshape(shape)  # noqa: E731
    av = to(adv) if token_adv else put(torch, adv)
    loss, counts, grad = iso.policy_loss(to(logp), to(old), av, ref_logp=to(ref), mask=to(mask),
                                         seq_off=put(torch, off), **kw)
    f = lambda a: None if a is None else a.astype(np.float64)  # noqa: E731
    w = losses.policy_loss(f(logp), f(old), f(ref), f(adv), mask, off, seqs, kw["clip_lo"], kw["clip_hi"], kw["kl_coef"],
                           kw["seq_mean"], token_adv, kw["norm"], 2.0)
    near(loss, w[0], 100.0 * (1 + seqs))
    assert np.array_equal(counts.cpu().numpy(), w[1])
    near(grad.reshape(-1), w[2], w[3] + 1e-3)
    only = iso.policy_loss(to(logp), to(old), av, ref_logp=to(ref), mask=to(mask), seq_off=put(torch, off),
                           grad=False, **kw)
    assert only[2] is None and torch.equal(only[0], loss) and torch.equal(only[1], counts)


def test_live_nan_is_told(torch):
    """A NaN at a live token reaches the loss and its own gradient, no other."""
    logp = torch.full((8,), -1.0, device="cuda")
    logp[3] = math.nan
    loss, _, grad = iso.policy_loss(logp, torch.full((8,), -1.0, device="cuda"), torch.ones(2, device="cuda"),
                                    seq_off=torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    assert bool(torch.isnan(loss[:2]).all()) and torch.isnan(grad).nonzero().flatten().tolist() == [3]
    loss, each, reward, grad = iso.pref_loss(logp.reshape(4, 2), None)
    assert bool(torch.isnan(loss)) and torch.isnan(each).tolist() == [True, False]


# ---- the policy loss from logits ----

HEADS = [(1, 1, 1), (1, 7, 1), (3, 64, 2), (17, 257, 4), (40, 1000, 3), (5, 16385, 1), (130, 4099, 9), (3, 65536, 1),
         (2, 131072, 1), (2, 131075, 2), (1, 262144, 1), (600, 2048, 11), (1, 300007, 1)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,vocab,seqs", HEADS)
def test_policy_loss_logits(torch, name, rows, vocab, seqs):
    dtype = dtype_of(torch, name)
    say(f"[losses] head {name} {rows}x{vocab}/{seqs}")
    rng = np.random.default_rng(rows + vocab)
    temperature = 1.0 if rows % 2 else 1.3
    logits, target, x, _ = make(torch, dtype, rows, vocab, rows * 77 + vocab, pad=vocab % 5, shift=vocab % 2)
    if rows > 2:
        target[rows // 2] = -1
    tgt = target.numpy()
    lp, _, _, err = losses.token_logp(x, tgt, temperature)
    off = offsets(rng, seqs, rows)
    adv = rng.normal(size=seqs).astype(np.float32)
    # ratios away from the clip's borders: far inside, or far outside
    gap = rng.choice([-0.6, -0.1, 0.0, 0.1, 0.6], rows)
    old, ref = (lp + gap).astype(np.float32), (lp + rng.normal(0, 0.3, rows)).astype(np.float32)
    seq_mean, kl = bool(rows % 3), 0.05
    tg, o, r = target.cuda(), put(torch, old), put(torch, ref)
    loss, counts, logp, grad = iso.policy_loss_logits(logits, tg, o, put(torch, adv), ref_logp=r, seq_off=put(torch, off),
                                                      temperature=temperature, kl_coef=kl, seq_mean=seq_mean,
                                                      grad_scale=4.0)
    live = tgt >= 0
    w = losses.policy_loss(lp, old.astype(np.float64), ref.astype(np.float64), adv.astype(np.float64), live, off, seqs,
                           kl_coef=kl, seq_mean=seq_mean, grad_scale=4.0)
    assert np.array_equal(counts.cpu().numpy(), w[1])
    moved = U * (err + 2)  # what logp may be off by
    got = logp.double().cpu().numpy()
    assert np.all(np.abs(got - lp) <= U * np.abs(lp) + moved)
    # the loss moves by its gradient times that, and by its own rounding
    tol = (np.abs(w[2]) / 4.0 * moved + w[3] / 4.0 * moved).sum() * 2 + 1e-12
    for k in range(3):
        assert abs(float(loss[k]) - w[0][k]) <= U * abs(w[0][k]) + tol * (1 if k < 2 else 1 / kl), k
    want, werr = losses.token_logp_vjp(x, tgt, losses.token_logp(x, tgt, temperature)[1], w[2], temperature=temperature)
    shape, _ = losses.token_logp_vjp(x, tgt, losses.token_logp(x, tgt, temperature)[1], np.ones(rows),
                                     temperature=temperature)
    # the coefficient is off by w[3] moved, and rounded once to f32; each p by its row's log-sum
    tol = werr + np.abs(shape) * ((w[3] + np.abs(w[2])) * moved + np.abs(w[2]) * 2 * U)[:, None]
    tol += half(torch, dtype) * np.abs(want) + floor_of(torch, dtype)
    bad = np.abs(grad.double().cpu().numpy() - want) - tol
    assert bad.max() <= 0, bad.max()
    only = iso.policy_loss_logits(logits, tg, o, put(torch, adv), ref_logp=r, seq_off=put(torch, off),
                                  temperature=temperature, kl_coef=kl, seq_mean=seq_mean, grad=False)
    assert only[3] is None and torch.equal(only[2], logp) and torch.equal(only[1], counts)
    back = iso.policy_loss_logits(logits, tg, o, put(torch, adv), ref_logp=r, seq_off=put(torch, off),
                                  temperature=temperature, kl_coef=kl, seq_mean=seq_mean, grad_scale=4.0, out=logits)
    assert torch.equal(back[3], grad) and torch.equal(logits, grad) and torch.equal(back[0], loss)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("vocab", [11, 5000, 70001])
def test_policy_loss_logits_broken_rows(torch, name, vocab):
    """Ignored rows of NaN do nothing; a live broken row has NaN logp and
    gradient, its neighbours' gradients are as without it."""
    dtype = dtype_of(torch, name)
    logits, target, x, _ = make(torch, dtype, 6, vocab, vocab + 1)
    logits[1] = math.nan
    target[1] = -1
    logits[2, ::2] = -math.inf
    target[2] = 1
    tg = target.cuda()
    old = torch.full((6,), -2.0, device="cuda")
    adv = torch.ones(1, device="cuda")
    fine = iso.policy_loss_logits(logits, tg, old, adv)
    assert not any(bool(torch.isnan(v.float()).any()) for v in fine)
    assert float(fine[3][1].float().abs().sum()) == 0.0 and float(fine[3][2, ::2].float().abs().sum()) == 0.0
    logits[4, 0] = math.nan
    target[5] = vocab
    tg = target.cuda()
    loss, counts, logp, grad = iso.policy_loss_logits(logits, tg, old, adv)
    assert bool(torch.isnan(loss[0])) and torch.isnan(logp).nonzero().flatten().tolist() == [4, 5]
    assert bool(torch.isnan(grad[4]).all()) and bool(torch.isnan(grad[5]).all())
    assert torch.equal(grad[:4], fine[3][:4]) and int(counts[0]) == 5


def test_no_rows(torch):
    e = torch.empty(0, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    lp, lse = iso.token_logp(x, t)
    assert lp.numel() == 0 and iso.token_logp_vjp(e, x, t, lse).numel() == 0
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    adv = torch.ones(3, device="cuda")
    loss, counts, g = iso.policy_loss(e, e, adv, seq_off=off)
    assert loss.tolist() == [0, 0, 0] and counts.tolist() == [0, 0]
    loss, counts, _, g = iso.policy_loss_logits(x, t, e, adv, seq_off=off)
    assert loss.tolist() == [0, 0, 0] and counts.tolist() == [0, 0]
    loss, each, reward, g = iso.pref_loss(e, e, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert abs(float(loss) - math.log(2)) < 1e-6 and reward.tolist() == [0, 0]
    loss, each, reward, g = iso.pref_loss(e, None, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert float(loss) == 0.0 and each.numel() == 0


def test_offsets_are_held(torch):
    """Offsets outside the tokens, or falling, touch nothing outside the arrays."""
    n = 5000
    store = torch.zeros(3 * n, device="cuda")
    lp = store[n:2 * n]
    lp.fill_(-1.0)
    for off in ([-100, 40, 1 << 30], [0, 9000, 17], [4000, 30, 5000], [-5, -4, -3], [6000, 7000, 8000]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        iso.pref_loss(lp, None, o)
        iso.policy_loss(lp, lp.clone(), torch.ones(2, device="cuda"), seq_off=o, seq_mean=True)
        x = torch.zeros(50, 9, device="cuda")
        iso.policy_loss_logits(x, torch.zeros(50, dtype=torch.int32, device="cuda"), lp[:50].clone(),
                               torch.ones(2, device="cuda"), seq_off=o, seq_mean=True)
        torch.cuda.synchronize()
    assert bool((store[:n] == 0).all()) and bool((store[2 * n:] == 0).all()) and bool((lp == -1).all())


def every_call(s):
    lp, lse, ent = iso.token_logp(s["x"], s["t"], entropy=True)
    return [lp, lse, ent, iso.token_logp_vjp(s["g"], s["x"], s["t"], lse, entropy=ent, g_entropy=s["g"]),
            *iso.pref_loss(s["lp"], s["ref"], s["off"], mask=s["mask"]),
            *iso.policy_loss(s["lp"], s["ref"], s["adv"], ref_logp=s["ref"], mask=s["mask"], seq_off=s["off"], kl_coef=0.1,
                             seq_mean=True),
            *iso.policy_loss_logits(s["x"], s["t"], s["lp"][:64], s["adv"], ref_logp=s["ref"][:64], seq_off=s["off64"],
                                    kl_coef=0.1)]


def fill(torch, s, seed):
    gen = torch.Generator().manual_seed(seed)
    s["x"].copy_(torch.randn(64, 5003, generator=gen) * 2)
    s["t"].copy_(torch.randint(-1, 5003, (64,), generator=gen))
    for k in ("lp", "ref"):
        s[k].copy_(-torch.rand(30000, generator=gen))
    s["mask"].copy_(torch.rand(30000, generator=gen) < 0.7)
    s["adv"].copy_(torch.randn(4, generator=gen))


def states(torch):
    z = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    return {"x": torch.zeros(64, 5003, dtype=torch.bfloat16, device="cuda"), "t": z(64, i32), "g": z(64) + 0.5,
            "lp": z(30000), "ref": z(30000), "mask": z(30000, torch.bool), "adv": z(4),
            "off": torch.tensor([0, 100, 9000, 9000, 30000], dtype=i32, device="cuda"),
            "off64": torch.tensor([0, 10, 10, 40, 64], dtype=i32, device="cuda")}


def test_results_do_not_depend_on_the_run(torch):
    s = states(torch)
    fill(torch, s, 1)
    a = every_call(s)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, every_call(s)))


def test_another_stream(torch):
    s = states(torch)
    fill(torch, s, 2)
    want = every_call(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    lp, lse, ent = iso.token_logp(s["x"], s["t"], entropy=True, stream=side)
    grad = iso.token_logp_vjp(s["g"], s["x"], s["t"], lse, entropy=ent, g_entropy=s["g"], stream=side)
    loss = iso.policy_loss(s["lp"], s["ref"], s["adv"], ref_logp=s["ref"], mask=s["mask"], seq_off=s["off"], kl_coef=0.1,
                           seq_mean=True, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip([lp, lse, ent, grad], want[:4]))
    assert torch.equal(loss[0], want[8]) and torch.equal(loss[2], want[10])


def test_captured_into_a_graph(torch):
    s = states(torch)
    fill(torch, s, 3)
    every_call(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every_call(s)
    for seed in (4, 5, 6, 7):
        fill(torch, s, seed)
        graph.replay()
        torch.cuda.synchronize()
        want = every_call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), seed
