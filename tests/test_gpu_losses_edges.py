"""The losses where a product of 0 and infinity, a cancellation or a range decides:
references that are only watched, advantages of 0, rows of one value, confident
targets, temperatures and gradients at the ends of their range; and what tests of
values do not show: streams, memory beside the outputs, arrays that begin anywhere.

Tolerances are derived at each test; U is half a step of f32.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import losses
from tests.test_gpu_losses import U, check_logp, check_vjp, dtype_of, floor_of, half, make, near, offsets, put, say, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def far_reference(rng, logp):
    """References whose u = ref - logp is beyond exp's range, infinite or NaN at some tokens."""
    ref = (logp + rng.normal(0, 0.2, logp.size)).astype(np.float32)
    at = rng.choice(logp.size, max(1, logp.size // 3), replace=False)
    ref[at] = rng.choice([750.0, 1e30, np.inf, -np.inf, np.nan], at.size).astype(np.float32)
    return ref


@pytest.mark.parametrize("seqs,tokens", [(2, 7), (6, 777), (40, 20011)])
@pytest.mark.parametrize("seq_mean", [False, True])
def test_a_reference_that_is_only_watched(torch, seqs, tokens, seq_mean):
    """kl_coef 0: the loss has no KL term, so the reference, whatever it holds,
    leaves the loss and its gradient as they are without it, bit by bit."""
    say(f"[losses] watched {seqs}x{tokens}")
    rng = np.random.default_rng(tokens)
    logp = -rng.exponential(1.0, tokens).astype(np.float32)
    old = (logp + rng.normal(0, 0.25, tokens)).astype(np.float32)
    logp[rng.choice(tokens, tokens // 5, replace=False)] = -np.inf  # a live token that the model cannot say
    off, adv = put(torch, offsets(rng, seqs, tokens)), put(torch, rng.normal(size=seqs).astype(np.float32))
    kw = dict(seq_off=off, seq_mean=seq_mean)
    want = iso.policy_loss(put(torch, logp), put(torch, old), adv, **kw)
    for ref in (far_reference(rng, logp), np.full(tokens, -1.0, np.float32)):
        got = iso.policy_loss(put(torch, logp), put(torch, old), adv, ref_logp=put(torch, ref), **kw)
        assert torch.equal(got[0][:2], want[0][:2]) and torch.equal(got[1], want[1])
        assert not bool(torch.isnan(got[2]).any()) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_a_reference_that_is_only_watched_from_logits(torch, name):
    rng = np.random.default_rng(5)
    logits, target, _, _ = make(torch, dtype_of(torch, name), 300, 517, 8)
    rows = torch.arange(0, 300, 7, device="cuda")
    at = target.cuda()
    logits[rows[::2], at[rows[::2]].long()] = -math.inf
    logits[rows[1::2], at[rows[1::2]].long()] = torch.finfo(logits.dtype).min
    old, adv = put(torch, np.full(300, -4.0, np.float32)), put(torch, rng.normal(size=1).astype(np.float32))
    want = iso.policy_loss_logits(logits, at, old, adv)
    ref = put(torch, far_reference(rng, np.full(300, -4.0, np.float32)))
    got = iso.policy_loss_logits(logits, at, old, adv, ref_logp=ref)
    assert torch.equal(got[0][:2], want[0][:2]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert not bool(torch.isnan(got[3]).any()) and torch.equal(got[3], want[3])


@pytest.mark.parametrize("seqs,tokens", [(4, 40), (40, 20011)])
@pytest.mark.parametrize("clip_hi", [0.2, math.inf])
def test_an_advantage_of_zero(torch, seqs, tokens, clip_hi):
    """r A is 0 at A = 0 for every finite difference, also where r is beyond f64."""
    rng = np.random.default_rng(tokens)
    off, adv = offsets(rng, seqs, tokens), rng.normal(size=seqs).astype(np.float32)
    adv[::2] = 0.0
    logp = -rng.exponential(1.0, tokens).astype(np.float32)
    old = (logp + rng.normal(0, 0.25, tokens)).astype(np.float32)
    zero = np.repeat(adv == 0, np.diff(off))
    old[zero] = rng.choice([-800.0, -705.0, -3e38, 3e38, -1.0], zero.sum()).astype(np.float32)
    loss, counts, grad = iso.policy_loss(put(torch, logp), put(torch, old), put(torch, adv), seq_off=put(torch, off),
                                         clip_hi=clip_hi)
    f = lambda a: a.astype(np.float64)  # noqa: E731
    w = losses.policy_loss(f(logp), f(old), None, f(adv), None, off, seqs, hi=clip_hi)
    assert np.all(np.isfinite(w[0])) and np.all(w[2][zero] == 0)
    near(loss, w[0], 100.0 * (1 + seqs))
    near(grad, w[2], w[3] + 1e-3)
    assert np.array_equal(counts.cpu().numpy(), w[1])


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [7, 1000, 70001])
def test_live_rows_of_one_value(torch, name, vocab):
    """A live row that a mask of the type's lowest value (or any one value) fills is
    the uniform distribution: logp = -log V, gradient g ([k = j] - 1/V).  Every
    term and factor is 1 or 1/V, so that log V, the coefficient g and the product
    g/V are rounded once each to f32, and the output once."""
    dtype = dtype_of(torch, name)
    low = torch.finfo(dtype).min
    values = [low, low / 2, -1e4, 0.0, 5.0]
    logits = torch.stack([torch.full((vocab,), v, dtype=dtype, device="cuda") for v in values])
    target = torch.tensor([0, vocab - 1, vocab // 2, 3, 1], dtype=torch.int32, device="cuda")
    old = torch.full((5,), -math.log(vocab), device="cuda")
    for temperature in (1.0, 0.7):
        _, _, logp, grad = iso.policy_loss_logits(logits, target, old, torch.ones(1, device="cuda"), temperature=temperature)
        assert np.all(np.abs(logp.double().cpu().numpy() + math.log(vocab)) <= 2 * U * math.log(vocab))
        # d = logp - old is off by old's rounding, and r = exp(d) with it
        g = -np.exp(-math.log(vocab) - old.double().cpu().numpy())[:, None] / 5 / temperature
        want = np.repeat(g * -1.0 / vocab, vocab, 1)
        want[np.arange(5), target.cpu().numpy()] = g[:, 0] * (1 - 1.0 / vocab)
        bad = np.abs(grad.double().cpu().numpy() - want) - (half(torch, dtype) + 4 * U) * np.abs(want) - floor_of(torch, dtype)
        assert bad.max() <= 0, bad.max()


def confident(torch, dtype, rows, vocab, seed, pad, temperature):
    """Rows whose target leaves 1e-2 to 1e-7 to the others, the targets at the rows' ends and anywhere."""
    logits, target, _, _ = make(torch, dtype, rows, vocab, seed, pad=pad, shift=seed % 3, scale=1.0)
    target[0], target[1] = 0, vocab - 1
    tg = target.cuda()
    x = logits.double().cpu().numpy()
    x[np.arange(rows), target.numpy()] = -np.inf
    rest = np.log(np.exp(x / temperature).sum(1))
    lift = torch.from_numpy((rest + np.linspace(math.log(1e2), math.log(1e7), rows)) * temperature)
    logits[torch.arange(rows, device="cuda"), tg.long()] = lift.to(dtype).cuda()
    return logits, target, logits.double().cpu().numpy()


CONFIDENT = [(24, 11), (24, 1000), (140, 4099), (24, 32003), (12, 70001), (6, 131075)]


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", CONFIDENT)
def test_confident_targets_vjp(torch, name, rows, vocab):
    """The target's entry g (1 - p) / T keeps its relative accuracy, p at the given
    log-sum: f64 up to one rounding to f32 and one to the type; z = x/T - lse and the
    entropy's z + H are off by a few of f64's steps of their parts."""
    dtype = dtype_of(torch, name)
    say(f"[losses] confident vjp {name} {rows}x{vocab}")
    for temperature in (1.0, 0.7):
        logits, target, x = confident(torch, dtype, rows, vocab, rows + vocab, vocab % 4, temperature)
        tg = target.cuda()
        _, lse, ent = iso.token_logp(logits, tg, temperature=temperature, entropy=True)
        gen = torch.Generator().manual_seed(rows)
        g, gent = torch.randn(rows, generator=gen).cuda(), torch.randn(rows, generator=gen).cuda()
        n = lambda t: t.double().cpu().numpy()  # noqa: E731
        at = np.arange(rows), target.numpy()
        xt = x[at] / temperature
        z = xt - n(lse)
        step = 2.0 ** -50 * (np.abs(xt) + np.abs(n(lse)))
        for entropies in (False, True):
            kw = dict(entropy=ent, g_entropy=gent) if entropies else {}
            for out in (None, logits.clone()):  # in place too
                src = logits if out is None else out
                grad = n(iso.token_logp_vjp(g, src, tg, lse, temperature=temperature, out=out, **kw))[at]
                want = -n(g) * np.expm1(z)
                moved = np.abs(n(g)) * step
                if entropies:
                    want = want - n(gent) * np.exp(z) * (z + n(ent))
                    moved = moved + np.abs(n(gent)) * (step + 2.0 ** -50 * np.abs(n(ent)))
                tol = (half(torch, dtype) + 2 * U) * np.abs(want) + moved
                bad = np.abs(grad - want / temperature) - tol / temperature - floor_of(torch, dtype)
                assert bad.max() <= 0, (temperature, entropies, bad.max())


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", CONFIDENT)
def test_confident_targets_from_logits(torch, name, rows, vocab):
    """The same in the loss from logits.  1 - p is the sum of the other entries'
    p, each off by its exponent's three roundings, its exp's two half steps and two a
    rescaling of the running sums (one a chunk, 16 at most here, and three joins);
    r = exp(logp - old) = 1 moves by what logp moves."""
    dtype = dtype_of(torch, name)
    say(f"[losses] confident head {name} {rows}x{vocab}")
    for temperature in (1.0, 0.7):
        logits, target, x = confident(torch, dtype, rows, vocab, rows + vocab, vocab % 4, temperature)
        at = np.arange(rows), target.numpy()
        z = (x - x[at][:, None]) / temperature
        others = np.exp(z)
        others[at] = 0.0
        s = others.sum(1)
        lp = -np.log1p(s)
        adv = torch.full((1,), 2.0, device="cuda")
        old = lp.astype(np.float32)
        for out in (None, logits.clone()):
            src = logits if out is None else out
            _, _, logp, grad = iso.policy_loss_logits(src, target.cuda(), put(torch, old), adv, temperature=temperature, out=out)
            off = U * ((others * (3 * np.abs(z) + 2)).sum(1) / s + 2 * 19) + 2.0 ** -50 / s
            assert np.all(np.abs(logp.double().cpu().numpy() - lp) <= (U + off) * np.abs(lp))
            want = -2.0 / rows * np.exp(lp - old.astype(np.float64)) * (s / (1 + s)) / temperature
            got = grad.double().cpu().numpy()[at]
            tol = (half(torch, dtype) + 2 * U + 2 * off) * np.abs(want) + floor_of(torch, dtype)
            assert np.all(np.abs(got - want) <= tol), (temperature, (np.abs(got - want) - tol).max())


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [9, 5000, 50021])
def test_temperatures_at_the_ends(torch, name, vocab):
    """1e-28: the largest logit takes all; 1e28: every distribution is uniform."""
    dtype = dtype_of(torch, name)
    logits, target, x, _ = make(torch, dtype, 6, vocab, vocab)
    logits[2, ::2] = -math.inf
    logits[3, 1:] = torch.finfo(dtype).min
    target[2], target[4] = 1, int(x[4].argmax())
    x = logits.double().cpu().numpy()
    tg, g = target.cuda(), torch.linspace(-1, 1, 6).cuda()
    for temperature in (1e-28, 1e28):
        got = iso.token_logp(logits, tg, temperature=temperature, entropy=True)
        lp, lse, ent, err = losses.token_logp(x, target.numpy(), temperature)
        for v, w in ((got[0], lp), (got[1], lse), (got[2], ent)):
            v = v.double().cpu().numpy()
            with np.errstate(over="ignore"):
                w32 = w.astype(np.float32).astype(np.float64)
            same = np.isinf(w32)
            assert np.array_equal(v[same], w32[same])
            assert np.all(np.abs(v - w)[~same] <= (U * (np.abs(w) + err))[~same])
        if temperature > 1:
            grad = iso.token_logp_vjp(g, logits, tg, got[1], temperature=temperature)
            check_vjp(torch, grad, x, target, got[1], g, None, None, temperature, dtype)
        old = put(torch, np.maximum(lp, -3e38).astype(np.float32))
        out = iso.policy_loss_logits(logits, tg, old, torch.ones(1, device="cuda"), temperature=temperature)
        assert torch.equal(out[2], got[0]) and not bool(torch.isnan(out[3]).any())


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("scale,temperature", [(1e9, 1.0), (1e20, 1.0), (1.0, 1e-10), (1e12, 0.7)])
def test_large_entropy_gradients_of_masked_entries(torch, name, scale, temperature):
    """A masked entry's gradient is 0 whatever g_entropy / T is."""
    dtype = dtype_of(torch, name)
    logits, target, _, _ = make(torch, dtype, 8, 1003, 3)
    logits *= temperature
    logits[:, 1::3] = -math.inf
    logits[:, 2::3] = torch.finfo(dtype).min
    target = target // 3 * 3
    x = logits.double().cpu().numpy()
    tg = target.cuda()
    _, lse, ent = iso.token_logp(logits, tg, temperature=temperature, entropy=True)
    g, gent = torch.linspace(-1, 1, 8).cuda(), torch.linspace(1, -1, 8).cuda() * scale
    grad = iso.token_logp_vjp(g, logits, tg, lse, temperature=temperature, entropy=ent, g_entropy=gent)
    check_vjp(torch, grad, x, target, lse, g, ent, gent, temperature, dtype)
    assert bool((grad[:, 1::3] == 0).all()) and bool((grad[:, 2::3] == 0).all())


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1000003), (3, 300007), (2, 131075), (140, 70001), (200, 50021), (260, 24577), (700, 16391),
                                        (40, 8195), (2000, 2051), (300, 1025)])
def test_every_entry_counts_once(torch, name, rows, vocab):
    """In a row of one value every term and factor is exactly 1: the sum is V, and
    log V is rounded once.  An entry left out or taken twice is 1 / V."""
    logits = torch.full((rows, vocab), 1.5, dtype=dtype_of(torch, name), device="cuda")
    target = torch.arange(rows, dtype=torch.int32, device="cuda")
    logp, lse, ent = iso.token_logp(logits, target, entropy=True)
    old = torch.full((rows,), -math.log(vocab), device="cuda")
    head = iso.policy_loss_logits(logits, target, old, torch.ones(1, device="cuda"))[2]
    tol = U * math.log(vocab) + 1e-12
    assert tol < 0.9 / vocab
    for v, w in ((logp, -math.log(vocab)), (ent, math.log(vocab)), (head, -math.log(vocab))):
        assert np.all(np.abs(v.double().cpu().numpy() - w) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - 1.5 - math.log(vocab)) <= U * (1.5 + math.log(vocab)) + 1e-12)


class Arena:
    """Device memory filled with a pattern, of which pieces are handed out with guards around them."""

    GUARD = 8192

    def __init__(self, torch, nbytes):
        self.torch = torch
        self.mem = torch.full((nbytes,), 0xA5, dtype=torch.uint8, device="cuda")
        self.end, self.used = self.GUARD, []

    def take(self, nbytes):
        at = self.end
        assert at + nbytes + self.GUARD <= self.mem.numel()
        self.used.append((at, at + nbytes))
        self.end = (at + nbytes + 255) // 256 * 256 + self.GUARD
        return self.mem.data_ptr() + at

    def untouched(self):
        """Every byte outside the pieces still holds the pattern."""
        keep = self.mem.clone()
        for a, b in self.used:
            keep[a:b] = 0xA5
        return bool((keep == 0xA5).all())


def broken_offsets(rng, seqs, n):
    yield rng.integers(-2 * n, 3 * n, seqs + 1)
    yield rng.integers(-2 ** 31, 2 ** 31, seqs + 1)
    yield np.sort(rng.integers(-n, 2 * n, seqs + 1))
    yield np.sort(rng.integers(0, n + 1, seqs + 1))[::-1]
    yield np.full(seqs + 1, n // 2)
    yield np.full(seqs + 1, n)
    yield np.full(seqs + 1, -1)
    yield np.full(seqs + 1, 2 ** 31 - 1)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("seqs,n", [(2, 100), (300, 5000), (2, 40000), (300, 40001), (9000, 20011)])
def test_nothing_beside_the_outputs_is_written(torch, seqs, n, masked):
    """Outputs and workspaces of exactly the sizes asked for, between guards, in calls with broken offsets."""
    say(f"[losses] guards {seqs}x{n} masked={masked}")
    rng = np.random.default_rng(seqs + n)
    lp = torch.full((n,), -1.0, device="cuda")
    mask = put(torch, rng.random(n) < 0.7) if masked else None
    adv = torch.ones(seqs, device="cuda")
    vocab = 9
    logits = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    target = torch.zeros(n, dtype=torch.int32, device="cuda")
    if masked:
        target[~mask] = -1
    m = None if mask is None else mask.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    sizes = [iso.iso_pref_loss_workspace_bytes(n, seqs // 2), iso.iso_policy_loss_workspace_bytes(n, seqs),
             iso.iso_policy_loss_logits_workspace_bytes(n, vocab, seqs, iso.ISO_DT_BF16)]
    for off in broken_offsets(rng, seqs, n):
        o = put(torch, off.astype(np.int32))
        for flags in (0, 1):
            a = Arena(torch, 2 * sum(sizes) + 40 * (n + seqs) + 20 * (Arena.GUARD + 256))
            st = iso.iso_pref_loss(lp.data_ptr(), None, m, o.data_ptr(), seqs // 2, n, 0.1, 0.0, a.take(4), a.take(2 * seqs),
                                   a.take(4 * seqs), a.take(4 * n), 1.0, a.take(sizes[0]), sizes[0], stream, flags)
            assert st == iso.ISO_OK
            for token_adv in (0, iso.ISO_POLICY_ADV_TOKEN):
                av = lp.data_ptr() if token_adv else adv.data_ptr()
                st = iso.iso_policy_loss(lp.data_ptr(), lp.data_ptr(), lp.data_ptr(), av, m, o.data_ptr(), seqs, n, 0.2, 0.2, 0.1,
                                         0.0, a.take(12), a.take(8), a.take(4 * n), 1.0, a.take(sizes[1]), sizes[1], stream,
                                         flags | token_adv)
                assert st == iso.ISO_OK
            st = iso.iso_policy_loss_logits(logits.data_ptr(), iso.ISO_DT_BF16, n, vocab, vocab, target.data_ptr(), 1.0,
                                            lp.data_ptr(), None, adv.data_ptr(), o.data_ptr(), seqs, 0.2, 0.2, 0.0, 0.0,
                                            a.take(12), a.take(8), a.take(4 * n), a.take(2 * n * vocab), vocab, 1.0,
                                            a.take(sizes[2]), sizes[2], stream, flags)
            assert st == iso.ISO_OK
            torch.cuda.synchronize()
            assert a.untouched(), (off[:4], flags)


@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 257), (5, 16385), (3, 131075), (130, 50021), (700, 2049)])
def test_nothing_beside_the_logits_outputs_is_written(torch, rows, vocab):
    code, ld = iso.ISO_DT_BF16, vocab + 3
    size = iso.iso_token_logp_workspace_bytes(rows, vocab, code)
    logits = torch.randn(rows, vocab, device="cuda").bfloat16()
    target = torch.arange(rows, dtype=torch.int32, device="cuda") % (vocab + 2) - 1  # ignored, in the vocabulary, past it
    g = torch.ones(rows, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for shift in (0, 1, 3):
        a = Arena(torch, size + 2 * rows * ld + 12 * rows + 6 * (Arena.GUARD + 512))
        logp, lse, ent = a.take(4 * rows), a.take(4 * rows), a.take(4 * rows)
        st = iso.iso_token_logp(logits.data_ptr(), code, rows, vocab, vocab, target.data_ptr(), 1.0, logp, lse, ent, a.take(size),
                                size, stream)
        assert st == iso.ISO_OK
        grad = a.take(2 * shift + 2 * rows * ld) + 2 * shift
        a.used.pop()
        base = grad - a.mem.data_ptr()
        a.used += [(base + 2 * ld * r, base + 2 * ld * r + 2 * vocab) for r in range(rows)]  # without the padding
        st = iso.iso_token_logp_vjp(logits.data_ptr(), code, rows, vocab, vocab, target.data_ptr(), 1.0, lse, ent, g.data_ptr(),
                                    g.data_ptr(), grad, ld, stream)
        assert st == iso.ISO_OK
        torch.cuda.synchronize()
        assert a.untouched(), shift


def stream_calls(s, **kw):
    lp, lse, ent = iso.token_logp(s["x"], s["t"], entropy=True, **kw)
    return [lp, lse, ent, iso.token_logp_vjp(s["g"], s["x"], s["t"], s["lse"], entropy=s["ent"], g_entropy=s["g"], **kw),
            *iso.pref_loss(s["lp"], s["ref"], s["off"], mask=s["mask"], **kw),
            *iso.policy_loss(s["lp"], s["ref"], s["adv"], ref_logp=s["ref"], mask=s["mask"], seq_off=s["off"], kl_coef=0.1,
                             seq_mean=True, **kw),
            *iso.policy_loss_logits(s["x"], s["t"], s["old"], s["adv"], ref_logp=s["lse"], seq_off=s["off64"], kl_coef=0.1,
                                    seq_mean=True, **kw)]


def stream_inputs(torch, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(64, 5003, generator=gen) * 2
    s = {"x": x.bfloat16(), "t": torch.randint(-1, 5003, (64,), generator=gen, dtype=torch.int32), "g": torch.randn(64, generator=gen),
         "lse": torch.logsumexp(x, 1), "ent": torch.rand(64, generator=gen) + 5, "lp": -torch.rand(30000, generator=gen),
         "ref": -torch.rand(30000, generator=gen), "old": -torch.rand(64, generator=gen) - 8,
         "mask": torch.rand(30000, generator=gen) < 0.7, "adv": torch.randn(4, generator=gen),
         "off": torch.tensor([0, 100 + seed, 9000, 9000, 30000], dtype=torch.int32),
         "off64": torch.tensor([0, 10 + seed, 20, 40, 64], dtype=torch.int32)}
    return {k: v.cuda() for k, v in s.items()}


def busy(torch, block):
    """Some tens of milliseconds of copies on the current stream."""
    for _ in range(200):
        block[1].copy_(block[0])


def test_calls_run_on_the_stream_they_are_given(torch):
    """New inputs are copied in on the other stream, behind other work there: a call
    that ran anywhere else would take the old ones."""
    s, new = stream_inputs(torch, 1), stream_inputs(torch, 2)
    block = torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    stream_calls(s)
    before = stream_calls(s)
    want = stream_calls(new)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy(torch, block)
        for k in s:
            s[k].copy_(new[k])
    got = stream_calls(s, stream=side)
    side.synchronize()
    for k, (a, b, c) in enumerate(zip(got, want, before)):
        assert torch.equal(a, b), k
        assert b.dtype == torch.int32 or not torch.equal(b, c), k  # the old inputs would have shown


def test_inputs_dropped_after_a_call_on_another_stream(torch):
    """The call still waits behind other work when its inputs are dropped and their sizes taken again and overwritten."""
    keep = stream_inputs(torch, 3)
    block = torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    want = stream_calls(keep)
    for v in keep.values():
        torch.empty_like(v).fill_(1)  # its kernels are loaded by now
    torch.cuda.synchronize()
    mine = {k: v.clone() for k, v in keep.items()}
    places = {v.data_ptr() for v in mine.values()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        busy(torch, block)
    got = stream_calls(mine, stream=side)
    mine.clear()
    again = [torch.empty_like(v) for v in keep.values()]
    assert not side.query()  # the calls have not run yet
    for v in again:
        v.fill_(1)  # on the current stream, at once
    assert not places & {v.data_ptr() for v in again}
    side.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), k


def placed(torch, a, shift):
    """A copy of a that begins `shift` elements into a buffer."""
    store = torch.empty(a.numel() + shift + 8, dtype=a.dtype, device="cuda")
    view = store[shift:shift + a.numel()]
    view.copy_(a)
    return view


@pytest.mark.parametrize("seqs,tokens", [(4, 777), (6, 8192), (40, 20011), (2, 70002), (3000, 90001)])
@pytest.mark.parametrize("shifts", [(1, 2, 3, 1), (2, 3, 1, 2), (3, 1, 2, 3)])
def test_token_arrays_that_begin_anywhere(torch, seqs, tokens, shifts):
    """Tokens' arrays at every multiple of their element and masks at every byte: the
    values do not depend on where they lie."""
    say(f"[losses] places {seqs}x{tokens} {shifts}")
    rng = np.random.default_rng(tokens)
    torch.manual_seed(tokens)
    logp = put(torch, -rng.exponential(1.0, tokens).astype(np.float32))
    old, ref = logp + 0.2 * torch.randn(tokens, device="cuda"), logp + 0.2 * torch.randn(tokens, device="cuda")
    mask = put(torch, rng.random(tokens) < 0.7)
    off = put(torch, offsets(rng, seqs, tokens))
    adv, per = torch.randn(seqs, device="cuda"), torch.randn(tokens, device="cuda")
    a, b, c, d = shifts
    p = lambda t, k: placed(torch, t, k)  # noqa: E731
    for m in (None, mask):
        pm = None if m is None else p(m, d)
        for mean in (False, True):
            want = iso.pref_loss(logp, ref, off, mask=m, mean=mean)
            got = iso.pref_loss(p(logp, a), p(ref, b), p(off, c), mask=pm, mean=mean)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            for token_adv in (False, True):
                kw = dict(kl_coef=0.1, seq_mean=mean, token_adv=token_adv)
                av = per if token_adv else adv
                want = iso.policy_loss(logp, old, av, ref_logp=ref, mask=m, seq_off=off, **kw)
                got = iso.policy_loss(p(logp, a), p(old, b), p(av, c), ref_logp=p(ref, d), mask=pm, seq_off=p(off, a), **kw)
                assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("rows,seqs", [(40, 3), (300, 5), (9001, 7)])
def test_rows_arrays_that_begin_anywhere(torch, rows, seqs):
    rng = np.random.default_rng(rows)
    torch.manual_seed(rows)
    logits = torch.randn(rows, 67, device="cuda").half()
    target = put(torch, rng.integers(-1, 67, rows).astype(np.int32))
    old, ref = put(torch, -rng.random(rows).astype(np.float32) - 3), put(torch, -rng.random(rows).astype(np.float32) - 3)
    off, adv = put(torch, offsets(rng, seqs, rows)), torch.randn(seqs, device="cuda")
    p = lambda t, k: placed(torch, t, k)  # noqa: E731
    logp, lse, ent = iso.token_logp(logits, target, entropy=True)
    grad = iso.token_logp_vjp(old, logits, target, lse, entropy=ent, g_entropy=ref)
    head = iso.policy_loss_logits(logits, target, old, adv, ref_logp=ref, seq_off=off, kl_coef=0.1, seq_mean=True)
    for k in (1, 2, 3):
        got = iso.token_logp(logits, p(target, k), entropy=True)
        assert all(torch.equal(x, y) for x, y in zip(got, (logp, lse, ent)))
        assert torch.equal(iso.token_logp_vjp(p(old, k), logits, p(target, k), p(lse, k), entropy=p(ent, k), g_entropy=p(ref, k)), grad)
        got = iso.policy_loss_logits(logits, p(target, k), p(old, k), p(adv, k), ref_logp=p(ref, k), seq_off=p(off, k), kl_coef=0.1,
                                     seq_mean=True)
        assert all(torch.equal(x, y) for x, y in zip(got, head))


@pytest.mark.parametrize("rows,vocab,name", [(36000, 1000, "f32"), (70000, 1003, "bf16"), (800, 50021, "f32"), (400, 99991, "f32"),
                                             (200, 180001, "f32"), (150, 500009, "f16"), (100, 700001, "bf16")])
def test_streamed_logits_in_every_workgroup_shape(torch, rows, vocab, name):
    """Calls past 128 MB, which read past the caches, by 64, 256, 512 and 1024 threads, whole rows and pieces."""
    dtype = dtype_of(torch, name)
    say(f"[losses] streamed {rows}x{vocab} {name}")
    assert rows * vocab * torch.finfo(dtype).bits // 8 > 128 << 20
    torch.manual_seed(rows)
    logits = (2 * torch.randn(rows, vocab, device="cuda")).to(dtype)
    target = torch.randint(0, vocab, (rows,), device="cuda").to(torch.int32)
    target[rows // 3] = -1
    got = iso.token_logp(logits, target, entropy=True)
    short = iso.token_logp(logits, target)
    pick = torch.tensor([0, 1, rows // 3, rows // 2, rows - 2, rows - 1], device="cuda")
    x, t = logits[pick].double().cpu().numpy(), target[pick].cpu()
    check_logp(torch, [v[pick] for v in got], x, t, 1.0)
    check_logp(torch, [v[pick] for v in short], x, t, 1.0, entropy=False)


@pytest.mark.parametrize("tokens", [5, 20011])
@pytest.mark.parametrize("place", [0, 4])
def test_an_infinite_difference_to_the_reference(torch, tokens, place):
    """exp(u) - u - 1 is infinite at both infinities of u, and so is its sum, beside a finite loss."""
    logp, ref = torch.full((tokens,), -1.0, device="cuda"), torch.full((tokens,), -1.1, device="cuda")
    old, adv = logp.clone(), torch.ones(1, device="cuda")
    for a in (logp, ref):
        b = a.clone()
        b[place] = -math.inf
        args = (b, ref) if a is logp else (logp, b)
        loss, _, grad = iso.policy_loss(args[0], old, adv, ref_logp=args[1])
        assert float(loss[2]) == math.inf and math.isfinite(float(loss[0])) and bool(torch.isfinite(grad).all())
        loss, _, grad = iso.policy_loss(args[0], old, adv, ref_logp=args[1], kl_coef=0.5)
        assert float(loss[2]) == math.inf and float(loss[0]) == math.inf
        want = -math.inf if a is logp else -1.0 / tokens + 0.5 / tokens  # -r A + kl_coef (1 - exp(u))
        got = float(grad[place])
        assert got == want or abs(got - want) <= 4 * U * abs(want)
