"""The decoding steps against their plain forms (oracle/decoding.py), through the
binding.

Whole numbers and copies are equal.  A score or log-probability is off by half a
step of f32 and by what its row's log-sum may be (decoding.row_logp's err in
units of U = 2^-24); a candidate may stand in another's place where their ranks
differ by less than the two may be off.
"""
from __future__ import annotations

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import decoding

pytestmark = pytest.mark.gpu

U = decoding.U
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


def place(torch, x, dtype, pad=0, shift=0):
    """x as a matrix in a wider store: row stride columns + pad, `shift` elements in."""
    rows, cols = x.shape
    store = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=dtype)
    torch.as_strided(store, (rows, cols), (cols + pad, 1), shift).copy_(x)
    return torch.as_strided(store.cuda(), (rows, cols), (cols + pad, 1), shift)


def n(t):
    return None if t is None else t.cpu().numpy()


def check_select(got, x, score, take, weight=None, ended=None, end_token=-1, temperature=1.0):
    batch, beams = score.shape
    out, logp, parent, token = (n(t) for t in got)
    assert out.shape == logp.shape == parent.shape == token.shape == (batch, take)
    for b, want in enumerate(decoding.beam_select(x, n(score), take, n(weight), n(ended), end_token, temperature)):
        count = min(take, len(want))
        assert np.all(parent[b, count:] == -1) and np.all(token[b, count:] == -1), (b, count)
        assert np.all(np.isneginf(out[b, count:])) and np.all(np.isneginf(logp[b, count:]))
        by = {(c["parent"], c["token"]): c for c in want}
        seen, last = set(), {}
        for i in range(count):
            key = (int(parent[b, i]), int(token[b, i]))
            assert key in by and key not in seen, (b, i, key)
            seen.add(key)
            c, w = by[key], want[i]
            assert abs(float(logp[b, i]) - c["logp"]) <= U * (abs(c["logp"]) + c["err"]), (b, i)
            assert abs(float(out[b, i]) - c["score"]) <= U * (abs(c["score"]) + c["err"]), (b, i)
            if c is not w:
                off = U * (2 * abs(c["rank"]) + 2 * abs(w["rank"]) + c["w"] * c["err"] + w["w"] * w["err"])
                assert abs(c["rank"] - w["rank"]) <= off, (b, i, c, w)
            # a beam's own candidates come in the order of their logits
            assert last.get(c["parent"], -1) < c["place"], (b, i)
            last[c["parent"]] = c["place"]


SIZES = [(1, 1, 1, 1), (2, 3, 2, 4), (1, 4, 7, 4), (3, 2, 63, 5), (2, 2, 64, 64), (1, 5, 65, 10), (4, 1, 255, 1), (2, 8, 1000, 16),
         (33, 2, 515, 2), (1, 128, 300, 128), (2, 3, 4095, 6), (2, 3, 4097, 6), (1, 2, 8191, 33), (1, 2, 8193, 128), (3, 3, 16385, 3),
         (2, 4, 50021, 8), (1, 4, 131072, 4), (1, 2, 300007, 20)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("batch,beams,vocab,take", SIZES)
def test_select(torch, name, batch, beams, vocab, take):
    say(f"[decoding] select {name} {batch}x{beams}x{vocab} take {take}")
    dtype, rows = dtype_of(torch, name), batch * beams
    gen = torch.Generator().manual_seed(rows * 1000 + vocab)
    x = (torch.randn(rows, vocab, generator=gen) * 2.5).to(dtype)
    score = -5 * torch.rand(batch, beams, generator=gen)
    temperature = 1.0 if vocab % 2 else 0.7
    logits = place(torch, x, dtype, pad=vocab % 5, shift=vocab % 3)
    got = iso.beam_select(logits, score.cuda(), take=take, temperature=temperature)
    check_select(got, x.double().numpy(), score, take, temperature=temperature)
    # the same with ended beams, weights and forbidden tokens
    ended = torch.rand(batch, beams, generator=gen) < 0.3
    weight = 0.2 + torch.rand(batch, beams, generator=gen)
    x[torch.rand(rows, vocab, generator=gen) < 0.4] = -float("inf")
    logits = place(torch, x, dtype, pad=vocab % 3, shift=vocab % 7)
    got = iso.beam_select(logits, score.cuda(), take=take, weight=weight.cuda(), ended=ended.cuda(), end_token=vocab // 2,
                          temperature=temperature)
    check_select(got, x.double().numpy(), score, take, weight, ended, vocab // 2, temperature)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("vocab", [9, 700, 9001, 40000])
def test_select_rows_without_candidates(torch, name, vocab):
    """NaN, infinities, scores and weights that leave a beam nothing, alone and together."""
    dtype, inf, nan = dtype_of(torch, name), float("inf"), float("nan")
    gen = torch.Generator().manual_seed(vocab)
    say(f"[decoding] empty rows {name} {vocab}")
    batch, beams, take = 4, 6, 7
    x = torch.randn(batch * beams, vocab, generator=gen).to(dtype)
    x[0] = -inf
    x[1, vocab // 2] = nan
    x[2, vocab - 1] = inf
    x[3, 1:] = -inf
    x[4] = torch.finfo(dtype).min
    x[6:12] = -inf  # an item of nothing
    score = -torch.rand(batch, beams, generator=gen)
    score[2] = torch.tensor([-inf, nan, inf, -1.0, -2.0, -inf])
    score[3, 1:] = -inf  # a first step
    weight = torch.ones(batch, beams)
    weight[2, 3] = 0.0
    for w in (None, weight):
        got = iso.beam_select(place(torch, x, dtype, 3, 1), score.cuda(), take=take, weight=None if w is None else w.cuda())
        check_select(got, x.double().numpy(), score, take, w)
    weight[0] = torch.tensor([nan, -1.0, inf, 0.0, 1e-30, 1e30])
    ended = torch.zeros(batch, beams, dtype=torch.bool)
    ended[1, 2] = ended[0, 1] = ended[2, 0] = True
    got = iso.beam_select(place(torch, x, dtype, 3, 1), score.cuda(), take=take, weight=weight.cuda(), ended=ended.cuda(), end_token=3)
    check_select(got, x.double().numpy(), score, take, weight, ended, 3)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("vocab,take", [(5, 8), (1000, 16), (20001, 64), (70000, 128)])
def test_select_ties(torch, name, vocab, take):
    """Equal logits by the lower token, equal beams by the lower beam; -0 is 0."""
    say(f"[decoding] ties {name} {vocab} take {take}")
    dtype = dtype_of(torch, name)
    x = torch.zeros(4, vocab).to(dtype)
    x[1::2] = -x[1::2]
    x[2, ::2] = 1.0
    x[3, ::2] = 1.0
    score = torch.zeros(2, 2)
    out, logp, parent, token = (n(t) for t in iso.beam_select(place(torch, x, dtype, 1, 1), score.cuda(), take=take))
    k = min(take, vocab)
    assert token[0, :k].tolist() == list(range(k)) and np.all(parent[0, :k] == 0)
    assert token[0, k:].tolist() == list(range(vocab))[:take - k] and np.all(parent[0, k:k + vocab] == 1)
    most = (vocab + 1) // 2
    want = [(2, 2 * i) for i in range(most)] + [(3, 2 * i) for i in range(most)]
    want += [(2, 2 * i + 1) for i in range(vocab // 2)] + [(3, 2 * i + 1) for i in range(vocab // 2)]
    assert list(zip(parent[1].tolist(), token[1].tolist()))[:take] == want[:take]


@pytest.mark.parametrize("rising", [True, False])
def test_select_of_sorted_logits(torch, rising):
    """The best tokens all lie in one place."""
    vocab, take = 50001, 128
    x = torch.arange(vocab, dtype=torch.float32) / 3000.0
    x = (x if rising else x.flip(0)).repeat(3, 1)
    score = torch.tensor([[-0.1, -0.3, -0.2]])
    got = iso.beam_select(place(torch, x, torch.float32, 0, 1), score.cuda(), take=take)
    check_select(got, x.double().numpy(), score, take)


# ---- states ----

def raw(torch, gen, shape, dtype):
    if dtype == torch.bool:
        return torch.rand(shape, generator=gen) < 0.5
    if dtype.is_floating_point:
        return torch.randn(shape, generator=gen).to(dtype)
    return torch.randint(-100, 100, shape, generator=gen).to(dtype)


REORDER = [("float32", (6, 5), 0), ("bfloat16", (2, 6, 3, 7, 5), 1), ("int64", (6,), 0), ("uint8", (6, 37), 0), ("bool", (3, 6), 1),
           ("float16", (2, 2, 6, 9), 2), ("float64", (6, 4, 2), 0), ("int32", (6, 1), 0), ("float32", (4, 6, 1111), 1),
           ("uint8", (5, 6, 3), 1), ("bfloat16", (2, 6, 4, 130, 64), 1)]


@pytest.mark.parametrize("batch,beams", [(1, 6), (2, 3), (6, 1), (3, 2)])
def test_reorder(torch, batch, beams):
    """Several states of several types and places in one call, and each by itself."""
    gen = torch.Generator().manual_seed(batch)
    rng = np.random.default_rng(batch)
    for trial in range(4):
        parent = (rng.integers(0, beams, (batch, beams)) + np.arange(batch)[:, None] * beams).astype(np.int32)
        if trial == 1:
            parent[:] = np.arange(6).reshape(batch, beams)
        if trial == 2:  # no rows, and rows of other items: they stay
            parent = rng.integers(-2, 8, (batch, beams)).astype(np.int32)
        if trial == 3:  # a cycle
            parent = (np.roll(np.arange(beams), 1) + np.arange(batch)[:, None] * beams).astype(np.int32)
        pt = torch.from_numpy(parent).cuda()
        states = [raw(torch, gen, s, getattr(torch, d)) for d, s, _ in REORDER]
        dims = [dim for _, _, dim in REORDER]
        say(f"[decoding] reorder {batch}x{beams} trial {trial}")
        dev = [s.cuda() for s in states]
        assert iso.beam_reorder(dev, pt, dim=dims) is dev
        for s, d, dim in zip(states, dev, dims):
            v = (lambda t: t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.numpy())
            assert np.array_equal(v(d.cpu()), decoding.beam_reorder(v(s), parent, dim)), (s.dtype, s.shape)
            one = s.cuda()
            iso.beam_reorder(one, pt, dim=dim)
            assert torch.equal(one, d)


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 13, 16, 17, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_reorder_views(torch, beams, shift):
    """Views with strides and odd bytes: what lies around them stays."""
    say(f"[decoding] reorder views {beams} shift {shift}")
    gen = torch.Generator().manual_seed(beams)
    batch = 3
    rows = batch * beams
    parent = torch.randint(0, beams, (batch, beams), generator=gen) + torch.arange(batch)[:, None] * beams
    pt = parent.to(torch.int32).cuda()
    store = torch.randint(0, 255, (2, rows, 3, 61), generator=gen, dtype=torch.uint8)
    dev = store.cuda()
    iso.beam_reorder(dev[:, :, :, shift:shift + 47], pt, dim=1)
    want = store.clone()
    want[:, :, :, shift:shift + 47] = store[:, parent.reshape(-1), :, shift:shift + 47]
    assert torch.equal(dev.cpu(), want)
    store = torch.randn(2, rows, 4, 9, 40, generator=gen)
    dev = store.cuda()
    iso.beam_reorder(dev[:, :, :, shift:shift + 5], pt, dim=1)
    want = store.clone()
    want[:, :, :, shift:shift + 5] = store[:, parent.reshape(-1), :, shift:shift + 5]
    assert torch.equal(dev.cpu(), want)


# ---- pages ----

def cache(rng, seqs, most, page, pages, shared=2, per=2):
    """Sequences that share their first pages in groups of `per`."""
    table, length = np.full((seqs, most), -1, np.int32), rng.integers(0, most * page // 2 + 1, seqs).astype(np.int32)
    ids = iter(rng.permutation(pages))
    for s in range(seqs):
        first = s - s % per
        length[s] = length[first] if rng.random() < 0.7 else min(int(length[s]), int(length[first]))
        for j in range(-(-int(length[s]) // page)):
            table[s, j] = table[first, j] if s != first and j < shared and table[first, j] >= 0 else next(ids)
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, length, refs


def pools_of(torch, gen, pages, page, heads_first, dtype="bfloat16"):
    dt = getattr(torch, dtype)
    shape = (3, pages, 2, page, 5) if heads_first else (3, pages, page, 2, 5)
    return [raw(torch, gen, shape, dt), raw(torch, gen, shape, dt)], 3 if heads_first else 2


def bits(t):
    import torch

    return t.contiguous().view(torch.uint8).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def run_fork(torch, table, length, refs, parent, page, grow, pools, token_dim):
    dev = [p.cuda() for p in pools]
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    g = grow if isinstance(grow, int) else i(grow)
    got = iso.pages_fork(i(table), i(length), i(refs), i(parent), page_size=page, grow=g, pools=dev, page_dim=1, token_dim=token_dim)
    each = np.full(len(parent), grow, np.int32) if isinstance(grow, int) else grow
    want = decoding.pages_fork(table, length, refs, parent, page, each, [p.float().numpy() for p in pools], 1, token_dim)
    for name, a, b in zip(("table", "length", "refs", "status"), got, want):
        assert np.array_equal(n(a), b), (name, n(a), b)
    for d, w in zip(dev, want[4]):
        assert np.array_equal(d.float().cpu().numpy(), w)
    return got, want


@pytest.mark.parametrize("page", [1, 2, 5, 16])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("seqs", [1, 3, 8, 40])
def test_fork(torch, page, heads_first, seqs):
    rng = np.random.default_rng(page * 100 + seqs)
    gen = torch.Generator().manual_seed(seqs)
    for trial, children in enumerate((0, 1, seqs, 2 * seqs + 1, 300)):
        most, per = 7, 1 + trial % 4
        pages = seqs * most + children * 3 + 5
        table, length, refs = cache(rng, seqs, most, page, pages, per=per)
        pools, token_dim = pools_of(torch, gen, pages, page, heads_first)
        parent = rng.integers(-1, seqs, children).astype(np.int32)
        grow = rng.integers(-1, page + 3, children).astype(np.int32)
        say(f"[decoding] fork page {page} seqs {seqs} children {children}")
        outside = rng.integers(0, pages, 3)  # pages held from outside the table
        refs[outside] += 1
        run_fork(torch, table, length, refs, parent, page, grow if trial % 2 else 1, pools, token_dim)


def test_fork_without_room(torch):
    """Too few pages, or too long children: nothing is done."""
    rng = np.random.default_rng(7)
    gen = torch.Generator().manual_seed(7)
    table, length, refs = cache(rng, 6, 5, 4, 60)
    refs[refs == 0] = 1
    pools, token_dim = pools_of(torch, gen, 60, 4, False)
    got, want = run_fork(torch, table, length, refs, np.array([0, 0, 1, -1], np.int32), 4, np.array([1, 4, 3, 9], np.int32), pools, token_dim)
    assert want[3][0] > 0 and n(got[3])[2:].tolist() == [0, 0, 0]
    table, length, refs = cache(rng, 6, 5, 4, 60)
    got, want = run_fork(torch, table, length, refs, np.array([0, 0, 1, -1], np.int32), 4, np.array([1, 2 ** 31 - 1, 30, 20], np.int32), pools,
                         token_dim)
    assert want[3][1] == 2
    # to the last page
    table, length, refs = np.array([[0, -1]], np.int32), np.array([3], np.int32), np.array([1, 0, 0], np.int32)
    pools, token_dim = pools_of(torch, gen, 3, 4, True)
    _, want = run_fork(torch, table, length, refs, np.array([0, 0], np.int32), 4, np.array([1, 2], np.int32), pools, token_dim)
    assert want[3].tolist() == [0, 0, 1, 2, 0]


def test_fork_of_broken_caches(torch):
    """Lengths, entries, counts and parents outside their ranges are held inside the arrays."""
    rng = np.random.default_rng(9)
    gen = torch.Generator().manual_seed(9)
    for trial in range(20):
        seqs, most, page, pages = 5, 4, 3, 40
        table = rng.integers(-3, pages + 3, (seqs, most)).astype(np.int32)
        table[trial % seqs, 1] = np.iinfo(np.int32).max
        length = rng.integers(-2, most * page + 5, seqs).astype(np.int32)
        length[0] = np.iinfo(np.int32).min if trial % 2 else np.iinfo(np.int32).max
        refs = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages).astype(np.int32) + 1
        refs[rng.integers(0, pages, 8)] = -3
        held = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages)
        refs[held > 0] = held[held > 0] + 1  # what the table holds is counted; other counts may be anything
        parent = rng.integers(-2, seqs + 2, 6).astype(np.int32)
        parent[0] = np.iinfo(np.int32).min
        pools, token_dim = pools_of(torch, gen, pages, page, False)
        say(f"[decoding] fork broken {trial}")
        run_fork(torch, table, length, refs, parent, page, rng.integers(-2, 2, 6).astype(np.int32), pools, token_dim)


@pytest.mark.parametrize("seqs,children,most,pages", [(5, 40, 6, 12288), (5, 40, 6, 12289), (1024, 1024, 3, 5000), (1025, 300, 3, 5000),
                                                       (20, 1025, 4, 6000), (30, 50, 2200, 9000), (700, 2500, 5, 40000), (3, 7, 9, 300000),
                                                       (64, 64, 1024, 12288), (3000, 3000, 4, 20000)])
def test_fork_of_many(torch, seqs, children, most, pages):
    """Many pages, sequences, children and long tables."""
    say(f"[decoding] fork {seqs} to {children}, {most} pages each of {pages}")
    rng = np.random.default_rng(seqs + pages)
    gen = torch.Generator().manual_seed(pages)
    page = 2
    table, length = np.full((seqs, most), -1, np.int32), np.zeros(seqs, np.int32)
    ids, left = rng.permutation(pages).astype(np.int32), pages // 2
    at = 0
    for s in range(seqs):
        take = int(rng.integers(0, min(most, max(1, left // max(1, seqs - s)) * 2) + 1))
        take = min(take, left)
        table[s, :take] = ids[at:at + take]
        if s % 3 == 1 and take > 1 and table[s - 1, 0] >= 0:
            table[s, 0] = table[s - 1, 0]  # a shared first page
        at, left = at + take, left - take
        length[s] = max(0, take * page - int(rng.integers(0, 2))) if take else 0
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    pools = [raw(torch, gen, (1, pages, page, 3), torch.bfloat16), raw(torch, gen, (2, pages, page, 1), torch.float32)]
    parent = rng.integers(-1, seqs, children).astype(np.int32)
    run_fork(torch, table, length, refs, parent, page, rng.integers(0, 2, children).astype(np.int32), pools, 2)
    same = np.arange(children, dtype=np.int32)
    run_fork(torch, table, length, refs, same, page, 1, pools, 2)
    run_fork(torch, table, length, refs, parent, page, most * page, pools, 2)  # too long


def run_compact(torch, table, refs, pools):
    dev = [p.cuda() for p in pools]
    got = iso.pages_compact(torch.from_numpy(table).cuda(), torch.from_numpy(refs).cuda(), pools=dev, page_dim=1)
    want = decoding.pages_compact(table, refs, [p.float().numpy() for p in pools], 1)
    for name, a, b in zip(("table", "refs", "moved", "status"), got, want):
        assert np.array_equal(n(a), b), name
    for d, w in zip(dev, want[4]):
        assert np.array_equal(d.float().cpu().numpy(), w)


@pytest.mark.parametrize("pages", [0, 1, 2, 63, 257, 2048, 2049, 5000, 70001])
def test_compact(torch, pages):
    rng = np.random.default_rng(pages)
    gen = torch.Generator().manual_seed(pages)
    for live in (0.0, 0.03, 0.5, 0.97, 1.0):
        say(f"[decoding] compact {pages} live {live}")
        refs = np.where(rng.random(pages) < live, rng.integers(1, 4, pages), rng.integers(-1, 1, pages)).astype(np.int32)
        table = rng.integers(-2, pages + 2, (4, 7)).astype(np.int32)
        run_compact(torch, table, refs, pools_of(torch, gen, pages, 3, False)[0])
    # all live ones at the end, and at the beginning
    half = np.zeros(pages, np.int32)
    half[pages // 2:] = 1
    run_compact(torch, np.arange(pages, dtype=np.int32), half, pools_of(torch, gen, pages, 2, True)[0])
    run_compact(torch, np.arange(pages, dtype=np.int32), 1 - half, [])


def test_a_beam_search(torch):
    """The steps together: a beam search over a bigram model whose states are a token history
    (reordered in place) and a paged cache of the tokens (forked), compacted on the way, against
    the same search by the plain forms."""
    gen = torch.Generator().manual_seed(11)
    batch, beams, vocab, page, most, steps, end = 3, 4, 61, 4, 8, 14, 0
    rows, pages = batch * beams, 110
    model = torch.randn(vocab, vocab, generator=gen) * 2
    dev = model.cuda()
    token = torch.randint(1, vocab, (batch, 1), generator=gen, dtype=torch.int32).expand(batch, beams).reshape(-1).contiguous()
    # every item's prompt of one token, forked to its beams
    table = torch.full((batch, most), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(batch, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    pool = torch.zeros(2, pages, page, 1, dtype=torch.int32, device="cuda")

    def write(table, length, values, live):
        table, at = table[live].long(), length[live].long() - 1
        pool[:, table.gather(1, (at // page)[:, None])[:, 0], at % page, 0] = values[live]

    new = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    table, length, refs, status = iso.pages_fork(table, length, refs, new, page_size=page, grow=1, pools=pool, page_dim=1, token_dim=2)
    write(table, length, token.view(batch, beams)[:, 0].cuda(), new < 0)
    to_beams = torch.arange(batch, dtype=torch.int32).repeat_interleave(beams).cuda()
    table, length, refs, status = iso.pages_fork(table, length, refs, to_beams, page_size=page, grow=0, pools=pool, page_dim=1, token_dim=2)
    assert n(status).tolist() == [0, 0, 0, 0, pages - batch]
    score = torch.full((batch, beams), -float("inf"))
    score[:, 0] = 0
    ended = torch.zeros(batch, beams, dtype=torch.bool)
    history = token[:, None].cuda().repeat(1, steps + 1)
    gs, ge, gt = score.cuda(), ended.cuda(), token.cuda()
    hs, he, ht, hh = score.clone(), ended.clone(), token.clone(), history.cpu().clone()
    for step in range(steps):
        say(f"[decoding] search step {step}")
        out, logp, parent, tok = iso.beam_select(dev[gt.long()], gs, ended=ge, end_token=end)
        iso.beam_reorder([history, ge.view(-1)], parent)
        at = parent.view(-1)
        grow = (~ge.view(-1)).to(torch.int32)
        table, length, refs, status = iso.pages_fork(table, length, refs, at, page_size=page, grow=grow, pools=pool, page_dim=1, token_dim=2)
        assert n(status)[:2].tolist() == [0, 0]
        history[:, step + 1] = tok.view(-1)
        write(table, length, tok.view(-1), ~ge.view(-1))  # an ended beam has no new token
        gs, gt = out, tok.view(-1)
        ge |= (tok == end)
        if step % 5 == 4:
            table, refs, moved, status = iso.pages_compact(table, refs, pools=pool, page_dim=1)
            assert int((refs > 0).sum()) == int(status[0]) and bool((refs[:int(status[0])] > 0).all())
        # the plain forms
        want = decoding.beam_select(model[ht.long()].double().numpy(), hs.numpy(), beams, None, he.numpy(), end)
        par = np.array([[c["parent"] for c in w[:beams]] for w in want])
        assert np.array_equal(n(parent), par) and np.array_equal(n(tok), np.array([[c["token"] for c in w[:beams]] for w in want]))
        hh = hh[par.reshape(-1)]
        he = he.view(-1)[torch.from_numpy(par.reshape(-1))].view(batch, beams)
        ht = tok.view(-1).cpu()
        hh[:, step + 1] = ht
        hs = out.cpu()
        he |= tok.cpu() == end
        assert torch.equal(history.cpu(), hh) and torch.equal(ge.cpu(), he)
        # the cache's tokens are the history up to the end
        tb, ln, pl = n(table), n(length), n(pool)
        for r in range(rows):
            told = [int(pl[1, tb[r, t // page], t % page, 0]) for t in range(int(ln[r]))]
            assert told == hh[r, :len(told)].tolist()
            assert len(told) == step + 2 or hh[r, len(told) - 1] == end
        assert np.array_equal(np.bincount(tb[tb >= 0], minlength=pages), n(refs))
