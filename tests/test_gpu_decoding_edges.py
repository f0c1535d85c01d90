"""The decoding steps where values do not show it: streams, graphs, memory beside
the outputs, arrays that begin anywhere, offsets past 32 bits, sizes at the
borders of their kernels, bounds that too many values reach."""
from __future__ import annotations

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import decoding
from tests.test_gpu_decoding import check_select, dtype_of, n, place, raw, run_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


def say(*a):
    print(*a, flush=True)


# ---- selection ----

@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("take", [32, 33])
def test_select_at_the_borders_of_its_pieces(torch, name, take):
    """Rows of 4, 8, 16 and 32 KB and a few bytes less and more, few and many of them."""
    dtype = dtype_of(torch, name)
    size = 4 if name == "f32" else 2
    gen = torch.Generator().manual_seed(take)
    for batch, beams in ((1, 2), (130, 3)):
        for row in (4096, 8192, 16384, 32768):
            for more in (-size, 0, size, 9 * size):
                vocab = (row + more) // size
                say(f"[decoding] pieces {name} {batch}x{beams}x{vocab} take {take}")
                x = (torch.randn(batch * beams, vocab, generator=gen) * 2).to(dtype)
                score = -torch.rand(batch, beams, generator=gen)
                got = iso.beam_select(place(torch, x, dtype, 1, 1), score.cuda(), take=take)
                for b in {0, batch // 2, batch - 1}:
                    pick = [t[b:b + 1] - (b * beams if i == 2 else 0) for i, t in enumerate(got)]
                    check_select(pick, x[b * beams:(b + 1) * beams].double().numpy(), score[b:b + 1], take)


@pytest.mark.parametrize("take", [18, 33])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_select_of_many_streamed_rows(torch, name, take):
    """Logits past half of the last-level cache."""
    dtype = dtype_of(torch, name)
    batch, beams, vocab = 70, 9, 60001 if name == "f32" else 120001
    say(f"[decoding] streamed {name}")
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randn(batch * beams, vocab, generator=gen, device="cuda") * 2).to(dtype)
    score = -torch.rand(batch, beams, generator=gen, device="cuda")
    got = iso.beam_select(x, score, take=take)
    for b in (0, 1, 33, 69):
        pick = [t[b:b + 1] - (b * beams if i == 2 else 0) for i, t in enumerate(got)]
        check_select(pick, x[b * beams:(b + 1) * beams].double().cpu().numpy(), score[b:b + 1].cpu(), take)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [900, 3000, 20001])
@pytest.mark.parametrize("take", [1, 5, 128])
def test_select_of_few_different_logits(torch, name, vocab, take):
    """Values that many tokens share, at the bound and elsewhere, and beams that are alike."""
    dtype = dtype_of(torch, name)
    rng = np.random.default_rng(vocab + take)
    say(f"[decoding] few logits {name} {vocab} take {take}")
    for levels in (1, 2, 5, 60):
        x = torch.from_numpy(rng.integers(0, levels, (6, vocab)).astype(np.float32) / 4.0).to(dtype)
        x[3] = x[1]
        score = torch.from_numpy(rng.integers(-2, 1, (2, 3)).astype(np.float32))
        score[1, 0] = score[0, 1]
        got = iso.beam_select(place(torch, x, dtype, 0, 1), score.cuda(), take=take)
        check_select(got, x.double().numpy(), score, take)
        # one beam's: exactly in the order of the definition
        one = iso.beam_select(place(torch, x[:1], dtype, 2, 3), score[:1, :1].cuda(), take=take)
        want = np.argsort(-x[0].double().numpy(), kind="stable")[:take]
        assert n(one[3])[0, :len(want)].tolist() == want.tolist()


@pytest.mark.parametrize("beams,take,live", [(128, 128, 1), (64, 64, 2), (128, 128, 128), (32, 64, 1), (7, 128, 1)])
def test_select_of_few_live_beams(torch, beams, take, live):
    """A first step of many beams: the keys of few lists."""
    vocab = 70001
    say(f"[decoding] {live} of {beams} beams live, take {take}")
    gen = torch.Generator().manual_seed(beams)
    x = torch.randn(live, vocab, generator=gen).repeat(beams // live, 1)
    x = torch.cat([x, x[:beams - len(x)]]).bfloat16()
    score = torch.full((1, beams), -float("inf"))
    score[0, beams - live:] = -torch.rand(live, generator=gen)
    got = iso.beam_select(place(torch, x, torch.bfloat16, 1, 0), score.cuda(), take=take)
    check_select(got, x.double().numpy(), score, take)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("batch,beams,vocab,take", [(2, 32, 50003, 64), (1, 128, 16390, 128), (3, 5, 200001, 100), (1, 1, 400000, 128)])
def test_select_of_many_keys(torch, name, batch, beams, vocab, take):
    """Items with more keys than one workgroup ranks: each row's are merged first."""
    say(f"[decoding] many keys {name} {batch}x{beams}x{vocab} take {take}")
    dtype, gen = dtype_of(torch, name), torch.Generator().manual_seed(vocab)
    x = (torch.randn(batch * beams, vocab, generator=gen) * 2).to(dtype)
    x[torch.rand(batch * beams, vocab, generator=gen) < 0.3] = -float("inf")
    score = -20 * torch.rand(batch, beams, generator=gen)
    ended = torch.rand(batch, beams, generator=gen) < 0.2
    weight = 0.3 + torch.rand(batch, beams, generator=gen)
    got = iso.beam_select(place(torch, x, dtype, 1, 1), score.cuda(), take=take, weight=weight.cuda(), ended=ended.cuda(), end_token=7)
    check_select(got, x.double().numpy(), score, take, weight, ended, 7)
    # every value the same: the lowest tokens of the best beam
    x.zero_()
    score[:, 0] = 1.0
    out = iso.beam_select(place(torch, x, dtype, 0, 1), score.cuda(), take=take)
    assert n(out[3])[:, :take].tolist() == [list(range(take))] * batch
    assert n(out[2]).tolist() == [[b * beams] * take for b in range(batch)]


def test_select_of_extreme_logits(torch):
    """The largest finite values, subnormals, and temperatures at their ends."""
    f32 = torch.finfo(torch.float32)
    for temperature in (1e-28, 1e-3, 1.0, 1e28):
        x = torch.zeros(4, 300)
        x[0, 5], x[0, 6], x[0, 7] = f32.max, f32.max, f32.min
        x[1] = -f32.max
        x[1, 9] = -f32.max / 2
        x[2, 3], x[2, 4] = 1e-45, 2e-45
        x[3] = torch.linspace(-1e4, 1e4, 300)
        score = torch.tensor([[-1.0, -1.0, -1.0, -1.0]])
        say(f"[decoding] extremes at {temperature}")
        got = iso.beam_select(x.cuda(), score.cuda(), take=8, temperature=temperature)
        out, logp, parent, token = (n(t)[0] for t in got)
        assert not np.isnan(out).any() and not np.isnan(logp).any()
        want = decoding.beam_select(x.double().numpy(), score.numpy(), 8, temperature=temperature)[0][:8]
        for i, c in enumerate(want):
            assert abs(float(out[i]) - c["score"]) <= decoding.U * (abs(c["score"]) + c["err"]), (i, c, out[i])


def test_select_refusals(torch):
    x, s = torch.zeros(6, 8, device="cuda"), torch.zeros(2, 3, device="cuda")
    bad = [dict(score=s[0]), dict(score=torch.zeros(2, 2, device="cuda")), dict(take=0), dict(take=129), dict(weight=s[:1]),
           dict(ended=torch.zeros(2, 2, dtype=torch.bool, device="cuda")), dict(end_token=1 << 31), dict(score=s.t().contiguous().t())]
    for kw in bad:
        a = dict(score=s)
        a.update(kw)
        with pytest.raises(ValueError):
            iso.beam_select(x, a.pop("score"), **a)
    for kw in (dict(weight=s.double()), dict(ended=s), dict(weight=s.cpu())):
        with pytest.raises(TypeError):
            iso.beam_select(x, s, **kw)
    for kw in (dict(temperature=0.0), dict(temperature=1e-29)):
        with pytest.raises(iso.IsoError):
            iso.beam_select(x, s, **kw)
    with pytest.raises(ValueError):
        iso.beam_select(x.t(), s)


def test_states_and_pages_refusals(torch):
    i = lambda *a: torch.zeros(*a, dtype=torch.int32, device="cuda")  # noqa: E731
    s = torch.zeros(6, 8, device="cuda")
    for args, kw in (((s, i(6)), {}), ((s, i(2, 4)), {}), ((s, i(2, 3)), dict(dim=1)), (([s, s], i(2, 3)), dict(dim=(0,))), ((s, i(2, 3)), dict(dim=2))):
        with pytest.raises(ValueError):
            iso.beam_reorder(*args, **kw)
    with pytest.raises(TypeError):
        iso.beam_reorder(s.cpu(), i(2, 3))
    with pytest.raises(TypeError):
        iso.beam_reorder(s, i(2, 3).long())
    for states in ([s, s], [s, s[:, 2:4]], [s.expand(6, 8), torch.as_strided(s, (6, 4), (0, 1))]):
        with pytest.raises(iso.IsoError):  # two arrays in one place; rows in one place
            iso.beam_reorder(states, i(2, 3))
    pool = torch.zeros(5, 4, 8, device="cuda")
    fork = lambda **kw: iso.pages_fork(i(2, 3), i(2), i(5), i(2), **{"page_size": 4, "pools": pool, **kw})  # noqa: E731
    fork()
    for kw in (dict(page_size=8), dict(pools=pool[:4]), dict(page_dim=1, token_dim=2), dict(token_dim=0), dict(grow=1 << 31), dict(grow=i(3)),
               dict(pools=pool.transpose(1, 2), token_dim=2)):
        with pytest.raises(ValueError):
            fork(**kw)
    with pytest.raises(TypeError):
        fork(grow=i(2).long())
    with pytest.raises(iso.IsoError):
        fork(pools=[pool, pool])
    with pytest.raises(ValueError):
        iso.pages_compact(i(2, 3), i(5), pools=pool[:3])


def test_nothing_to_do(torch):
    """Empty batches, caches and arrays."""
    i = lambda *a: torch.zeros(*a, dtype=torch.int32, device="cuda")  # noqa: E731
    out = iso.beam_select(torch.zeros(0, 9, device="cuda"), torch.zeros(0, 3, device="cuda"), take=4)
    assert all(t.shape == (0, 4) for t in out)
    e = torch.zeros(6, 0, 3, device="cuda")
    assert iso.beam_reorder(e, i(2, 3)) is e
    assert iso.beam_reorder([], i(2, 3)) == []
    table, length, refs, status = iso.pages_fork(i(0, 3), i(0), i(5), i(0), page_size=4)
    assert table.shape == (0, 3) and n(refs).tolist() == [0] * 5 and n(status).tolist() == [0, 0, 0, 0, 5]
    table, length, refs, status = iso.pages_fork(i(2, 0), i(2), i(0), i(3) - 1, page_size=4, grow=0)
    assert table.shape == (3, 0) and n(length).tolist() == [0, 0, 0] and n(status).tolist() == [0, 0, 0, 0, 0]
    table, length, refs, status = iso.pages_fork(i(2, 0), i(2), i(0), i(3), page_size=4)
    assert n(status).tolist() == [0, 3, 0, 0, 0]
    table, refs, moved, status = iso.pages_compact(i(0), i(0))
    assert n(status).tolist() == [0, 0]


# ---- streams, graphs, memory ----

def step_inputs(torch, seed):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    batch, beams, vocab, pages, page = 3, 4, 5003, 60, 4
    rows = batch * beams
    length = rng.integers(1, 12, rows).astype(np.int32)
    table, at = np.full((rows, 5), -1, np.int32), 0
    for r in range(rows):
        for j in range(-(-int(length[r]) // page)):
            table[r, j] = at
            at += 1
    refs = (np.arange(pages) < at).astype(np.int32)
    s = {"x": (torch.randn(rows, vocab, generator=gen) * 2).bfloat16(), "score": -torch.rand(batch, beams, generator=gen),
         "state": torch.randn(2, rows, 3, 77, generator=gen), "table": torch.from_numpy(table), "length": torch.from_numpy(length),
         "refs": torch.from_numpy(refs), "pool": torch.randn(2, pages, page, 24, generator=gen)}
    return {k: v.cuda() for k, v in s.items()}


def step(s, **kw):
    out, logp, parent, token = iso.beam_select(s["x"], s["score"], take=4, **kw)
    iso.beam_reorder(s["state"], parent, dim=1, **kw)
    t, l, r, st = iso.pages_fork(s["table"], s["length"], s["refs"], parent.view(-1), page_size=4, pools=s["pool"], page_dim=1, token_dim=2, **kw)
    return [out, logp, parent, token, s["state"], t, l, r, st, *iso.pages_compact(t, r, pools=s["pool"], page_dim=1, **kw), s["pool"]]


def busy(torch, block):
    """Some tens of milliseconds of copies on the current stream."""
    for _ in range(200):
        block[1].copy_(block[0])


def test_steps_run_on_the_stream_they_are_given(torch):
    """New inputs are copied in on the other stream, behind other work there: a call
    that ran anywhere else would take the old ones."""
    s, new = step_inputs(torch, 1), step_inputs(torch, 2)
    block = torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    before = [t.clone() for t in step({k: v.clone() for k, v in s.items()})]
    want = [t.clone() for t in step({k: v.clone() for k, v in new.items()})]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy(torch, block)
        for k in s:
            s[k].copy_(new[k])
        parent_view = s  # views are taken inside, on no stream of their own
    # the parent's view is no kernel, so the whole step can be given the stream
    got = step(parent_view, stream=side)
    side.synchronize()
    shows = 0
    for k, (a, b, c) in enumerate(zip(got, want, before)):
        assert torch.equal(a, b), k
        shows += not torch.equal(b, c)
    assert shows >= 8  # the old inputs would have shown


def test_inputs_dropped_after_a_step_on_another_stream(torch):
    """The calls still wait behind other work when their inputs are dropped and their sizes taken again and overwritten."""
    keep = step_inputs(torch, 3)
    block = torch.empty(2, 1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    want = [t.clone() for t in step({k: v.clone() for k, v in keep.items()})]
    for v in keep.values():
        torch.empty_like(v).fill_(1)
    torch.cuda.synchronize()
    mine = {k: v.clone() for k, v in keep.items()}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        busy(torch, block)
    got = step(mine, stream=side)
    mine.clear()
    again = [torch.empty_like(v) for v in keep.values()]
    assert not side.query()  # the calls have not run yet
    for v in again:
        v.fill_(1)
    side.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), k


def test_captured_into_a_graph(torch):
    """A step in a graph, replayed over other inputs, eager steps and waits between."""
    s = step_inputs(torch, 4)
    step({k: v.clone() for k, v in s.items()})
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for seed in (5, 6, 7, 8):
        new = step_inputs(torch, seed)
        want = step({k: v.clone() for k, v in new.items()})
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (seed, k)
        step({k: v.clone() for k, v in new.items()})


def test_two_streams_at_once(torch):
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    inputs = [step_inputs(torch, 9), step_inputs(torch, 10)]
    want = [[t.clone() for t in step({k: v.clone() for k, v in s.items()})] for s in inputs]
    copies = [[{k: v.clone() for k, v in s.items()} for _ in range(10)] for s in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(10):
        for k in (0, 1):
            got[k].append(step(copies[k][i], stream=sides[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for g in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[k]))


class Arena:
    """Device memory of one pattern, of which pieces are handed out with guards around them."""

    GUARD = 512

    def __init__(self, torch, size):
        self.mem = torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda")
        self.at, self.used = 0, []

    def take(self, nbytes):
        begin = (self.at + self.GUARD + 255) // 256 * 256
        self.at = begin + nbytes
        assert self.at + self.GUARD <= self.mem.numel()
        self.used.append((begin, self.at))
        return self.mem.data_ptr() + begin

    def untouched(self):
        keep = self.mem != 0x5a
        for a, b in self.used:
            keep[a:b] = False
        return not bool(keep.any())


@pytest.mark.parametrize("batch,beams,vocab,take", [(1, 1, 1, 1), (2, 3, 700, 40), (3, 2, 9001, 5), (1, 2, 50021, 128), (130, 3, 16390, 7)])
def test_nothing_beside_the_selection_is_written(torch, batch, beams, vocab, take):
    code = iso.ISO_DT_BF16
    say(f"[decoding] guards select {batch}x{beams}x{vocab}")
    size = iso.iso_beam_select_workspace_bytes(batch, beams, vocab, take, code)
    x = torch.randn(batch * beams, vocab, device="cuda").bfloat16()
    x[0] = 0
    score = torch.zeros(batch, beams, device="cuda")
    a = Arena(torch, size + 16 * batch * take + 6 * (Arena.GUARD + 512))
    out = [a.take(4 * batch * take) for _ in range(4)]
    st = iso.iso_beam_select(x.data_ptr(), code, batch, beams, vocab, vocab, score.data_ptr(), None, None, 0, 1.0, take, *out,
                             a.take(size), size, torch.cuda.current_stream().cuda_stream)
    assert st == iso.ISO_OK
    torch.cuda.synchronize()
    assert a.untouched()


@pytest.mark.parametrize("seqs,children,most,pages", [(1, 1, 1, 1), (5, 9, 4, 50), (5, 9, 4, 13001), (40, 1100, 3, 5000), (2, 0, 3, 7)])
def test_nothing_beside_the_cache_is_written(torch, seqs, children, most, pages):
    """Also of caches whose entries, lengths, counts and parents are anything."""
    rng = np.random.default_rng(pages)
    say(f"[decoding] guards pages {seqs} to {children}")
    top = 2 ** 31 - 1
    for trial in range(8):
        wild = trial >= 2
        table = rng.integers(-5 if wild else 0, pages + (5 if wild else 0), (seqs, most)).astype(np.int32)
        length = rng.integers(-3 if wild else 0, most * 3 + (9 if wild else 1), seqs).astype(np.int32)
        refs = rng.integers(-2 if wild else 0, 3, pages).astype(np.int32)
        parent = rng.integers(-3, seqs + 3, children).astype(np.int32)
        grow = rng.integers(-3, 9, children).astype(np.int32)
        if trial >= 5:
            for v in (table, length, refs, parent, grow):
                v.reshape(-1)[rng.random(v.size) < 0.3] = top if trial % 2 else -top - 1
        t = [torch.from_numpy(v).cuda() for v in (table, length, refs, parent, grow)]
        stream = torch.cuda.current_stream().cuda_stream
        s1, s2 = iso.iso_pages_fork_workspace_bytes(seqs, children, pages), iso.iso_pages_compact_workspace_bytes(pages)
        token = 5
        a = Arena(torch, s1 + s2 + 4 * (children * most + children + 3 * pages + seqs * most) + 2 * pages * 3 * token + 20 * (Arena.GUARD + 512))
        pools = (iso.Blocks * 2)(iso.Blocks(a.take(pages * 3 * token), 1, 0, 3 * token, 1, 0, 3 * token),
                                 iso.Blocks(a.take(pages * 3 * token), 1, 0, 3 * token, 1, 0, 3 * token))
        st = iso.iso_pages_fork(t[0].data_ptr(), t[1].data_ptr(), seqs, most, t[2].data_ptr(), pages, 3, t[3].data_ptr(), t[4].data_ptr(), 0,
                                children, pools, 2, a.take(4 * children * most), a.take(4 * children), a.take(4 * pages), a.take(20),
                                a.take(s1), s1, stream)
        assert st == iso.ISO_OK
        st = iso.iso_pages_compact(t[0].data_ptr(), seqs * most, t[2].data_ptr(), pages, pools, 2, a.take(4 * seqs * most), a.take(4 * pages),
                                   a.take(4 * pages), a.take(8), a.take(s2), s2, stream)
        assert st == iso.ISO_OK
        torch.cuda.synchronize()
        assert a.untouched(), trial


def test_arrays_that_begin_anywhere(torch):
    """int32 and f32 arrays at every element: the values do not depend on where they lie.  (A row of
    logits is summed in vectors from its first aligned element on; it stays where it is.)"""
    s = step_inputs(torch, 12)
    want = [t.clone() for t in step({k: v.clone() for k, v in s.items()})]
    for shift in (1, 2, 3):
        moved = {}
        for k, v in s.items():
            if k == "x":
                moved[k] = v
                continue
            store = torch.zeros(v.numel() + shift + 4, dtype=v.dtype, device="cuda")
            view = store[shift:shift + v.numel()].view(v.shape)
            view.copy_(v)
            moved[k] = view
        for k, (a, b) in enumerate(zip(step(moved), want)):
            assert torch.equal(a, b), (shift, k)


def test_offsets_past_32_bits(torch):
    """Rows, states and pages whose places are more than 4 GB apart."""
    say("[decoding] far rows")
    gen = torch.Generator().manual_seed(1)
    far = 2_400_000_000  # bytes between rows
    store = torch.zeros(2 * far + (1 << 20), dtype=torch.uint8, device="cuda")
    x = (torch.randn(3, 5001, generator=gen) * 2).bfloat16()
    logits = torch.as_strided(store.view(torch.bfloat16), (3, 5001), (far // 2, 1))
    logits.copy_(x)
    score = torch.zeros(1, 3)
    check_select(iso.beam_select(logits, score.cuda(), take=6), x.double().numpy(), score, 6)
    say("[decoding] far states")
    state = torch.as_strided(store, (3, 1000), (far, 1))
    rows = torch.randint(0, 255, (3, 1000), generator=gen, dtype=torch.uint8)
    state.copy_(rows)
    iso.beam_reorder(state, torch.tensor([[2, 0, 0]], dtype=torch.int32, device="cuda"))
    assert torch.equal(state.cpu(), rows[[2, 0, 0]])
    say("[decoding] far pages")
    page, token = 4, 1000
    pages = store.numel() // (page * token)
    pool = store[:pages * page * token].view(pages, page, token)
    last = pages - 1
    pool[last] = torch.randint(0, 255, (page, token), generator=gen, dtype=torch.uint8).cuda()
    keep = pool[last].clone()
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 3] = 0
    table = torch.full((1, 3), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = last
    length = torch.tensor([3], dtype=torch.int32, device="cuda")
    refs[last] = 1
    out, ln, rf, st = iso.pages_fork(table, length, refs, torch.zeros(2, dtype=torch.int32, device="cuda"), page_size=page, pools=pool)
    assert n(st).tolist() == [0, 0, 1, 1, 0] and n(out)[:, 0].tolist() == [last, pages - 3]
    assert torch.equal(pool[pages - 3, :3], keep[:3])
    refs.zero_()
    refs[last] = 1
    t2, r2, moved, st = iso.pages_compact(table, refs, pools=pool)
    assert n(st).tolist() == [1, 1] and n(t2)[0, 0] == 0 and torch.equal(pool[0], keep)


@pytest.mark.parametrize("inner", [1, 3, 7, 15, 16, 17, 31, 33, 100, 4097])
def test_blocks_of_every_width(torch, inner):
    """Forked and compacted pages, and reordered rows, of odd bytes: what lies between stays."""
    say(f"[decoding] blocks of {inner}")
    rng = np.random.default_rng(inner)
    gen = torch.Generator().manual_seed(inner)
    page, pages = 3, 30
    table = np.arange(12, dtype=np.int32).reshape(4, 3)
    length = np.array([9, 7, 2, 5], np.int32)
    held = [3, 3, 1, 2]
    refs = np.zeros(pages, np.int32)
    for s in range(4):
        refs[table[s, :held[s]]] += 1
    store = torch.randint(0, 255, (2, pages, 2, page, inner + 3), generator=gen, dtype=torch.uint8)
    pools = [store[..., :inner].contiguous().float().to(torch.float16), store[..., :inner].contiguous().float().to(torch.float32)]
    run_fork(torch, table, length, refs, np.array([0, 1, 1, 2, 3, 3, 3], np.int32), page, 1, pools, 3)
    wide = store.cuda()
    part = wide[:, :, :, :, :inner]
    keep = store.clone()
    live = torch.from_numpy((rng.random(pages) < 0.5).astype(np.int32))
    # runs with room between them
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    iso.pages_compact(one, live.cuda(), pools=part, page_dim=1)
    _, _, _, _, (want,) = decoding.pages_compact(np.zeros(1, np.int32), live.numpy(), [keep[..., :inner].numpy()], 1)
    got = wide.cpu()
    assert np.array_equal(got[..., :inner].numpy(), want) and torch.equal(got[..., inner:], keep[..., inner:])
    # one run that begins anywhere
    wide.copy_(keep)
    flat = lambda t: t.view(2, pages, -1)[:, :, 1:1 + inner]  # noqa: E731
    iso.pages_compact(one, live.cuda(), pools=flat(wide), page_dim=1)
    _, _, _, _, (want,) = decoding.pages_compact(np.zeros(1, np.int32), live.numpy(), [flat(keep).numpy()], 1)
    got = wide.cpu()
    assert np.array_equal(flat(got).numpy(), want)
    flat(got).copy_(flat(keep))
    assert torch.equal(got, keep)


def test_reorder_of_large_states(torch):
    """More than 128 MB, which is streamed, with a tail behind each block's last 16 bytes."""
    say("[decoding] large states")
    gen = torch.Generator(device="cuda").manual_seed(2)
    state = torch.randint(0, 1 << 20, (3, 6, 5, 400003), generator=gen, device="cuda", dtype=torch.int32)
    part = state[:, :, :, 1:400002]
    parent = torch.tensor([[1, 2, 0], [3, 3, 4]], dtype=torch.int32, device="cuda")
    want = state.clone()
    want[:, :, :, 1:400002] = state[:, parent.view(-1).long(), :, 1:400002]
    iso.beam_reorder(part, parent, dim=1)
    assert torch.equal(state, want)
