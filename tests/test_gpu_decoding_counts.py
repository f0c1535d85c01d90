"""Caches whose counts are below what their tables hold: a page that children go on
to write is theirs, every other count ends at 0, and the result is the plain
form's, whichever kernels a step's size takes."""
from __future__ import annotations

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import decoding
from tests.test_gpu_decoding import pools_of, run_fork


def short_cache(rng, seqs, most, page, pages, children):
    """Sequences that hold any of a few pages, also the ones they end in, counted too low, and children of theirs."""
    few = rng.permutation(pages)[:3 * seqs]
    table = rng.choice(few, (seqs, most)).astype(np.int32)
    length = rng.integers(0, most * page, seqs).astype(np.int32)
    held = np.arange(most)[None, :] < -(-length[:, None] // page)
    refs = np.bincount(table[held], minlength=pages).astype(np.int32)
    refs -= rng.integers(0, 4, pages).astype(np.int32) * (rng.random(pages) < 0.6)
    refs[few] -= (rng.random(len(few)) < 0.2) * refs[few]
    parent = rng.integers(-1, seqs, children).astype(np.int32)
    grow = rng.integers(0, 2, children).astype(np.int32)
    return table, length, refs, parent, grow


def test_the_plain_form_keeps_what_is_written():
    """No page that a child goes on to write is given out or copied onto, and no count is below 0."""
    rng = np.random.default_rng(1)
    shown = 0
    for trial in range(200):
        page, pages = 3, 60
        table, length, refs, parent, grow = short_cache(rng, 6, 3, page, pages, 9)
        pool = np.arange(pages * page).reshape(pages, page).copy()
        out, ln, new, status, (held,) = decoding.pages_fork(table, length, refs, parent, page, grow, [pool])
        assert status[:2].tolist() == [0, 0] and new.min() >= 0
        written, sources, given = set(), set(), set()
        for i, p in enumerate(parent):
            before = int(length[p]) if p >= 0 else 0
            if grow[i] and before % page:
                source, mine = int(table[p, before // page]), int(out[i, before // page])
                assert mine not in written, (i, mine)  # every child writes a page of its own
                written.add(mine)
                sources.add(source)
                assert held[mine, :before % page].tolist() == pool[source, :before % page].tolist()
                shown += int(refs[source]) <= 0
                if mine != source:
                    given.add(mine)
            elif grow[i]:
                given.add(int(out[i, before // page]))
        assert not given & sources
        assert all(new[q] >= 1 for q in written | sources)
        assert np.array_equal(held[sorted(sources)], pool[sorted(sources)])
    assert shown > 100


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,children,most,pages", [(1, 2, 2, 9), (12, 30, 4, 200), (12, 30, 4, 13001), (300, 900, 3, 20000),
                                                       (12, 0, 4, 13001), (40, 1500, 3, 6000), (700, 2500, 5, 40000)])
def test_fork_of_counts_that_are_too_low(torch, seqs, children, most, pages):
    rng = np.random.default_rng(seqs + children + pages)
    gen = torch.Generator().manual_seed(pages)
    page = 3
    for trial in range(6):
        table, length, refs, parent, grow = short_cache(rng, seqs, most, page, pages, children)
        pools, token_dim = pools_of(torch, gen, pages, page, trial % 2 == 1)
        print(f"[decoding] counts too low {seqs} to {children} of {pages}, {trial}", flush=True)
        if trial == 4:  # nobody begins or ends: only what is written is shared
            table, length, refs = table[:min(seqs, children)], length[:min(seqs, children)], refs
            parent = np.arange(len(length), dtype=np.int32)
            parent = np.concatenate([parent, np.full(children - len(parent), -1, np.int32)])
        if trial == 5:  # too few pages
            refs[refs <= 0] = np.where(rng.random(int((refs <= 0).sum())) < 0.9, 1, 0)
            grow[:] = page
        got, want = run_fork(torch, table, length, refs, parent, page, grow, pools, token_dim)
        again, _ = run_fork(torch, table, length, refs, parent, page, grow, pools, token_dim)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("seqs,children,pages", [(12, 30, 200), (12, 30, 13001), (60, 900, 20000), (40, 1500, 6000)])
def test_counts_that_pass_32_bits(torch, seqs, children, pages):
    """Counts at the ends of their type, of pages with many holders more and fewer: what is given out are pages, each once."""
    rng = np.random.default_rng(seqs + pages)
    top = 2 ** 31 - 1
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for trial in range(6):
        print(f"[decoding] counts past 32 bits {seqs} to {children} of {pages}, {trial}", flush=True)
        table, length, refs, parent, grow = short_cache(rng, seqs, 4, 3, pages, children)
        table[:, :2] = rng.choice(table[:4, 0], (seqs, 2))  # a few pages that all hold
        held = np.unique(table)
        refs[held] = rng.choice([top, top - 1, top - 20, 0, 1, 5], len(held))
        pool = torch.zeros(pages, 3, 2, dtype=torch.uint8, device="cuda")
        out, ln, new, status = iso.pages_fork(i(table), i(length), i(refs), i(parent), page_size=3, grow=i(grow), pools=pool)
        out, new, status = out.cpu().numpy(), new.cpu().numpy(), status.tolist()
        assert out.min() >= -1 and out.max() < pages
        if status[:2] == [0, 0]:
            given = []
            for k, p in enumerate(parent):
                before = int(length[p]) if p >= 0 else 0
                given += out[k, -(-before // 3):-(-(before + int(grow[k])) // 3)].tolist()
            assert len(set(given)) == len(given) and status[3] == len(given) + status[2]
            assert status[3] + status[4] <= pages
