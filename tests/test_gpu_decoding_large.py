"""The decoding steps at sizes where a launch's workgroups come around for more
than one row, item, column or block of pages."""
from __future__ import annotations

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from tests.test_gpu_decoding import U, check_select, n, raw, run_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("vocab", [8, 1027])
def test_select_of_a_million_items(torch, vocab):
    """One beam each, a piece of a wave or two: every item's two best and their log-probabilities, off by half
    a step of f32 and by what decoding.row_logp counts, U (3 |z - zmax| + 5) at most with |z - zmax| below 16 here."""
    batch = (1 << 20) + 3
    say(f"[decoding] {batch} items of {vocab}")
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.rand(batch, vocab, generator=gen, device="cuda") * 16
    score = -torch.rand(batch, 1, generator=gen, device="cuda")
    out, logp, parent, token = iso.beam_select(x, score, take=2)
    for a in range(0, batch, 1 << 17):
        part = slice(a, min(batch, a + (1 << 17)))
        z = x[part].double()
        lse = torch.logsumexp(z, 1, keepdim=True)
        top = z.max(1)
        assert torch.equal(token[part, 0].long(), torch.where(z == top.values[:, None], torch.arange(vocab, device="cuda"), vocab).min(1).values)
        want = z.gather(1, token[part].long()) - lse
        assert bool((token[part, 0] != token[part, 1]).all())
        rest = z.scatter(1, token[part, :1].long(), -1.0).max(1).values
        assert torch.equal(z.gather(1, token[part, 1:].long())[:, 0], rest)
        assert bool(((logp[part] - want).abs() <= U * (want.abs() + 53)).all())
        both = score[part].double() + want
        assert bool(((out[part] - both).abs() <= U * (both.abs() + 53)).all())
    assert torch.equal(parent, torch.arange(batch, device="cuda", dtype=torch.int32)[:, None].expand(batch, 2))


def test_select_of_a_million_rows_of_many_keys(torch):
    """128 beams an item, two pieces a row: each row's lists are merged."""
    batch, beams, vocab, take = 8193, 128, 1030, 32
    say(f"[decoding] {batch} x {beams} rows of {vocab}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(batch * beams, vocab, generator=gen, device="cuda") * 2
    score = -8 * torch.rand(batch, beams, generator=gen, device="cuda")
    got = iso.beam_select(x, score, take=take)
    rng = np.random.default_rng(1)
    for b in [0, 1, 8190, 8191, 8192, *rng.integers(2, 8190, 12).tolist()]:
        pick = [t[b:b + 1] - (b * beams if i == 2 else 0) for i, t in enumerate(got)]
        check_select(pick, x[b * beams:(b + 1) * beams].double().cpu().numpy(), score[b:b + 1].cpu(), take)


@pytest.mark.parametrize("batch,beams,shape,inner", [(20011, 2, (7,), 5), (3, 128, (2, 140000, 24), 17), (1, 128, (3, 5600016), 5600013),
                                                     (9001, 3, (3, 40), 33)])
def test_reorder_of_many_items_and_columns(torch, batch, beams, shape, inner):
    rows = batch * beams
    say(f"[decoding] reorder {batch} x {beams} of {shape}")
    gen = torch.Generator(device="cuda").manual_seed(rows)
    outer = len(shape) == 3 or (batch == 9001)
    full = (shape[0], rows, *shape[1:]) if outer else (rows, *shape)
    state = torch.randint(-128, 127, full, generator=gen, device="cuda", dtype=torch.int8)
    parent = (torch.randint(0, beams, (batch, beams), generator=gen, device="cuda") + torch.arange(batch, device="cuda")[:, None] * beams).int()
    want = state.clone()
    want[..., :inner] = state[..., :inner].index_select(1 if outer else 0, parent.view(-1))
    iso.beam_reorder(state[..., :inner], parent, dim=1 if outer else 0)
    assert torch.equal(state, want)


@pytest.mark.parametrize("pages", [2200001, 4400001])
@pytest.mark.parametrize("seqs,children", [(7, 40), (300, 1100)])
def test_fork_over_millions_of_pages(torch, pages, seqs, children):
    """Blocks of pages past a launch's workgroups, and blocks of more pages."""
    say(f"[decoding] fork {seqs} to {children} of {pages}")
    rng, gen = np.random.default_rng(pages + seqs), torch.Generator().manual_seed(seqs)
    page, most = 2, 6
    ids = rng.permutation(pages)[:seqs * most].astype(np.int32).reshape(seqs, most)
    length = rng.integers(0, (most - 2) * page, seqs).astype(np.int32)
    table = np.where(np.arange(most)[None, :] < -(-length[:, None] // page), ids, -1).astype(np.int32)
    refs = (rng.random(pages) < 0.9999).astype(np.int32)  # the free pages are spread over all blocks
    refs[ids.reshape(-1)] = 0
    refs[table[table >= 0]] = 1
    free = np.flatnonzero(refs == 0)
    refs[rng.choice(free, max(0, len(free) - 2 * children - seqs), replace=False)] = 1
    pools = [raw(torch, gen, (1, pages, page, 1), torch.float16)]
    parent = rng.integers(-1, seqs, children).astype(np.int32)
    got, want = run_fork(torch, table, length, refs, parent, page, rng.integers(0, 2, children).astype(np.int32), pools, 2)
    assert want[3][:2].tolist() == [0, 0] and want[3][3] > children // 4
    run_fork(torch, table, length, refs, parent, page, 4 * page, pools, 2)  # too few pages or too long


@pytest.mark.parametrize("pages", [2200001, 4400001])
def test_compact_over_millions_of_pages(torch, pages):
    rng, gen = np.random.default_rng(pages), torch.Generator(device="cuda").manual_seed(1)
    for live in (0.02, 0.5, 0.999):
        say(f"[decoding] compact {pages}, live {live}")
        refs = np.where(rng.random(pages) < live, rng.integers(1, 4, pages), rng.integers(-1, 1, pages)).astype(np.int32)
        table = rng.integers(-2, pages + 2, (4, 7)).astype(np.int32)
        pool = torch.randint(0, 1 << 20, (pages, 3), generator=gen, device="cuda", dtype=torch.int32)
        keep = pool.cpu().numpy()
        got = iso.pages_compact(torch.from_numpy(table).cuda(), torch.from_numpy(refs).cuda(), pools=pool)
        at = np.flatnonzero(refs > 0)
        count = len(at)
        holes, movers = np.flatnonzero(refs[:count] <= 0), at[at >= count]
        moved = np.full(pages, -1, np.int32)
        moved[at] = at
        moved[movers] = holes
        new = np.zeros(pages, np.int32)
        new[moved[at]] = refs[at]
        inside = (table >= 0) & (table < pages)
        assert np.array_equal(n(got[0]), np.where(inside, moved[np.where(inside, table, 0)], -1))
        assert np.array_equal(n(got[1]), new) and np.array_equal(n(got[2]), moved) and n(got[3]).tolist() == [count, len(movers)]
        keep[holes] = keep[movers]
        assert np.array_equal(pool.cpu().numpy(), keep)
