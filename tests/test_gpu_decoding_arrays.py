"""States and pools of more arrays than one launch takes: a cache of a tensor each
for the keys and the values of every layer."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from oracle import decoding
from tests.test_decoding_abi import ARG, OK, _Fake, array, blocks, compact_args, fork_args, mem  # noqa: F401
from tests.test_gpu_decoding import cache, n, raw, run_compact, run_fork


def rows_of(mem, count, step=64, inner=4):
    return [dict(base=mem(0) + step * i, outer=1, outer_stride=0, row_stride=8, mid=1, mid_stride=0, inner=inner) for i in range(count)]


def test_many_arrays_are_checked_together(mem):
    """Any two of 40 arrays of 6 rows may not overlap, nor may one overlap another argument; 512 at most."""
    for a, b in ((0, 39), (3, 17), (20, 21), (39, 5)):
        bad = rows_of(mem, 40)
        bad[a]["base"] = bad[b]["base"] + 40
        for call in (lambda p: iso.iso_beam_reorder(p, 40, mem(5), 2, 3, None), lambda p: iso.iso_pages_fork(*fork_args(mem, pools=p, count=40)),
                     lambda p: iso.iso_pages_compact(*compact_args(mem, pools=p, count=40))):
            assert call(blocks(*bad)) == ARG, (a, b)
    bad = rows_of(mem, 40)
    bad[33]["base"] = mem(5) - 8
    assert iso.iso_beam_reorder(blocks(*bad), 40, mem(5), 2, 3, None) == ARG
    bad[33]["base"] = mem(14) + 16
    assert iso.iso_pages_fork(*fork_args(mem, pools=blocks(*bad), count=40)) == ARG
    assert iso.iso_pages_compact(*compact_args(mem, pools=blocks(*bad), count=40)) == ARG
    bad[33] = array(mem, row_stride=1)
    assert iso.iso_beam_reorder(blocks(*bad), 40, mem(5), 2, 3, None) == ARG
    none = rows_of(mem, 513, inner=0)
    assert iso.iso_beam_reorder(blocks(*none[:512]), 512, mem(5), 2, 3, None) == OK
    assert iso.iso_beam_reorder(blocks(*none), 513, mem(5), 2, 3, None) == ARG


def test_many_tensors_as_blocks():
    import torch

    states = [torch.zeros(i % 3 + 1, 6, 5) if i % 2 else torch.zeros(6, i + 1) for i in range(37)]
    dims = [i % 2 for i in range(37)]
    got, count = iso._arrays(_Fake(), states, dims, 6)
    assert count == 37
    for b, t, dim in zip(got, states, dims):
        one = iso._blocks(_Fake(), t, dim, 6)[0][0]
        assert all(getattr(b, f) == getattr(one, f) for f, _ in iso.Blocks._fields_) and b.base == t.data_ptr()
    assert ctypes.sizeof(got) == 37 * ctypes.sizeof(iso.Blocks)
    assert iso._arrays(_Fake(), states[0::2], 0, 6)[1] == 19
    for args in ((states, dims[:-1], 6), (states, 0, 6), (states[0::2], 0, 5), (states[0::2] * 28, 0, 6)):
        with pytest.raises(ValueError):
            iso._arrays(_Fake(), *args)


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("count", [16, 17, 37, 64])
def test_reorder_of_many_arrays(torch, count):
    print(f"[decoding] reorder of {count} arrays", flush=True)
    gen = torch.Generator().manual_seed(count)
    parent = torch.tensor([[1, 0, 0], [5, 4, 3]], dtype=torch.int32)
    kinds = [((6, 5), torch.float32, 0), ((2, 6, 3, 9), torch.float16, 1), ((6, 37), torch.uint8, 0), ((3, 6), torch.int64, 1)]
    states = [raw(torch, gen, *kinds[i % 4][:2]) for i in range(count)]
    dims = [kinds[i % 4][2] for i in range(count)]
    dev = [s.cuda() for s in states]
    assert iso.beam_reorder(dev, parent.cuda(), dim=dims) is dev
    for s, d, dim in zip(states, dev, dims):
        assert np.array_equal(d.cpu().numpy(), decoding.beam_reorder(s.numpy(), parent.numpy(), dim))
    with pytest.raises(iso.IsoError):
        iso.beam_reorder(dev[:-1] + dev[:1], parent.cuda(), dim=dims[:-1] + dims[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("count", [17, 35])
@pytest.mark.parametrize("seqs,children,pages", [(5, 40, 300), (5, 40, 13001), (30, 1100, 4000)])
def test_pages_of_many_arrays(torch, count, seqs, children, pages):
    print(f"[decoding] {count} pools, {seqs} to {children} of {pages}", flush=True)
    rng, gen = np.random.default_rng(pages), torch.Generator().manual_seed(pages)
    page = 3
    table, length, refs = cache(rng, seqs, 4, page, pages)
    pools = [raw(torch, gen, (1 + i % 2, pages, page, 1 + i % 3), torch.float16) for i in range(count)]
    parent, grow = rng.integers(-1, seqs, children).astype(np.int32), rng.integers(0, 4, children).astype(np.int32)
    run_fork(torch, table, length, refs, parent, page, grow, pools, 2)
    run_fork(torch, table, length, refs, parent, page, 1, pools, 2)
    run_compact(torch, table, refs, pools)
    run_compact(torch, table, (rng.random(pages) < 0.5).astype(np.int32), pools)


@pytest.mark.gpu
def test_many_arrays_in_a_graph(torch):
    gen = torch.Generator().manual_seed(3)
    states = [torch.randn(6, 4, 3, generator=gen).cuda() for _ in range(33)]
    parent = torch.tensor([[1, 2, 0], [3, 3, 5]], dtype=torch.int32, device="cuda")
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    fork = (i(0, 2).view(2, 1), i(3, 2), i(1, 0, 1, 0, 0, 0), i(0, 0, 1, 1))

    def steps(states):
        iso.beam_reorder(states, parent)
        return iso.pages_fork(*fork, page_size=4, pools=states)

    steps([s.clone() for s in states])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = steps(states)
    for k in range(4):
        new = [torch.randn(6, 4, 3, generator=gen).cuda() for _ in states]
        want = [s.clone() for s in new]
        eager = steps(want)
        for s, v in zip(states, new):
            s.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(states, want)), k
        assert all(torch.equal(a, b) for a, b in zip(out, eager)) and n(out[3])[2] == 2
