"""Refusals and sizes of the decoding steps, through the C ABI and the binding.
No kernel is launched here."""
from __future__ import annotations

import ctypes

import pytest

from lower_convex_hull_amd import iso

ARG, WS, OK = iso.ISO_ERR_ARG, iso.ISO_ERR_WORKSPACE, iso.ISO_OK


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 17)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    place = lambda k=0: base + 4096 * k  # noqa: E731
    place.keep = buf
    return place


def select_args(m, **over):
    a = dict(logits=m(0), dtype=iso.ISO_DT_F32, batch=2, beams=3, vocab=8, ld=8, score=m(1), weight=None, ended=None,
             end_token=2, temperature=1.0, take=4, out_score=m(2), out_logp=m(3), out_parent=m(4), out_token=m(5),
             ws=m(6), ws_bytes=1 << 14, stream=None)
    a.update(over)
    return list(a.values())


BAD_SELECT = [dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(beams=0), dict(beams=129), dict(take=0), dict(take=129),
              dict(vocab=0), dict(vocab=1 << 31), dict(ld=7), dict(temperature=0.0), dict(temperature=-1.0),
              dict(temperature=1e-29), dict(temperature=float("nan")), dict(temperature=float("inf")), dict(logits=None),
              dict(score=None), dict(out_score=None), dict(out_logp=None), dict(out_parent=None), dict(out_token=None),
              dict(batch=1 << 30), dict(batch=1 << 24, ld=1 << 60)]


@pytest.mark.parametrize("over", BAD_SELECT, ids=str)
def test_select_refuses(mem, over):
    assert iso.iso_beam_select(*select_args(mem, **over)) == ARG


def test_select_refuses_places(mem):
    for over in (dict(logits=mem(0) + 2), dict(score=mem(1) + 2), dict(weight=mem(7) + 1), dict(out_token=mem(5) + 2),
                 dict(out_score=mem(0) + 64), dict(out_logp=mem(2) + 4), dict(out_parent=mem(1)), dict(weight=mem(3)),
                 dict(ended=mem(4) + 1), dict(ws=mem(6) + 8)):
        assert iso.iso_beam_select(*select_args(mem, **over)) == ARG, over
    need = iso.iso_beam_select_workspace_bytes(2, 3, 8, 4, iso.ISO_DT_F32)
    assert need > 0
    assert iso.iso_beam_select(*select_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_beam_select(*select_args(mem, ws=None, ws_bytes=0)) == WS
    assert iso.iso_beam_select(*select_args(mem, batch=0, logits=None, score=None)) == OK


def test_select_workspace_of_bad_sizes():
    for a in ((-1, 3, 8, 4, 0), (1, 0, 8, 4, 0), (1, 129, 8, 4, 0), (1, 3, 0, 4, 0), (1, 3, 8, 129, 0), (1, 3, 8, 4, 3),
              (1 << 31, 1, 8, 4, 0)):
        assert iso.iso_beam_select_workspace_bytes(*a) == 0


def blocks(*rows):
    out = (iso.Blocks * max(1, len(rows)))()
    for b, r in zip(out, rows):
        for name, value in r.items():
            setattr(b, name, value)
    return out


def array(m, k=0, **over):
    a = dict(base=m(k), outer=2, outer_stride=1024, row_stride=128, mid=2, mid_stride=64, inner=48)
    a.update(over)
    return a


BAD_ARRAYS = [dict(outer=-1), dict(mid=-1), dict(inner=-1), dict(base=None), dict(outer_stride=-1024), dict(row_stride=-128),
              dict(mid_stride=-64), dict(mid_stride=32), dict(row_stride=64), dict(outer_stride=512), dict(inner=65),
              dict(inner=1 << 41), dict(outer=1 << 31), dict(outer_stride=1 << 62, outer=3), dict(row_stride=1 << 61)]


@pytest.mark.parametrize("over", BAD_ARRAYS, ids=str)
def test_arrays_are_refused(mem, over):
    """6 rows of 2 x 2 blocks: one array that is not right, in each call that takes some."""
    bad = blocks(array(mem, **over))
    assert iso.iso_beam_reorder(bad, 1, mem(5), 2, 3, None) == ARG
    assert iso.iso_pages_fork(*fork_args(mem, pools=bad, count=1, page_size=4)) == ARG
    assert iso.iso_pages_compact(*compact_args(mem, pools=bad, count=1)) == ARG


def test_reorder_refuses(mem):
    good = blocks(array(mem))
    assert iso.iso_beam_reorder(good, 1, None, 2, 3, None) == ARG
    assert iso.iso_beam_reorder(good, 1, mem(5) + 2, 2, 3, None) == ARG
    assert iso.iso_beam_reorder(good, 1, mem(0) + 512, 2, 3, None) == ARG  # parents inside the states
    assert iso.iso_beam_reorder(good, 1, mem(5), 2, 0, None) == ARG
    assert iso.iso_beam_reorder(good, 1, mem(5), 2, 129, None) == ARG
    assert iso.iso_beam_reorder(good, 1, mem(5), -1, 3, None) == ARG
    assert iso.iso_beam_reorder(good, -1, mem(5), 2, 3, None) == ARG
    assert iso.iso_beam_reorder(None, 1, mem(5), 2, 3, None) == ARG
    assert iso.iso_beam_reorder(blocks(*[array(mem)] * 17), 17, mem(5), 2, 3, None) == ARG
    assert iso.iso_beam_reorder(blocks(array(mem), array(mem)), 2, mem(5), 2, 3, None) == ARG  # the same twice
    assert iso.iso_beam_reorder(blocks(array(mem), array(mem, base=mem(0) + 1776 - 4)), 2, mem(5), 2, 3, None) == ARG
    # nothing to do
    assert iso.iso_beam_reorder(None, 0, mem(5), 2, 3, None) == OK
    assert iso.iso_beam_reorder(good, 1, None, 0, 3, None) == OK
    assert iso.iso_beam_reorder(blocks(array(mem, inner=0), array(mem, outer=0), array(mem, mid=0)), 3, mem(5), 2, 3, None) == OK


def fork_args(m, **over):
    a = dict(table=m(8), length=m(9), seqs=2, max_pages=3, refs=m(10), pages=6, page_size=4, parent=m(11), grow=None,
             grow_all=1, children=2, pools=None, count=0, new_table=m(12), new_length=m(13), new_refs=m(14), status=m(15),
             ws=m(16), ws_bytes=1 << 14, stream=None)
    a.update(over)
    return list(a.values())


BAD_FORK = [dict(seqs=-1), dict(seqs=(1 << 20) + 1), dict(children=-1), dict(children=(1 << 20) + 1), dict(pages=-1),
            dict(pages=1 << 31), dict(max_pages=-1), dict(max_pages=1 << 31), dict(page_size=0), dict(page_size=-4),
            dict(page_size=1 << 31), dict(table=None), dict(length=None), dict(refs=None), dict(parent=None),
            dict(new_table=None), dict(new_length=None), dict(new_refs=None), dict(status=None), dict(count=1), dict(count=-1)]


@pytest.mark.parametrize("over", BAD_FORK, ids=str)
def test_fork_refuses(mem, over):
    assert iso.iso_pages_fork(*fork_args(mem, **over)) == ARG


def test_fork_refuses_places(mem):
    for over in (dict(table=mem(8) + 2), dict(length=mem(9) + 1), dict(refs=mem(10) + 2), dict(parent=mem(11) + 2),
                 dict(grow=mem(17) + 2), dict(new_table=mem(12) + 2), dict(status=mem(15) + 2), dict(new_table=mem(8)),
                 dict(new_refs=mem(10)), dict(new_length=mem(11)), dict(status=mem(12)), dict(grow=mem(13)),
                 dict(ws=mem(16) + 8)):
        assert iso.iso_pages_fork(*fork_args(mem, **over)) == ARG, over
    pool = blocks(array(mem))
    assert iso.iso_pages_fork(*fork_args(mem, pools=pool, count=1, page_size=5)) == ARG  # 48 bytes are not 5 tokens
    assert iso.iso_pages_fork(*fork_args(mem, pools=pool, count=1, table=mem(0) + 64)) == ARG
    assert iso.iso_pages_fork(*fork_args(mem, pools=pool, count=1, new_refs=mem(0) + 64)) == ARG
    need = iso.iso_pages_fork_workspace_bytes(2, 2, 6)
    assert need > 0
    assert iso.iso_pages_fork(*fork_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_pages_fork(*fork_args(mem, ws=None)) == WS
    for a in ((-1, 2, 6), (2, -1, 6), (2, 2, -1), (1 << 21, 2, 6), (2, 1 << 21, 6), (2, 2, 1 << 31)):
        assert iso.iso_pages_fork_workspace_bytes(*a) == 0


def compact_args(m, **over):
    a = dict(table=m(8), entries=6, refs=m(10), pages=6, pools=None, count=0, new_table=m(12), new_refs=m(14), moved=m(13),
             status=m(15), ws=m(16), ws_bytes=1 << 14, stream=None)
    a.update(over)
    return list(a.values())


BAD_COMPACT = [dict(entries=-1), dict(entries=1 << 51), dict(pages=-1), dict(pages=1 << 31), dict(table=None), dict(refs=None),
               dict(new_table=None), dict(new_refs=None), dict(moved=None), dict(status=None), dict(count=1), dict(count=17)]


@pytest.mark.parametrize("over", BAD_COMPACT, ids=str)
def test_compact_refuses(mem, over):
    assert iso.iso_pages_compact(*compact_args(mem, **over)) == ARG


def test_compact_refuses_places(mem):
    for over in (dict(table=mem(8) + 2), dict(refs=mem(10) + 1), dict(moved=mem(13) + 2), dict(new_table=mem(8)),
                 dict(new_refs=mem(10)), dict(moved=mem(14) + 4), dict(status=mem(12)), dict(ws=mem(16) + 16)):
        assert iso.iso_pages_compact(*compact_args(mem, **over)) == ARG, over
    need = iso.iso_pages_compact_workspace_bytes(6)
    assert need > 0
    assert iso.iso_pages_compact(*compact_args(mem, ws_bytes=need - 1)) == WS
    assert iso.iso_pages_compact(*compact_args(mem, ws=None)) == WS
    assert iso.iso_pages_compact_workspace_bytes(-1) == 0 and iso.iso_pages_compact_workspace_bytes(1 << 31) == 0


def test_binding_refuses_cpu_tensors():
    import torch

    x, s = torch.zeros(6, 8), torch.zeros(2, 3)
    i = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda: iso.beam_select(x, s), lambda: iso.beam_reorder(x, i), lambda: iso.pages_fork(i, i[0], i[0], i[0], page_size=4),
                 lambda: iso.pages_compact(i, i[0])):
        with pytest.raises(TypeError):
            call()


class _Fake:
    """What _blocks asks of a launch."""

    index, other, dev = -1, None, "cpu"


def as_rows(t, dim, token_dim=None):
    """Every row's bytes as the description says they lie, by rows."""
    b = iso._blocks(_Fake(), t, dim, t.shape[dim], token_dim)[0][0]
    rows = []
    for r in range(t.shape[dim]):
        rows.append(b"".join(ctypes.string_at(b.base + o * b.outer_stride + r * b.row_stride + m * b.mid_stride, b.inner)
                             for o in range(b.outer) for m in range(b.mid)))
    return b, rows


def test_tensors_as_blocks():
    """The blocks hold each row's elements, in order, whatever the tensor's shape and strides."""
    import torch

    base = torch.arange(2 * 4 * 3 * 6 * 5, dtype=torch.int32)
    full = base.view(2, 4, 3, 6, 5)
    cases = [(full, 0, None, 1, 1), (full, 1, None, 2, 1), (full, 2, None, 8, 1), (full, 3, None, 24, 1), (full, 4, None, 144, 1),
             (full[:, :, :, :4], 1, None, 2, 3), (full[:, :, :, :4], 1, 3, 2, 3), (full[:, :, 1:2, :, :], 1, None, 2, 1),
             (full[:, :, :, 2:3], 1, None, 2, 3), (full, 1, 2, 2, 1), (full, 1, 4, 2, 18), (base, 0, None, 1, 1), (base[::3], 0, None, 1, 1),
             (full[0, :, 0], 0, None, 1, 1)]
    for t, dim, token_dim, outer, mid in cases:
        b, rows = as_rows(t, dim, token_dim)
        assert (b.outer, b.mid) == (outer, mid), (t.shape, dim)
        for r, got in enumerate(rows):
            assert got == t.select(dim, r).contiguous().numpy().tobytes()
    for t, dim, token_dim in ((full[:, :, :2, :4], 0, None), (full[:, 1:3], 2, None), (full[..., :3], 1, 3), (full, 1, 1), (full, 1, 5)):
        with pytest.raises(ValueError):
            iso._blocks(_Fake(), t, dim, t.shape[dim], token_dim)
    for tensors, dims, rows in ((full, 5, 5), (full, -1, 5), ([full] * 17, 0, 2), ([full, base], (0, 0, 0), 2), (full, 1, 5)):
        with pytest.raises(ValueError):
            iso._blocks(_Fake(), tensors, dims, rows)


def test_numbers_past_32_bits_are_refused():
    assert iso._int32(-1 << 31, "x") == -1 << 31 and iso._int32((1 << 31) - 1, "x") == (1 << 31) - 1
    for x in (1 << 31, (-1 << 31) - 1):
        with pytest.raises(ValueError):
            iso._int32(x, "x")
