"""The plain forms of the decoding steps (oracle/decoding.py) against worked
examples and what must hold whatever the inputs."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import decoding


def test_select_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.125, 0.5, 0.375]]))
    score = np.array([[-1.0, -1.5]], np.float32)
    got = decoding.beam_select(x, score, 4)[0]
    want = [(0, 0, -1 + math.log(0.5)), (1, 1, -1.5 + math.log(0.5)), (0, 1, -1 + math.log(0.25)), (0, 2, -1 + math.log(0.25)),
            (1, 2, -1.5 + math.log(0.375)), (1, 0, -1.5 + math.log(0.125))]
    assert [(c["parent"], c["token"]) for c in got] == [w[:2] for w in want]
    assert np.allclose([c["score"] for c in got], [w[2] for w in want], atol=1e-12)


def test_select_ended_first_and_masks():
    x = np.array([[0.0, -np.inf, 0.0], [1.0, np.nan, 0.0], [-np.inf] * 3, [np.inf, 0.0, 0.0]])
    score = np.zeros((1, 4), np.float32)
    got = decoding.beam_select(x, score, 3)[0]
    assert [(c["parent"], c["token"]) for c in got] == [(0, 0), (0, 2)]
    ended = np.array([[False, True, False, False]])
    got = decoding.beam_select(x, score, 3, ended=ended, end_token=9)[0]
    assert [(c["parent"], c["token"], c["logp"]) for c in got][0] == (1, 9, 0.0)
    score[0, 0] = -np.inf
    assert [c["parent"] for c in decoding.beam_select(x, score, 3, ended=ended)[0]] == [1]
    weight = np.array([[1, 0, 1, 1]], np.float32)
    assert decoding.beam_select(x, score, 3, ended=ended, weight=weight)[0] == []


def test_select_is_the_largest_of_all_scores():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((12, 50))
    score = -rng.random((3, 4)).astype(np.float32)
    for b, got in enumerate(decoding.beam_select(x, score, 7)):
        every = np.concatenate([score[b, k] + decoding.row_logp(x[4 * b + k])[0] for k in range(4)])
        assert np.allclose([c["score"] for c in got[:7]], np.sort(every)[::-1][:7], atol=1e-12)
        assert math.isclose(np.exp(decoding.row_logp(x[4 * b])[0]).sum(), 1.0)


def test_reorder_keeps_rows_without_a_parent():
    s = np.arange(12).reshape(6, 2)
    got = decoding.beam_reorder(s, np.array([[1, 1, -1], [3, 0, 4]], np.int32))
    assert got[:, 0].tolist() == [2, 2, 4, 6, 8, 8]


def cache(rng, seqs, most, page, pages, shared=2):
    """Sequences that share their first pages in groups of two."""
    table, length = np.full((seqs, most), -1, np.int32), rng.integers(0, most * page // 2 + 1, seqs).astype(np.int32)
    length[1::2] = length[0:seqs - seqs % 2:2]
    ids = iter(rng.permutation(pages))
    for s in range(seqs):
        for j in range(-(-int(length[s]) // page)):
            table[s, j] = table[s - 1, j] if s % 2 and j < shared else next(ids)
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, length, refs


def test_fork_by_hand():
    # two sequences of 5 and 4 tokens, pages of 4: 7 -> [2, 0], 4 -> [3]; page 1 free, 4 held from outside
    table, length = np.array([[2, 0, -1], [3, -1, -1]], np.int32), np.array([5, 4], np.int32)
    refs = np.array([1, 0, 1, 1, 1, 0], np.int32)
    pool = np.arange(6 * 4).reshape(6, 4)
    out, ln, rf, status, pools = decoding.pages_fork(table, length, refs, np.array([0, 0, -1], np.int32), 4,
                                                     np.array([1, 1, 3], np.int32), [pool])
    # sequence 1 ends (3 is free again); child 0 keeps page 0, child 1 copies its token to 1, the new one takes 3
    assert out.tolist() == [[2, 0, -1], [2, 1, -1], [3, -1, -1]] and ln.tolist() == [6, 6, 3]
    assert rf.tolist() == [1, 1, 2, 1, 1, 0] and status.tolist() == [0, 0, 1, 2, 1]
    assert pools[0][1].tolist() == [0, 5, 6, 7]
    # held from outside too: nobody keeps page 0, and there is one page too few
    refs[0], refs[5] = 2, 1
    out, ln, rf, status, _ = decoding.pages_fork(table, length, refs, np.array([0, 0, -1], np.int32), 4,
                                                 np.array([1, 1, 3], np.int32))
    assert status.tolist() == [1, 0, 0, 0, 0] and rf.tolist() == refs.tolist() and (out == -1).all()


@pytest.mark.parametrize("page", [1, 3, 8])
def test_fork_invariants(page):
    """Counts are the entries; a token is in one page of each holder, and a page that a child goes on to write is its own."""
    rng = np.random.default_rng(page)
    for _ in range(30):
        seqs, most, pages = int(rng.integers(1, 7)), 9, 120
        table, length, refs = cache(rng, seqs, most, page, pages)
        stamp = rng.integers(1, 1 << 40, (pages, page))
        children = int(rng.integers(0, 12))
        parent = rng.integers(-1, seqs, children).astype(np.int32)
        grow = rng.integers(0, page + 2, children).astype(np.int32)
        out, ln, rf, status, (pool,) = decoding.pages_fork(table, length, refs, parent, page, grow, [stamp])
        assert status[:2].tolist() == [0, 0]
        assert np.array_equal(np.bincount(out[out >= 0], minlength=pages), rf)
        assert status[4] == (rf == 0).sum()
        for i in range(children):
            old = int(length[parent[i]]) if parent[i] >= 0 else 0
            for t in range(old):
                assert pool[out[i, t // page], t % page] == stamp[table[parent[i], t // page], t % page]
            for t in range(old, int(ln[i])):
                others = [k for k in range(children) if out[i, t // page] in out[k]]
                assert rf[out[i, t // page]] == 1 and others == [i]


def test_compact_invariants():
    rng = np.random.default_rng(3)
    for _ in range(30):
        pages = int(rng.integers(0, 40))
        refs = rng.integers(-1, 3, pages).astype(np.int32)
        table = rng.integers(-2, pages + 2, (3, 5)).astype(np.int32)
        stamp = rng.integers(0, 1 << 40, (pages, 2))
        out, rf, moved, status, (pool,) = decoding.pages_compact(table, refs, [stamp])
        n = int((refs > 0).sum())
        assert status[0] == n and (rf[:n] > 0).all() and (rf[n:] == 0).all()
        for q in range(pages):
            if refs[q] > 0:
                assert rf[moved[q]] == refs[q] and (pool[moved[q]] == stamp[q]).all() and (q >= n or moved[q] == q)
            else:
                assert moved[q] == -1
