"""Steps of a paged cache at the sizes where one workgroup hands over to several,
and past the sizes at which a launch's workgroups take more than one block each."""
from __future__ import annotations

import numpy as np
import pytest

from lower_convex_hull_amd import iso
from tests.test_gpu_decoding import cache, pools_of, run_compact, run_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t

    assert t.cuda.is_available()
    iso.lib()
    return t


@pytest.mark.parametrize("seqs,most,pages", [(32, 1024, 9000), (32, 1025, 9000), (1024, 32, 12288), (1024, 33, 12288), (8, 12, 12288), (8, 12, 12289)])
def test_fork_where_one_workgroup_ends(torch, seqs, most, pages):
    print(f"[decoding] {seqs} sequences of {most}, {pages} pages", flush=True)
    rng, gen = np.random.default_rng(most), torch.Generator().manual_seed(most)
    page = 2
    table, length, refs = cache(rng, seqs, min(most, pages // seqs - 2), page, pages)
    table = np.concatenate([table, np.full((seqs, most - table.shape[1]), -1, np.int32)], 1)
    pools, token_dim = pools_of(torch, gen, pages, page, False)
    parent = rng.integers(-1, seqs, seqs).astype(np.int32)
    run_fork(torch, table, length, refs, parent, page, rng.integers(0, 3, seqs).astype(np.int32), pools, token_dim)
    run_fork(torch, table, length, refs, np.arange(seqs, dtype=np.int32), page, 1, pools, token_dim)


@pytest.mark.parametrize("pages", [1023, 1024, 4095, 4096, 4097, 12288, 12289])
def test_compact_where_one_workgroup_ends(torch, pages):
    print(f"[decoding] compact {pages}", flush=True)
    rng, gen = np.random.default_rng(pages), torch.Generator().manual_seed(pages)
    for live in (0.02, 0.5, 0.98):
        refs = np.where(rng.random(pages) < live, rng.integers(1, 4, pages), rng.integers(-1, 1, pages)).astype(np.int32)
        run_compact(torch, rng.integers(-2, pages + 2, (5, 9)).astype(np.int32), refs, pools_of(torch, gen, pages, 2, True)[0])


def test_fork_of_a_large_pool(torch):
    """A pool past 128 MB of which little and of which much is copied."""
    page, pages, seqs = 4, 3000, 24
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(-100, 100, (2, pages, page, 6001), generator=gen, device="cuda", dtype=torch.int8)
    keep = pool.clone()
    table = torch.arange(seqs, dtype=torch.int32, device="cuda")[:, None] * 7
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[:, 0].long()] = 1
    length = torch.full((seqs,), 3, dtype=torch.int32, device="cuda")
    for children in (30, 2000):
        print(f"[decoding] large pool, {children} children", flush=True)
        parent = torch.arange(children, dtype=torch.int32, device="cuda") % seqs
        table2 = torch.cat([table, table * 0 - 1], 1).contiguous()
        out, ln, new, status = iso.pages_fork(table2, length, refs, parent, page_size=page, pools=pool, page_dim=1, token_dim=2)
        assert status.tolist()[:4] == [0, 0, children - min(children, seqs), children - min(children, seqs)]
        at = out[:, 0].long()
        assert torch.equal(pool[:, at, :3], keep[:, table[parent.long(), 0].long(), :3])
        rest = torch.ones(pages, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert torch.equal(pool[:, rest], keep[:, rest]) and torch.equal(pool[:, :, 3], keep[:, :, 3])
        pool.copy_(keep)
