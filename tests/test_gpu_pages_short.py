"""Reservations that the pool has too few free pages for: nothing is changed,
whatever the number of CTAs that count the pages and of requests that ask."""
import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.serving_ref import fork_ref, reserve_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _reserve(n, lens, table, held, refs, P):
    """The call on the device, equal to the replica's in every entry; (table, held, refs, copies, missing, error)."""
    B, cols = table.shape
    desc = da.Desc.make(B=B, H_kv=1, G=8, D_qk=64, D_v=64, page_size=P, max_pages_per_seq=cols, num_pages=len(refs), kv_dtype=da.KV_BF16)
    d = [_dev(x) for x in (lens, table, held, refs)]
    copies, missing, err = _dev([[5, 5]] * B), _dev([77]), _dev([0])
    da.reserve_pages(desc, *d, copies, missing, new_tokens=_dev(n), device_error=err)
    want = reserve_ref(n, lens, table, held, refs, P)
    torch.cuda.synchronize()
    for name, a, b in zip(("table", "held", "refs", "copies"), d[1:] + [copies], want):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert int(missing) == want[4] and int(err) == want[5]
    return want


def _unchanged(want, table, held, refs, missing):
    """A replica's result that says: `missing` pages too few, and so nothing was done."""
    assert want[4] == missing and want[5] == da.DA_DEV_NO_PAGES
    assert np.array_equal(want[0], table) and np.array_equal(want[1], held) and np.array_equal(want[2], refs)
    assert (want[3] == -1).all()


@pytest.mark.parametrize("pages", [60, 8192, 8193, 20000, 70001, 300000, 1 << 21])
def test_the_last_free_pages_lie_in_several_shares(pages):
    """One to sixteen CTAs: four free pages in different shares, a row that needs five, two that need five together, and
    then as many as there are."""
    B, P, cols = 5, 16, 40
    refs = np.ones(pages, np.int32)                       # a prefix cache has all of them
    free = sorted({1, pages // 3, pages // 2, pages - 1})
    refs[free] = 0
    table, held, lens = np.full((B, cols), -9, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    table[0, :2], held[0], lens[0] = (5, 6), 2, 32        # full pages, shared with the prefix cache
    refs[[5, 6]] += 1
    for n in ([80, 0, 0, 0, 0], [0, 0, 0, 80, 0], [40, 0, 20, 0, 0]):
        _unchanged(_reserve(n, lens, table, held, refs, P), table, held, refs, 1)
    _unchanged(_reserve([0, 16 * 40, 0, 0, 0], lens, table, held, refs, P), table, held, refs, 36)
    got = _reserve([33, 0, 0, 16, 0], lens, table, held, refs, P)
    assert got[4] == got[5] == 0 and got[0][0, :5].tolist() == [5, 6] + free[:3] and got[0][3, 0] == free[3]
    _unchanged(_reserve([0, 1, 0, 0, 0], lens, got[0], got[1], got[2], P), got[0], got[1], got[2], 1)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 4000, 8192])
@pytest.mark.parametrize("outsider", [False, True])
def test_many_rows_that_share_last_pages(B, outsider):
    """Rows in families of one to five that share a partly filled last page. All of them write (the lowest of a family keeps
    the page), or one of some families does not, and some pages are held by a prefix cache too (no one keeps them): one free
    page too few, and then just enough."""
    g, P, cols = np.random.RandomState(B), 4, 3
    family, b = np.zeros(B, np.int64), 0
    while b < B:
        n = int(g.randint(1, 6))
        family[b:b + n] = b
        b += n
    pool = 3 * B
    lens, table, held, refs = np.zeros(B, np.int32), np.full((B, cols), -9, np.int32), np.zeros(B, np.int32), np.zeros(pool, np.int32)
    firsts = np.unique(family)
    n = np.zeros(B, np.int64)
    n[firsts] = 6
    table, held, refs = reserve_ref(n.tolist(), lens, table, held, refs, P)[:3]
    lens[firsts] = 6                                      # two pages, the second half full
    table, held, lens, refs = fork_ref(family.tolist(), lens, table, held, refs, np.full_like(table, -9), P)[:4]
    asks = np.where(g.rand(B) < 0.3, 5, 1)                # five tokens: a page more
    if outsider:
        asks[g.rand(B) < 0.15] = 0
        refs[table[firsts[g.rand(len(firsts)) < 0.3], 1]] += 1
    need = reserve_ref(asks.tolist(), lens, table, held, refs, P)
    assert need[4] == 0 and (need[3][:, 0] >= 0).any()
    used = int((need[2][refs == 0] > 0).sum())            # fresh pages that it takes
    free = np.flatnonzero(refs == 0)
    for left in (used - 1, 0, used):
        tight = refs.copy()
        tight[g.permutation(free)[left:]] = 1
        got = _reserve(asks.tolist(), lens, table, held, tight, P)
        if left < used:
            _unchanged(got, table, held, tight, used - left)
        else:
            assert got[4] == got[5] == 0 and not (got[2] == 0).any()
