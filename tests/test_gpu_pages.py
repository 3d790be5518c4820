"""The pages of a cache: fork, reserve, free, compact, copy, against a replica
in Python: every table entry, count and pair equal, and the tokens that rows
read stay theirs through long random runs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.serving_ref import compact_ref, fork_ref, reserve_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _desc(B, P, cols, pages, s_q=1, **kw):
    base = dict(H_kv=1, G=8, D_qk=64, D_v=64, kv_dtype=da.KV_BF16)
    return da.Desc.make(B=B, page_size=P, max_pages_per_seq=cols, num_pages=pages, s_q=s_q, **{**base, **kw})


class State:
    """Rows on the device and their replica; `owner[page][slot]` says which token text is there."""

    def __init__(self, B, P, cols, pages):
        self.B, self.P, self.cols, self.pages = B, P, cols, pages
        self.desc = _desc(B, P, cols, pages)
        self.table, self.other = np.full((B, cols), -9, np.int32), np.full((B, cols), -9, np.int32)
        self.held, self.lens, self.refs = np.zeros(B, np.int32), np.zeros(B, np.int32), np.zeros(pages, np.int32)

    def reserve(self, n, kind="list"):
        d = [_dev(x) for x in (self.lens, self.table, self.held, self.refs)]
        copies, missing, err = _i32([[5, 5]] * self.B), _i32([77]), _i32([0])
        desc = self.desc if kind == "list" else _desc(self.B, self.P, self.cols, self.pages, s_q=n[0])
        da.reserve_pages(desc, *d, copies, missing, new_tokens=_i32(n) if kind == "list" else None, device_error=err)
        want = reserve_ref(n, self.lens, self.table, self.held, self.refs, self.P)
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "held", "refs", "copies"), d[1:] + [copies], want):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert int(missing) == want[4] and int(err) == want[5]
        self.table, self.held, self.refs = want[:3]
        return want[3], want[4], want[5]

    def fork(self, parents):
        d = [_dev(x) for x in (self.lens, self.table, self.held, self.refs, self.other)]
        held, lens, err = _i32([-1] * self.B), _i32([-1] * self.B), _i32([0])
        da.fork_pages(self.desc, _i32(parents), *d, held, lens, device_error=err)
        want = fork_ref(parents, self.lens, self.table, self.held, self.refs, self.other, self.P)
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "held", "lens", "refs"), [d[4], held, lens, d[3]], want):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert int(err) == want[4]
        self.other = self.table
        self.table, self.held, self.lens, self.refs = want[:4]

    def free(self, done):
        d = [_dev(x) for x in (self.lens, self.table, self.held, self.refs)]
        da.free_pages(self.desc, _i32(done), *d)
        for b, x in enumerate(done):
            if x:
                np.subtract.at(self.refs, self.table[b, :self.held[b]], 1)
                self.held[b] = self.lens[b] = 0
        torch.cuda.synchronize()
        for name, a, b in zip(("lens", "table", "held", "refs"), d, (self.lens, self.table, self.held, self.refs)):
            assert np.array_equal(a.cpu().numpy(), b), name

    def compact(self):
        into, refs, page = _dev(self.other), _i32([-5] * self.pages), _i32([-5] * self.pages)
        copies, counts = torch.full((self.pages // 2, 2), -5, dtype=torch.int32, device="cuda"), _i32([-1, -1])
        da.compact_pages(self.desc, _dev(self.table), _dev(self.held), _dev(self.refs), into, refs, page, copies, counts)
        want = compact_ref(self.table, self.held, self.refs, self.other)
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "refs", "page"), (into, refs, page), want):
            assert np.array_equal(a.cpu().numpy(), b), name
        m = len(want[3])
        assert counts.tolist() == [want[4], m] and [tuple(x) for x in copies[:m].tolist()] == want[3]
        assert (copies[m:] == -5).all()
        self.other = self.table
        self.table, self.refs = want[:2]
        return want[3]


@pytest.mark.parametrize("B,P,cols,pages,seed", [(1, 16, 8, 20, 0), (5, 16, 12, 60, 1), (37, 8, 30, 700, 2), (8, 64, 4, 33, 3), (16, 3, 40, 500, 4),
                                                 (64, 1, 100, 5000, 5)])
def test_random_runs_of_all_of_them(B, P, cols, pages, seed):
    """Rows grow, fork, shrink (refused drafts), end and are packed; every row's text is read back through its table."""
    g = np.random.RandomState(seed)
    s = State(B, P, cols, pages)
    text = [[] for _ in range(B)]                         # what each row has written
    pool = np.full((pages, P), -1, np.int64)
    stamp, short = 0, 0

    def write(b, n):
        nonlocal stamp
        for _ in range(n):
            L = int(s.lens[b])
            page = int(s.table[b, L // P])
            assert s.refs[page] == 1                      # nobody else reads what is written
            pool[page, L % P] = stamp
            text[b].append(stamp)
            stamp += 1
            s.lens[b] += 1

    def read_back():
        for b in range(B):
            assert [int(pool[s.table[b, t // P], t % P]) for t in range(s.lens[b])] == text[b]
    for step in range(60):
        what = g.choice(["grow", "grow", "grow", "fork", "shrink", "free", "compact"])
        if what == "grow":
            n = g.choice([0, 1, 1, 2, 5, 40], size=B)
            copies, missing, err = s.reserve(n.tolist())
            short += missing > 0
            if not err & 256:
                for src, dst in copies.tolist():
                    if src >= 0:
                        pool[dst] = pool[src]
                for b in range(B):
                    if s.lens[b] + n[b] <= cols * P:
                        write(b, n[b])
        elif what == "fork":
            parents = g.randint(-1, B, size=B)
            s.fork(parents.tolist())
            text = [list(text[r]) if r >= 0 else [] for r in parents]
        elif what == "shrink":
            for b in range(B):
                k = int(g.randint(0, min(s.lens[b], 2 * P) + 1)) if g.rand() < 0.5 else 0
                s.lens[b] -= k
                text[b] = text[b][:s.lens[b]]
        elif what == "free":
            done = (g.rand(B) < 0.3).astype(int).tolist()
            s.free(done)
            text = [[] if d else x for d, x in zip(done, text)]
        else:
            old = pool.copy()
            for src, dst in s.compact():
                pool[dst] = old[src]
        read_back()
        held = np.zeros(pages, np.int64)
        for b in range(B):
            np.add.at(held, s.table[b, :s.held[b]], 1)
        assert np.array_equal(held, s.refs)               # every hold is a table entry


def test_many_rows():
    """More rows than find out by a hash table who keeps a page, and the largest number of them."""
    g = np.random.RandomState(7)
    for B in (1024, 1025, 2500, 8192):
        s = State(B, 4, 12, 6 * B)
        s.reserve(g.randint(0, 12, size=B).tolist())
        s.lens = np.maximum(s.held * 4 - g.randint(0, 4, size=B), 0).astype(np.int32)
        for _ in range(2):
            s.fork((np.arange(B) - g.randint(0, 3, size=B) % (np.arange(B) + 1)).tolist())
            copies, missing, _ = s.reserve(g.choice([0, 1, 5], size=B).tolist())
            assert missing == 0 and (copies[:, 0] >= 0).any()
        s.free((g.rand(B) < 0.5).astype(int).tolist())
        s.compact()


def test_a_pool_of_one_page():
    s = State(1, 16, 1, 1)
    s.reserve([5])
    s.lens[0] = 5
    assert s.compact() == []
    s.fork([0])
    s.reserve([11])
    s.fork([-1])
    assert s.compact() == [] and s.refs[0] == 0


def test_every_holder_of_a_page_writes_to_it():
    """Six rows share one partly filled page: the lowest keeps it; when one of them sits out, all writers copy."""
    s = State(6, 16, 4, 12)
    s.reserve([20, 0, 0, 0, 0, 0])
    s.lens[0] = 20
    s.fork([0] * 6)
    assert s.refs[s.table[0, 1]] == 6
    copies, _, _ = s.reserve([1, 1, 1, 0, 1, 1])
    assert (copies[[0, 1, 2, 4, 5], 0] >= 0).all() and copies[3, 0] == -1
    for pages in (12, 13):                                # two are in use; five copies and one page more each: eleven
        s2 = State(6, 16, 4, pages)
        s2.reserve([20, 0, 0, 0, 0, 0])
        s2.lens[0] = 20
        s2.fork([0] * 6)
        copies, missing, _ = s2.reserve([13] * 6)
        if pages == 12:
            assert missing == 1 and (copies == -1).all()
        else:
            assert copies[0, 0] == -1 and (copies[1:, 0] >= 0).all() and (s2.held == 3).all()


def test_reservations_that_do_not_fit_change_nothing():
    s = State(4, 16, 8, 9)
    s.reserve([40, 0, 0, 0])
    s.lens[0] = 40
    s.fork([0, 0, 0, -1])
    before = s.refs.copy()
    _, missing, err = s.reserve([80, 80, 9, 80])          # five, five, one and five more, and copies of the shared last page
    assert missing > 0 and err == 256 and np.array_equal(before, s.refs)
    _, missing, err = s.reserve([1, 0, 200, 0])           # a row past its table is left alone, the other served
    assert missing == 0 and err == 2
    s.lens[3] = -4
    _, missing, err = s.reserve([0, 0, 0, 3], )
    assert missing == 0 and err == 4 and s.held[3] == 1
    s.reserve([2, 2, 2, 2], kind="s_q")


def test_errors_of_tables_and_parents():
    d = _desc(3, 16, 4, 10)
    refs, err = _i32([1] * 10), _i32([0])
    table = _i32([[0, 1, 2, 3], [4, 77, 5, -1], [6, 7, 8, 9]])
    new, held, lens = _i32([[-3] * 4] * 3), _i32([0] * 3), _i32([0] * 3)
    da.fork_pages(d, _i32([1, 3, -1]), _i32([33, 40, 10]), table, _i32([3, 3, 9]), refs, new, held, lens, device_error=err)
    assert int(err) == da.DA_DEV_BAD_PAGE | da.DA_DEV_BAD_REQUEST
    assert held.tolist() == [3, 0, 0] and lens.tolist() == [40, 0, 0] and new.tolist() == [[4, 77, 5, -3], [-3] * 4, [-3] * 4]
    assert refs.tolist() == [0, 0, 0, 1, 1, 1, 0, 0, 0, 0]
    err.zero_()
    da.free_pages(d, _i32([0, 7, 0]), lens, new, _i32([3, 0, 0]), refs, device_error=err)
    assert int(err) == 0
    copies, missing = _i32([[0, 0]] * 3), _i32([0])
    da.reserve_pages(d, _i32([20, 0, 0]), table.roll(-1, 0).contiguous(), _i32([2, 0, 0]), refs, copies, missing, device_error=err)
    assert int(err) == da.DA_DEV_BAD_PAGE and copies.tolist() == [[-1, -1]] * 3 and int(missing) == 0


@pytest.mark.parametrize("pages", [8192, 8193, 20000, 70001, 300000, 1 << 21])
def test_large_pools_take_clusters(pages):
    """Counts spread over one to sixteen CTAs: a long reservation over the holes, then all of it packed."""
    g = np.random.RandomState(pages % 97)
    B, P = 40, 16
    s = State(B, P, 600, pages)
    s.refs = (g.rand(pages) < 0.4).astype(np.int32)       # held by others: a prefix cache
    s.refs[pages - 7:] = 0
    s.reserve(g.randint(0, 16 * 90, size=B).tolist())
    s.lens = np.maximum(s.held * P - 3, 0).astype(np.int32)
    s.fork(g.randint(0, B, size=B).tolist())
    s.reserve([30] * B)
    s.compact()
    s.reserve([60] * B)
    full = s.refs.copy()
    s.refs[s.refs == 0] = 1
    s.refs[[3 % pages, pages // 2, pages - 1]] = 0        # three pages left, for a row that needs four
    _, missing, err = s.reserve([0, 80] + [0] * (B - 2))
    assert (missing == 0) == (err == 0)
    s.refs = full


FORMATS = [(da.KV_BF16, 3, 64, 16), (da.KV_BF16, 2, 128, 64), (da.KV_BF16, 1, 8, 3), (da.KV_FP8, 2, 128, 8), (da.KV_FP8_BLOCK, 3, 128, 16),
           (da.KV_INT8_BLOCK, 8, 128, 192), (da.KV_MLA656, 1, 576, 16)]


@pytest.mark.parametrize("kv,H,D,P", FORMATS)
def test_copies_of_every_format(kv, H, D, P):
    pages, g = 41, torch.Generator().manual_seed(P)
    latent, blocks = kv == da.KV_MLA656, kv in (da.KV_FP8_BLOCK, da.KV_INT8_BLOCK)
    d = _desc(1, P, 4, pages, H_kv=H, G=128 if latent else 8, D_qk=D, D_v=512 if latent else D, kv_dtype=kv)
    row = 656 if latent else D * (2 if kv == da.KV_BF16 else 1)
    pools = [torch.randint(0, 256, (pages, P, H, row), generator=g).to(torch.uint8) for _ in range(1 if latent else 2)]
    scales = [torch.randn(pages, H, P // 16, generator=g) for _ in range(2)] if blocks else [None, None]
    weights = torch.randn(pages, H, P, generator=g)
    perm = torch.randperm(pages, generator=g)
    pairs = torch.stack([perm[:15], perm[15:30]], 1).int()
    pairs[4, 0], pairs[9] = -1, torch.tensor([-1, -1], dtype=torch.int32)
    bad = torch.tensor([[pages, 0], [1, pages], [2, -1]], dtype=torch.int32)
    for count, with_bad in ((None, False), (7, False), (0, False), (None, True), (99, False)):
        dev = [p.cuda() for p in pools]
        sc = [None if s is None else s.cuda() for s in scales]
        w, err = weights.cuda(), _i32([0])
        c = torch.cat([pairs, bad]) if with_bad else pairs
        da.copy_pages(d, c.cuda(), dev[0], None if latent else dev[1], *sc, weights=w, num_copies=None if count is None else _i32([count]),
                      device_error=err)
        assert int(err) == (da.DA_DEV_BAD_PAGE if with_bad else 0)
        for got, was in zip(dev + sc + [w], pools + scales + [weights]):
            if was is None:
                continue
            want = was.clone()
            for src, dst in pairs[:count].tolist():
                if src >= 0:
                    want[dst] = was[src]
            assert torch.equal(got.cpu(), want)


def test_a_beam_step_captured_and_replayed():
    """fork, reserve, copy as a graph whose two tables take turns, against the same calls without one."""
    B, P, cols, pages, H, D = 8, 16, 20, 200, 2, 64
    d = _desc(B, P, cols, pages, H_kv=H, D_qk=D, D_v=D)
    g = torch.Generator().manual_seed(2)
    parents = torch.randint(0, B, (12, B), generator=g).int().cuda()

    def state():
        table = torch.full((2, B, cols), -1, dtype=torch.int32, device="cuda")
        held, lens, refs = torch.zeros(2, B, dtype=torch.int32, device="cuda"), torch.zeros(2, B, dtype=torch.int32, device="cuda"), _i32([0] * pages)
        copies, missing = _i32([[0, 0]] * B), _i32([0])
        da.reserve_pages(d, lens[0], table[0], held[0], refs, copies, missing, new_tokens=_i32([50] * B))
        lens[0] = 50
        k = torch.randn(pages, P, H, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
        return dict(table=table, held=held, lens=lens, refs=refs, copies=copies, missing=missing, k=k, v=k.clone(), par=_i32([0] * B),
                    err=_i32([0]))

    def step(s, a, b):
        da.fork_pages(d, s["par"], s["lens"][a], s["table"][a], s["held"][a], s["refs"], s["table"][b], s["held"][b], s["lens"][b],
                      device_error=s["err"])
        da.reserve_pages(d, s["lens"][b], s["table"][b], s["held"][b], s["refs"], s["copies"], s["missing"], device_error=s["err"])
        da.copy_pages(d, s["copies"], s["k"], s["v"], device_error=s["err"])
        s["lens"][b].add_(1)
    x, y = state(), state()
    graphs, stream = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph, stream=stream):
            step(x, i, 1 - i)
    for t in range(12):
        x["par"].copy_(parents[t])
        y["par"].copy_(parents[t])
        graphs[t % 2].replay()
        step(y, t % 2, 1 - t % 2)
    torch.cuda.synchronize()
    assert all(torch.equal(x[k], y[k]) for k in x) and int(x["err"]) == 0
