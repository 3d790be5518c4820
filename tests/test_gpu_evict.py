"""GPU parity of decode_attn_evict against the oracle: the kept positions, the
lengths, every byte of the pools and every weight are exact, ties, NaN,
infinities and bad pages included."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.ops_ref import evict_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16, FP8, MLA = da.KV_BF16, da.KV_FP8, da.KV_MLA656


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


class Case:
    def __init__(self, kv, H, D, P, lens, budget, first=0, last=0, kind="spread", seed=0, max_pages=None):
        r = np.random.default_rng(seed)
        self.__dict__.update(kv=kv, H=H, D=D, P=P, lens=list(lens), budget=budget, first=first, last=last, B=len(lens))
        self.max_pages = max_pages or max(1, -(-max(max(lens), budget) // P))
        need = [min(self.max_pages, -(-max(0, n) // P)) for n in lens]
        out = [-(-min(max(0, n), budget) // P) for n in lens]
        self.num_pages = sum(need) + sum(out) + 2
        perm = r.permutation(self.num_pages)
        self.table = np.full((self.B, self.max_pages), -1, dtype=np.int32)
        self.into = np.full((self.B, self.max_pages), -1, dtype=np.int32)
        at = 0
        for t, n in ((self.table, need), (self.into, out)):
            for b in range(self.B):
                t[b, :n[b]] = perm[at:at + n[b]]
                at += n[b]
        row = 656 if kv == MLA else D * (2 if kv == BF16 else 1)
        self.pools = [r.integers(0, 256, (self.num_pages, P, H, row), dtype=np.uint8) for _ in range(1 if kv == MLA else 2)]
        n = (self.num_pages, H, P)
        self.weights = {"spread": lambda: np.exp(r.standard_normal(n) * 3 - 5), "zero": lambda: np.zeros(n),
                        "few": lambda: r.integers(0, 4, n) / 4, "fine": lambda: 1 + r.integers(0, 50, n) * 2.0 ** -23,
                        "tied": lambda: 1 + r.integers(0, 400, n) / 2048, "close": lambda: 1 + r.integers(0, 400, n) / 2048 + r.integers(0, 7, n) * 2.0 ** -23,
                        "wild": lambda: r.choice([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-40, -1e-40, 3e38], n),
                        }[kind]().astype(np.float32)

    def desc(self):
        return da.Desc.make(B=self.B, H_kv=self.H, G=8, D_qk=self.D, D_v=512 if self.kv == MLA else self.D, page_size=self.P,
                            max_pages_per_seq=self.max_pages, num_pages=self.num_pages, kv_dtype=self.kv)

    def tensors(self):
        c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        pools = [c(p) for p in self.pools] + [None] * (2 - len(self.pools))
        return dict(lens=torch.tensor(self.lens, dtype=torch.int32, device="cuda"), table=c(self.table), into=c(self.into), k=pools[0],
                    v=pools[1], w=c(self.weights), kept=torch.full((self.B, self.H, self.budget), -7, dtype=torch.int32, device="cuda"),
                    new=torch.full((self.B,), -7, dtype=torch.int32, device="cuda"),
                    err=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def call(self, t, stream=None):
        da.evict(self.desc(), self.budget, t["lens"], t["table"], t["into"], t["k"], t["v"], t["w"], t["kept"], t["new"],
                 keep_first=self.first, keep_last=self.last, device_error=t["err"], stream=stream)

    def check(self, t=None):
        if t is None:
            t = self.tensors()
            self.call(t)
        torch.cuda.synchronize()
        kept, new, pools, weights, err = evict_ref(self.lens, self.table, self.into, self.pools, self.weights, self.budget,
                                                   self.first, self.last)
        assert int(t["err"].item()) == err
        assert t["new"].cpu().numpy().tolist() == new.tolist()
        assert np.array_equal(t["kept"].cpu().numpy(), kept)
        for got, want in zip((t["k"], t["v"]), pools):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(t["w"].cpu().numpy().view(np.uint32), weights.view(np.uint32))


CASES = [
    (BF16, 1, 64, 16, [1], 1), (BF16, 2, 64, 16, [5, 0, 33], 1), (BF16, 3, 96, 8, [40, 7, 100, 64], 24, 2, 5),
    (BF16, 8, 128, 64, [700, 64, 65, 1500], 257, 4, 32), (BF16, 1, 72, 32, [1000], 999, 0, 0), (BF16, 2, 64, 16, [50, 49], 48, 24, 24),
    (BF16, 4, 64, 256, [1537], 512, 0, 512), (FP8, 2, 128, 32, [333, 40], 100, 1, 3), (FP8, 1, 16, 8, [90], 17, 0, 1),
    (FP8, 5, 48, 64, [1100, 3], 300, 10, 0), (MLA, 1, 576, 64, [400, 129], 130, 1, 16), (MLA, 1, 576, 192, [600], 77, 0, 7),
]


@pytest.mark.parametrize("kind", ["spread", "zero", "few", "fine", "wild"])
@pytest.mark.parametrize("case", CASES)
def test_evict(case, kind):
    Case(*case, kind=kind, seed=len(kind) + case[2] + case[5]).check()


@pytest.mark.parametrize("kind", ["spread", "zero", "wild"])
@pytest.mark.parametrize("lens,P", [([9000], 64), ([20000, 500], 32), ([70001], 64), ([40961 + 7, 8193], 256)])
def test_long_rows_are_shared_by_a_cluster(lens, P, kind):
    """Lengths at which two, four, eight and sixteen CTAs select together, one request far shorter than the table allows."""
    Case(MLA, 1, 576, P, lens, 2003, 3, 64, kind=kind, seed=len(lens) + P).check()


@pytest.mark.parametrize("kind", ["tied", "close"])
@pytest.mark.parametrize("lens", [[20000], [80000], [100001, 60000], [8000]])
def test_the_last_kept_among_a_few_near_equals(lens, kind):
    """About 20 to 250 tokens of a row share the upper bits of the last weight kept, in one CTA and over clusters."""
    Case(MLA, 1, 576, 64, lens, 3011, 2, 17, kind=kind, seed=len(lens)).check()


@pytest.mark.parametrize("near", [1, 2, 255, 256, 257, 300])
@pytest.mark.parametrize("n", [1200, 21000])
def test_counts_of_near_equals_about_what_is_compared_directly(n, near):
    c = Case(BF16, 1, 64, 64, [n], 600, 0, 0, seed=near + n)
    w = np.zeros(n, np.float32)
    r = np.random.default_rng(near)
    order = r.permutation(n)
    w[order[:near]] = 1 + r.integers(0, 60, near) * np.float32(2.0 ** -23)       # one 20-bit prefix
    w[order[near:near + 600 - (near + 1) // 2]] = 2 + r.random(600 - (near + 1) // 2)   # and the budget ends among them
    for t in range(n):
        c.weights[c.table[0, t // 64], 0, t % 64] = w[t]
    c.check()


def test_a_share_beyond_shared_memory():
    """Many rows, so that one CTA selects from each, and a row longer than the keys that it holds."""
    lens = [50] * 80 + [45000]
    Case(FP8, 1, 16, 64, lens, 1500, 1, 9, seed=5).check()


def test_bad_pages_and_lengths():
    c = Case(BF16, 2, 64, 16, [100, 60, 30, 200, 90], 40, 2, 3, seed=7)
    c.table[0, 2], c.table[1, 3], c.into[2, 1], c.into[4, 0] = -1, c.num_pages, c.num_pages + 5, -9
    c.lens[3] = -5
    c.check()
    c = Case(BF16, 1, 64, 16, [64, 64], 20, seed=8)
    c.lens[1] = 1 << 30                                    # clamped to the table's 4 pages
    c.check()
    c = Case(BF16, 1, 64, 16, [100], 90, seed=9)
    c.table[0, :] = -1                                     # nothing can be read: everything weighs the same
    c.check()


def test_the_other_tokens_of_a_shared_page_stay():
    """Slots of the last new page past the length, and all other pages, keep their bytes (checked by the oracle's
    copies); a request of length 0 writes nothing at all."""
    c = Case(BF16, 2, 128, 64, [0, 0], 5, seed=11)
    c.check()


def test_odd_pages_and_many_heads():
    """Pages of any size, and as many heads as the library takes (one token a copy tile)."""
    Case(BF16, 2, 64, 3, [50, 7, 31], 11, 1, 2, seed=20).check()
    Case(FP8, 3, 16, 7, [300], 123, seed=21).check()
    Case(BF16, 4096, 8, 2, [5, 3], 3, 1, 1, seed=22).check()


def test_first_call_of_a_process_in_a_capture():
    """The first call in a process asks the device what clusters it holds; that happens inside a capture too."""
    code = """
import torch
import test_gpu_evict as m
c = m.Case(m.MLA, 1, 576, 64, [70001], 2003, 3, 64, seed=5)
t = c.tensors()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.call(t)
g.replay()
c.check(t)
print("same")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_captured_replayed_other_stream_and_repeated():
    c = Case(BF16, 4, 64, 16, [300, 20, 150], 64, 2, 8, seed=12)
    t = c.tensors()
    c.call(t, stream=torch.cuda.Stream())
    c.check(t)
    t = c.tensors()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(t)
    graph.replay()
    graph.replay()                                         # the old pages are only read: the same again
    c.check(t)
    c = Case(MLA, 1, 576, 64, [30000], 4000, 2, 8, seed=13)
    a, b = c.tensors(), c.tensors()
    for _ in range(5):
        c.call(a)
        c.call(b)
    c.check(a)
    c.check(b)
