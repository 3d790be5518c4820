"""GPU parity of decode_attn_verify_drafts against the oracle: accepted counts,
tokens, lengths and error bits are exact (the oracle's sums are Python
integers)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.ops_ref import verify_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


class Case:
    def __init__(self, B, K, V, dtype=torch.float32, q=True, seed=0, peak=2.5, mix=0.3, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.K, self.V, self.dtype, self.pad = B, K, V, dtype, pad

        def probs(n):
            return torch.softmax(torch.randn(B, n, V, generator=g) * peak, -1)
        p = probs(K + 1)
        self.u = torch.rand(B, K + 1, generator=g)
        self.tokens, self.q = torch.zeros(B, K, dtype=torch.int32), None
        if K:
            d = (1 - mix) * p[:, :K] + mix * probs(K)
            self.tokens = torch.multinomial(d.reshape(B * K, V), 1, generator=g).view(B, K).int()
            self.q = d.to(dtype) if q else None
        self.p = p.to(dtype)
        self.lens = torch.randint(K + 1, 1000, (B,), generator=g).int()

    def tensors(self):
        def wide(t):        # rows further apart than the vocabulary
            if t is None:
                return None
            w = torch.full(t.shape[:2] + (self.V + self.pad,), math.nan, dtype=t.dtype)
            w[..., :self.V] = t
            return w.cuda()[..., :self.V]
        e = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(p=wide(self.p), q=wide(self.q), x=self.tokens.cuda() if self.K else None, u=self.u.cuda(), a=e(self.B),
                    out=e(self.B, self.K + 1), lens=self.lens.cuda(), new=e(self.B),
                    err=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def call(self, t, stream=None):
        da.verify_drafts(t["p"], t["q"], t["x"], t["u"], t["a"], t["out"], cache_seqlens=t["lens"], new_seqlens=t["new"],
                         device_error=t["err"], stream=stream)

    def check(self, t=None):
        if t is None:
            t = self.tensors()
            self.call(t)
        torch.cuda.synchronize()
        p, q, err = self.p.float().numpy(), None if self.q is None else self.q.float().numpy(), 0
        for b in range(self.B):
            a, out, e = verify_ref(p[b], None if q is None else q[b], self.tokens[b].tolist(), self.u[b].numpy(), self.V)
            err |= e
            assert int(t["a"][b]) == a and t["out"][b].tolist() == out, b
            assert int(t["new"][b]) == int(self.lens[b]) - self.K + a
        assert int(t["err"].item()) == err
        return t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,K,V,q,pad", [
    (1, 0, 1, True, 0), (3, 1, 2, True, 0), (2, 3, 31, False, 5), (5, 2, 1000, True, 0), (4, 3, 1023, True, 3), (2, 1, 1025, False, 0),
    (3, 7, 4097, True, 1), (1, 3, 32000, True, 0), (1, 2, 100003, True, 0), (6, 0, 9001, True, 7), (40, 1, 16385, True, 0),
])
def test_verify(B, K, V, q, pad, dtype):
    Case(B, K, V, dtype, q, seed=B + K + V, pad=pad).check()


def test_long_chains():
    c = Case(3, 63, 50, seed=1, mix=0.02)
    c.check()
    c.u[0, :63] = 0.0                                    # everything with a probability is accepted
    t = c.check()
    assert int(t["a"][0]) == 63
    c = Case(3, 33, 40, seed=2)
    c.u[:, :33] = 0.0
    c.u[1, 32] = 1.0                                     # refused at the first draft of the upper half, or accepted by p > q
    c.check()


def test_ragged_chains_and_bad_tokens():
    c = Case(6, 4, 300, seed=3, mix=0.0)
    c.u[:, :4] = 0.0
    c.tokens[0, 0], c.tokens[1, 2], c.tokens[2, 3], c.tokens[3, 1], c.tokens[4, 0] = -1, -5, -1, 300, 1 << 30
    t = c.check()
    assert t["a"].tolist() == [0, 2, 3, 1, 0, 4] and int(t["err"].item()) == da.DA_DEV_BAD_TOKEN


def test_random_numbers_at_the_ends():
    for V in (70, 5000):
        for u in (0.0, -1.0, math.nan, 1.0, 5.0, float(np.nextafter(np.float32(1), np.float32(0))), 2.0 ** -24, 1e-30, 1e-42):
            c = Case(4, 1, V, seed=4)
            c.u[:, 1] = u
            c.u[:2, 0] = 1.0                             # refused unless p > q
            c.p[:, :, 0] = 1e-20                         # less than a step
            c.p[3, :, 60:] = 0                           # a tail without weight
            c.check()


def test_probabilities_that_are_none():
    c = Case(8, 1, 2500, seed=5, q=True)
    c.u[:, 0] = 0.9999
    c.p[0, :, ::7] = math.nan
    c.p[1, :, 100:200] = -0.5
    c.p[2, :, 2400] = math.inf                           # counts as 1
    c.p[3] = 0.0                                         # nothing to draw from
    c.p[4] = math.nan
    c.p[5, 0, :] = c.q[5, 0, :] * 0.5                    # refused, and nothing of p - q is left: drawn from p
    c.p[6, 0, int(c.tokens[6, 0])] = math.nan            # a comparison with NaN refuses
    c.q[7, 0, int(c.tokens[7, 0])] = math.nan
    t = c.check()
    assert t["out"][3].tolist() == [-1, -1] and int(t["err"].item()) == da.DA_DEV_BAD_PROBS
    c = Case(3, 1, 2500, seed=6, q=False)
    c.p[:] = 0
    c.p[0, 0, int(c.tokens[0, 0])] = 1e-3                # a certain draft refused, all weight on it: drawn from p
    c.u[:, 0] = 0.5
    c.check()


def test_sums_that_only_whole_steps_tell_apart():
    """Flat and nearly flat rows, where an fp32 running sum of 2^17 entries would be off by whole tokens."""
    V = 1 << 17
    c = Case(3, 0, V, seed=7)
    c.p[0] = 1.0 / V
    c.p[1] = 3e-6
    c.p[2, 0] = torch.from_numpy((np.arange(V) % 5 + 1).astype(np.float32) * np.float32(1.7e-6))
    for u in (0.1, 0.5, 0.875, 0.99999):
        c.u[:] = u
        c.check()


def test_every_share_of_a_cluster_is_reached():
    for V, B in ((100000, 1), (40000, 2), (20000, 30), (70000, 60)):
        c = Case(B, 0, V, seed=V)
        c.u[:, 0] = (torch.arange(B).float() + 0.5) / B
        c.check()
        c.p[:] = 0
        for b in range(B):                               # all weight on one entry, somewhere
            c.p[b, 0, (V - 1) * b // max(1, B - 1)] = 1e-9
        c.check()


def test_largest_vocabulary():
    c = Case(1, 1, (1 << 20) - 1, seed=8)
    c.check()
    c.p[:] = 1.0                                         # sums as large as they get
    c.u[:, 1] = 0.75
    c.check()


def test_lengths_in_place_and_left_out():
    c = Case(5, 2, 600, seed=9)
    t = c.tensors()
    da.verify_drafts(t["p"], t["q"], t["x"], t["u"], t["a"], t["out"], cache_seqlens=t["lens"], new_seqlens=t["lens"])
    assert torch.equal(t["lens"], (c.lens.cuda() - 2 + t["a"]))
    t2 = c.tensors()
    da.verify_drafts(t2["p"], t2["q"], t2["x"], t2["u"], t2["a"], t2["out"])
    assert torch.equal(t2["out"], t["out"]) and (t2["new"] == -7).all()
    none = torch.empty(5, 0, 600, device="cuda")           # no drafts: their tensors may be empty ones
    one = (t["p"][:, :1].contiguous(), none, torch.empty(5, 0, dtype=torch.int32, device="cuda"), t["u"][:, :1].contiguous())
    a, b = [torch.full((5, 1), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    da.verify_drafts(*one, t2["a"], a)
    da.verify_drafts(one[0], None, None, one[3], t2["a"], b)
    assert torch.equal(a, b) and (a >= 0).all() and (t2["a"] == 0).all()
    with pytest.raises(da.DecodeAttnError):
        da.verify_drafts(t["p"].double(), t["q"], t["x"], t["u"], t["a"], t["out"])
    with pytest.raises(da.DecodeAttnError):
        da.verify_drafts(t["p"], t["q"].half(), t["x"], t["u"], t["a"], t["out"])
    with pytest.raises(da.DecodeAttnError):
        da.verify_drafts(t["p"].transpose(0, 1).contiguous().transpose(0, 1), t["q"], t["x"], t["u"], t["a"], t["out"])


def test_refuses_rows_that_are_not_there():
    """Expanded probabilities (stride 0) are not packed ones; a single row may be any."""
    c = Case(3, 2, 50, seed=11)
    t = c.tensors()
    for name, bad in (("p", t["p"][:1].expand(3, 3, 50)), ("p", t["p"][:, :1].expand(3, 3, 50)), ("q", t["q"][:1, :1].expand(3, 2, 50)),
                      ("p", t["p"][:, :, :1].expand(3, 3, 50)), ("q", t["q"][0]), ("x", t["x"][:1].expand(3, 2)),
                      ("u", t["u"].double()), ("a", t["a"].long())):
        with pytest.raises(da.DecodeAttnError):
            c.call({**t, name: bad})
    one = Case(1, 0, 50, seed=12)
    o = one.tensors()
    o["p"] = torch.cat([o["p"], o["p"]], 2)[:, :, :50]
    one.call(o)
    one.check(o)


def test_captured_replayed_and_on_another_stream():
    c = Case(4, 3, 30000, seed=10)
    t = c.tensors()
    c.call(t, stream=torch.cuda.Stream())
    c.check(t)
    t = c.tensors()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(t)
    graph.replay()
    c.check(t)
    t["u"].copy_(torch.rand(4, 4, device="cuda"))        # other numbers, the same graph
    c.u = t["u"].cpu()
    graph.replay()
    c.check(t)
