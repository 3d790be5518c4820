"""GPU parity of decode_attn_accum_weights against the float64 oracle.

Tolerance of a weight: the new terms e_i = exp(s_i - lse) have relative error
at most d_i = A_i (D / 16 + 2) 2^-22 + (A_i + |lse|) 2^-22 + 2^-21, A_i = sigma
sum |q||k|: D / 16 fp32 accumulations of a warp MMA (each within an ulp of the
largest partial, 2^-22 of A_i at most with truncation), the products and the
roundings of the exponent (score and lse scaled by log2 e, one fused
multiply-add: four roundings of at most 2^-24 of their values), and exp2
within 2 ulp. The sum of n = G s_q terms and the old weight rounds n + 2 times:
(n + 2) 2^-24 of the result. sum e_i A_i and sum e_i |lse| come from the oracle."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.ops_ref import accum_ref
from workloads import KV_BF16, KV_FP8, KV_MLA656, WorkloadSpec, make_workload

from gpu_util import DeviceWorkload, ensure_built, make_desc, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _spec(kv, B, H_kv, D, P, lens, s_q=1, splits=0, seed=0):
    if kv == KV_MLA656:
        return WorkloadSpec(name="t", B=B, H_kv=1, G=128, D_qk=576, D_v=512, page_size=P, kv_dtype=kv, lengths=lens,
                            splits=splits, seed=seed, s_q=s_q, extra_pages=2)
    return WorkloadSpec(name="t", B=B, H_kv=H_kv, G=8, D_qk=D, D_v=D, page_size=P, kv_dtype=kv, lengths=lens, splits=splits,
                        seed=seed, s_q=s_q, extra_pages=2)


class Step:
    """A decode step on a workload: its attention call, then the accumulation."""

    def __init__(self, spec, accepted=None, weighted=None, decay=1.0, nan_fresh=True):
        self.w, self.s = make_workload(spec), spec
        self.accepted, self.weighted, self.decay = accepted, weighted, decay
        g = torch.Generator().manual_seed(spec.seed + 1)
        self.weights = torch.rand(self.w.num_pages, spec.H_kv, spec.page_size, generator=g)
        wl = self.w.lengths if weighted is None else weighted
        if nan_fresh:                       # what a slot without a weight holds does not matter
            for b, L in enumerate(self.w.lengths):
                for t in range(max(0, wl[b]), L):
                    self.weights[self.w.block_table[b, t // spec.page_size], :, t % spec.page_size] = math.nan
        self.dw = DeviceWorkload(self.w)
        self.out, self.lse, self.meta, self.desc = run(self.w, dw=self.dw)

    def run(self, weights=None, stream=None):
        d = self.dw
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        weights = self.weights.cuda() if weights is None else weights
        da.accum_weights(self.desc, d.q, d.k_pool, d.k_scale, d.block_table, d.cache_seqlens, self.meta, self.lse, weights,
                         num_accepted=i32(self.accepted), weighted_lens=i32(self.weighted), decay=self.decay, stream=stream)
        torch.cuda.synchronize()
        return weights

    def check(self, got):
        w, s = self.w, self.s
        P, H, D, s_q = s.page_size, s.H_kv, s.D_qk, s.s_q
        G = s.G
        if s.kv_dtype == KV_MLA656:       # NoPE as the attention kernel has it: bf16(fp32(e4m3) * scale)
            scale = w.k_pool[..., 512:528].contiguous().view(torch.float32).repeat_interleave(128, -1)
            nope = (w.k_pool[..., :512].view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16).float()
            kp = torch.cat([nope, w.k_pool[..., 528:].contiguous().view(torch.bfloat16).float()], -1)
        else:
            kp = w.k_pool.float() if w.k_scale is None else w.k_pool.view(torch.float8_e4m3fn).float() * w.k_scale.view(H, 1)

        def k_of(b):
            L = w.lengths[b]
            pages = w.block_table[b, :-(-L // P)].long()
            return kp[pages].reshape(-1, H, D)[:L].double().numpy()
        lse = self.lse.cpu().double().numpy().reshape(s.B, s_q, H, G)
        q = w.q.double().numpy().reshape(s.B, s_q, H, G, D)
        add, mag = accum_ref(q, k_of, w.lengths, lse, w.softmax_scale, s_q, self.accepted)
        want, tol = self.weights.double().clone(), torch.zeros(got.shape, dtype=torch.float64)
        wl = w.lengths if self.weighted is None else self.weighted
        for b, L in enumerate(w.lengths):
            for t in range(L):
                at = (w.block_table[b, t // P].long(), slice(None), t % P)
                old = want[at] * float(np.float32(self.decay)) if t < wl[b] else torch.zeros(H, dtype=torch.float64)
                want[at] = old + torch.from_numpy(add[b][t])
                tol[at] = torch.from_numpy(mag[b][t] * (D / 16 + 3) * 2.0 ** -22 + add[b][t] * 2.0 ** -21) + \
                    want[at].abs() * (G * s_q + 2) * 2.0 ** -24
        off = (got.cpu().double() - want).abs()
        keep = torch.isnan(want)             # stale NaN in slots that are not a token's stays there
        assert torch.equal(torch.isnan(got.cpu()), keep)
        assert (off[~keep] <= tol[~keep]).all(), (off - tol)[~keep].max()
        return want


CASES = [
    # kv, B, H_kv, D, P, lens, s_q, splits
    (KV_BF16, 1, 1, 64, 16, [1], 1, 0),
    (KV_BF16, 4, 2, 128, 8, [0, 1, 7, 250], 1, 0),
    (KV_BF16, 3, 1, 64, 256, [700, 65, 64], 1, 8),
    (KV_BF16, 5, 3, 128, 64, [63, 64, 65, 1000, 16], 2, 0),
    (KV_BF16, 4, 2, 64, 32, [3, 1, 2, 500], 3, 0),
    (KV_BF16, 3, 2, 128, 16, [2, 333, 40], 4, 3),
    (KV_BF16, 2, 8, 128, 192, [385, 100], 1, 1),
    (KV_FP8, 4, 2, 128, 32, [0, 1, 95, 1029], 1, 0),
    (KV_FP8, 3, 4, 128, 8, [33, 600, 17], 2, 2),
    (KV_FP8, 2, 1, 128, 64, [129, 1], 4, 0),
    (KV_FP8, 70, 1, 128, 16, [(37 * i) % 150 for i in range(70)], 3, 0),
    (KV_MLA656, 1, 1, 576, 64, [1], 1, 0),
    (KV_MLA656, 4, 1, 576, 16, [0, 1, 31, 300], 1, 0),
    (KV_MLA656, 3, 1, 576, 8, [33, 97, 5], 2, 3),
    (KV_MLA656, 2, 1, 576, 192, [200, 64], 4, 1),
    (KV_MLA656, 1, 1, 576, 64, [2500], 1, 1),            # several units of a cache to a CTA, one of them ragged
    (KV_MLA656, 2, 1, 576, 32, [1301, 770], 3, 1),       # and a pass for each query token
    (KV_MLA656, 40, 1, 576, 16, [(53 * i) % 300 for i in range(40)], 1, 8),   # several parts to a CTA
    (KV_MLA656, 100, 1, 576, 8, [(29 * i) % 140 for i in range(100)], 2, 0),  # several requests to a part
    (KV_BF16, 3, 4, 64, 192, [385, 100, 1], 1, 0),       # two heads to a CTA
    (KV_BF16, 3, 3, 64, 16, [85, 0, 230], 1, 0),         # an odd number of them
    (KV_FP8, 2, 3, 128, 16, [200, 77], 1, 2),
    (KV_BF16, 40, 6, 64, 8, [(53 * i) % 300 for i in range(40)], 1, 8),
    (KV_FP8, 40, 4, 128, 64, [(71 * i) % 500 for i in range(40)], 1, 5),
]


@pytest.mark.parametrize("case", CASES)
def test_accum(case):
    kv, B, H, D, P, lens, s_q, splits = case
    s = Step(_spec(kv, B, H, D, P, lens, s_q, splits, seed=B + D + P))
    s.check(s.run())
    assert da.get_error(s.meta) == 0


@pytest.mark.parametrize("kv", [KV_BF16, KV_FP8, KV_MLA656])
def test_accepted_rows_fresh_tokens_and_decay(kv):
    lens = [100, 3, 0, 64, 513, 2] if kv != KV_MLA656 else [100, 3, 0, 64, 65, 2]
    G = 128 if kv == KV_MLA656 else 8
    for decay in (1.0, 0.5, 0.0):
        s = Step(_spec(kv, 6, 2, 128, 16, lens, 4, 0, seed=21), accepted=[0, 3, 1, -1, 2, 60], weighted=[96, 0, 5, 64, 1000, -2],
                 decay=decay)
        s.check(s.run())
    # rows sum to the query rows that count: G heads each, over the tokens that they see (their lse is within 2^-18)
    s = Step(_spec(kv, 2, 1, 128, 16, [90, 40], 2, 0, seed=22), accepted=[0, 1], weighted=[0, 0])
    s.weights.zero_()
    w = s.run().cpu().double()
    for b, n in ((0, G), (1, 2 * G)):
        total = sum(float(w[s.w.block_table[b, t // 16], 0, t % 16]) for t in range(s.w.lengths[b]))
        assert abs(total - n) < 1e-3 * G / 8


def test_repeats_are_bitwise_equal_and_any_split_gives_the_same():
    for kv in (KV_BF16, KV_FP8, KV_MLA656):
        _repeats(kv)


def _repeats(kv):
    base = None
    for splits in (0, 1, 5):
        s = Step(_spec(kv, 4, 2, 128, 32, [77, 300, 1, 640], 2, splits, seed=31))
        if base is not None:
            s.lse = base.lse
        a, b = s.run(), s.run()
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
        if base is None:
            base, first = s, a
        assert torch.equal(a.view(torch.int32), first.view(torch.int32))


@pytest.mark.parametrize("kv", [KV_BF16, KV_MLA656])
def test_bad_page_long_length_and_foreign_meta(kv):
    s = Step(_spec(kv, 3, 2, 128, 16, [100, 50, 20], 1, 0, seed=41))
    good = s.run().cpu()
    bad = s.dw.block_table.clone()
    bad[0, 2], bad[1, 1] = -1, s.w.num_pages
    keep, s.dw.block_table = s.dw.block_table, bad
    got = s.run().cpu()
    assert da.get_error(s.meta) & da.DA_DEV_BAD_PAGE
    for b, j in ((0, 2), (1, 1)):            # those pages are not touched, the others come out as before
        page = int(keep[b, j])
        assert torch.equal(got[page], s.weights[page])
        got[page] = good[page]
    assert torch.equal(got, good)
    s.dw.block_table = keep
    other = da.Desc.make(**{**{n: getattr(s.desc, n) for n, _ in s.desc._fields_}, "softmax_scale": 0.0, "s_q": 2})
    meta = torch.empty(da.sched_meta_bytes(other), dtype=torch.uint8, device="cuda")
    da.sched_meta(other, s.dw.cache_seqlens, meta)
    s.meta = torch.cat([meta, torch.zeros(max(0, da.sched_meta_bytes(s.desc) - meta.numel()), dtype=torch.uint8, device="cuda")])
    got = s.run().cpu()
    assert torch.equal(got.view(torch.int32), s.weights.view(torch.int32))
    assert da.get_error(s.meta) & da.DA_DEV_META_MISMATCH


def test_nan_key_poisons_its_request_and_head_only():
    s = Step(_spec(KV_BF16, 2, 2, 64, 16, [40, 40], 1, 0, seed=51))
    page = int(s.w.block_table[0, 1])
    s.dw.k_pool[page, 3, 1, 5] = math.nan
    s.out, s.lse, s.meta, s.desc = run(s.w, dw=s.dw)
    got = s.run().cpu()
    for b in range(2):
        for t in range(40):
            v = got[int(s.w.block_table[b, t // 16]), :, t % 16]
            assert torch.isnan(v[1]).item() == (b == 0) and not torch.isnan(v[0]).item()


@pytest.mark.parametrize("kv,H,s_q", [(KV_BF16, 2, 1), (KV_FP8, 2, 1), (KV_BF16, 1, 3), (KV_MLA656, 1, 2)])
def test_rows_without_a_sum(kv, H, s_q):
    """An lse of -inf (nothing was seen) or +inf adds nothing, NaN poisons its KV head's weights and no other's."""
    s = Step(_spec(kv, 2, H, 128 if kv == KV_FP8 else 64, 16, [70, 45], s_q, 0, seed=71))
    s.lse[0, ..., 3], s.lse[0, ..., 6], s.lse[1, ..., :8] = -math.inf, math.inf, -math.inf
    s.check(s.run())
    if H > 1:
        s.lse[0, ..., 9] = math.nan
        got = s.run().cpu()
        for t in range(70):
            v = got[int(s.w.block_table[0, t // 16]), :, t % 16]
            assert torch.isnan(v[1]) and not torch.isnan(v[0])


def test_captured_replayed_and_on_another_stream():
    for kv in (KV_FP8, KV_MLA656):
        _captured(kv)


def _captured(kv):
    s = Step(_spec(kv, 3, 2, 128, 32, [200, 31, 90], 1, 0, seed=61), decay=0.5, weighted=[199, 30, 89])
    want = s.run()
    assert torch.equal(s.run(stream=torch.cuda.Stream()), want)
    wl = torch.tensor(s.weighted, dtype=torch.int32, device="cuda")
    weights, d = s.weights.cuda(), s.dw
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.accum_weights(s.desc, d.q, d.k_pool, d.k_scale, d.block_table, d.cache_seqlens, s.meta, s.lse, weights,
                         weighted_lens=wl, decay=0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(weights.view(torch.int32), want.view(torch.int32))


def test_calls_at_once_on_three_streams():
    """Accumulations of three formats at the same time, with the attention calls of the same steps between them."""
    steps = [Step(_spec(kv, 3, 2, 128, 32, [900, 31, 2000], 2, 0, seed=81 + kv)) for kv in (KV_BF16, KV_FP8, KV_MLA656)]
    want = [s.run() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    got = [s.weights.cuda() for s in steps]
    out, lse = [torch.empty_like(s.out) for s in steps], [torch.empty_like(s.lse) for s in steps]
    torch.cuda.synchronize()
    for rep in range(4):
        for s, st, w, o, l in zip(steps, streams, got, out, lse):
            d = s.dw
            with torch.cuda.stream(st):
                da.fwd(s.desc, d.q, d.k_pool, d.v_pool, d.k_scale, d.v_scale, d.block_table, d.cache_seqlens, s.meta, o, l)
                w.copy_(s.weights.cuda())
                da.accum_weights(s.desc, d.q, d.k_pool, d.k_scale, d.block_table, d.cache_seqlens, s.meta, l, w)
    torch.cuda.synchronize()
    for s, g, w, l in zip(steps, got, want, lse):
        assert torch.equal(l, s.lse) and torch.equal(g.view(torch.int32), w.view(torch.int32))
        assert da.get_error(s.meta) == 0
