"""Probabilities out of logits: penalties, biases, masks, temperature, against
float64, with bounds derived from the roundings of the fp32 steps."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.serving_ref import adjusted, probs_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(B, K, V, seed, hist=0, bias=0, mask=None, temps=(1.0, 0.7, 0.0), scale=2.5):
    g = np.random.RandomState(seed)
    c = dict(logits=(g.randn(B, K + 1, V) * scale).astype(np.float32), temperature=g.choice(temps, B).astype(np.float32),
             repetition=g.choice([1.0, 1.25, 0.5], B).astype(np.float32), frequency=g.choice([0.0, 0.3, -0.2], B).astype(np.float32),
             presence=g.choice([0.0, 0.6], B).astype(np.float32), history=None, prompt=None, lens=None, drafts=None, bias=None, allowed=None)
    if hist:
        c["history"] = g.randint(0, max(1, min(V, hist // 3 + 1)), (B, hist)).astype(np.int32)
        c["lens"], c["prompt"] = g.randint(0, hist + 1, B).astype(np.int32), g.randint(0, hist + 1, B).astype(np.int32)
    if K:
        c["drafts"] = g.randint(0, V, (B, K)).astype(np.int32)
    if bias:
        n = g.randint(0, bias + 1, B)
        starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        c["bias"] = (starts, g.randint(0, V, starts[-1]).astype(np.int32), (g.randn(starts[-1]) * 3).astype(np.float32))
    if mask is not None:
        c["allowed"] = g.rand(B, K + 1, V) < mask
    return c


def _bits(allowed):
    B, rows, V = allowed.shape
    pad = np.zeros((B, rows, -(-V // 32) * 32), bool)
    pad[..., :V] = allowed
    pad[..., V:] = True                                   # bits past the vocabulary say nothing
    return np.packbits(pad, axis=-1, bitorder="little").view(np.int32)


def _run(c, tin=F32, tout=F32, want_err=0, in_place=False, pad=0):
    """The call on the device against the oracle; returns the probabilities."""
    B, rows, V = c["logits"].shape
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    logits = torch.from_numpy(c["logits"]).to(tin)
    held = logits.float().numpy()
    store = torch.full((B * rows, V + pad), 77.0, dtype=tin, device="cuda")
    li = store[:, pad:].view(B, rows, V) if pad == 0 else torch.as_strided(store, (B, rows, V), (rows * (V + pad), V + pad, 1), pad)
    li.copy_(logits)
    out = li if in_place else torch.full((B, rows, V), 55.0, dtype=tout, device="cuda")
    err = _i32([0])
    da.token_probs(li, out, temperature=dev(c["temperature"]), repetition=dev(c["repetition"]), frequency=dev(c["frequency"]),
                   presence=dev(c["presence"]), history=dev(c["history"]), history_lens=dev(c["lens"]), prompt_lens=dev(c["prompt"]),
                   draft_tokens=dev(c["drafts"]), bias=None if c["bias"] is None else tuple(dev(x) for x in c["bias"]),
                   allowed=None if c["allowed"] is None else dev(_bits(c["allowed"])), device_error=err)
    torch.cuda.synchronize()
    assert int(err) == want_err
    got = out.float().cpu().double().numpy()
    if pad and in_place:
        assert (store[:, :pad] == 77).all()
    eps, tiny = {F32: (2.0 ** -24, 2.0 ** -126), BF16: (2.0 ** -8, 2.0 ** -126), F16: (2.0 ** -11, 2.0 ** -25)}[tout if not in_place else tin]
    for b in range(B):
        n = 0 if c["lens"] is None else min(max(int(c["lens"][b]), 0), c["history"].shape[1])
        text = [] if n == 0 else c["history"][b, :n].tolist()
        bias = []
        if c["bias"] is not None:
            lo, hi = c["bias"][0][b:b + 2]
            bias = list(zip(c["bias"][1][lo:hi].tolist(), c["bias"][2][lo:hi].tolist()))
        for j in range(rows):
            ok = np.ones(V, bool) if c["allowed"] is None else c["allowed"][b, j]
            T = float(c["temperature"][b])
            args = (text, 0 if c["prompt"] is None else int(c["prompt"][b]), [] if c["drafts"] is None else c["drafts"][b].tolist(), j,
                    float(c["repetition"][b]), float(c["frequency"][b]), float(c["presence"][b]), bias, V)
            x64 = adjusted(held[b, j], np.float64, *args)
            if not T > 0:
                want, _ = probs_ref(adjusted(held[b, j], np.float32, *args).astype(np.float64), ok, T)
                assert np.array_equal(got[b, j], want), (b, j)
                continue
            p, d = probs_ref(x64, ok, T)
            if np.isnan(p).any():
                assert np.isnan(got[b, j]).all(), (b, j)
                continue
            # x: the quotient or product, two differences and a product, one sum per bias, each 2^-24 of magnitudes up to `big` (its
            # own logit and x, what is taken off, all biases; an infinite one is exact); the exponent: x - max, its scale and their
            # product, 4 * 2^-24 |x - max| / T; ex2 2 ulp (2^-22) of the value and of two factors; sums of at most 32 groups of eight a
            # thread (32 + 3 additions), 5 + 4 over its CTA, 4 over the cluster. All of it for the token, for the largest, and (averaged over p) for the total.
            said = max([1] + [text.count(t) for t in set(text)])
            mag = np.where(ok & np.isfinite(x64), np.maximum(np.abs(held[b, j].astype(np.float64)), np.abs(x64)), 0.0)
            big = 2 * mag + abs(args[5]) * (said + j) + args[6] + sum(abs(v) for _, v in bias if math.isfinite(v))
            u = 2.0 ** -24
            one = (5 + len(bias)) * u * big / T
            one = one + (p * one).sum() + one[p.argmax()]
            rel = np.where(p > 0, one + 4 * u * (d + (p * d).sum()) / T + 3 * 4 * u + 90 * u, 0.0)
            tol = p * ((1 + rel) * np.exp(np.minimum(rel, 100.0)) * (1 + eps) - 1) + tiny
            assert (np.abs(got[b, j] - p) <= tol).all(), (b, j, np.abs(got[b, j] - p).max())
            assert (got[b, j][~ok] == 0).all()
    return out


@pytest.mark.parametrize("tin", [F32, BF16, F16])
@pytest.mark.parametrize("tout", [F32, BF16, F16])
def test_types_with_everything_at_once(tin, tout):
    _run(_case(5, 2, 1003, 1, hist=300, bias=20, mask=0.5), tin, tout)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 32, 33, 511, 4096, 4097, 8191, 32771])
def test_vocabularies(V):
    _run(_case(4, 1, V, V, hist=40, bias=3, mask=0.7 if V > 1 else None))
    _run(_case(3, 0, V, V + 1), BF16, BF16)


@pytest.mark.parametrize("V,B", [(128259, 1), (128256, 3), (262144, 1), (300007, 1), ((1 << 19) - 7, 1)])
def test_long_rows_take_clusters(V, B):
    _run(_case(B, 1, V, 3, hist=500, bias=5, mask=0.9), BF16, F32)
    _run(_case(1, 0, V, 4), F32, F32)


def test_many_rows():
    _run(_case(40, 3, 16384, 5, hist=100), BF16, BF16)


@pytest.mark.parametrize("tin", [BF16, F32])
def test_many_long_rows_with_long_histories(tin):
    """Rows enough for one CTA each, whose shares stream and list tokens past 2^16; against float64 on the device."""
    B, V, n = 170, 130999, 5000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(B, 1, V, device="cuda", generator=g) * 2.5).to(tin)
    hist = torch.randint(0, V, (B, n), device="cuda", generator=g, dtype=torch.int32)
    lens = torch.randint(0, n + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    prompt = lens // 2
    rep, freq, pres, T = (torch.rand(B, device="cuda", generator=g) + 0.5 for _ in range(4))
    out = torch.empty(B, 1, V, device="cuda")
    da.token_probs(x, out, temperature=T, repetition=rep, frequency=freq, presence=pres, history=hist, history_lens=lens, prompt_lens=prompt)
    i = torch.arange(n, device="cuda")
    there, asked = i < lens[:, None], i < prompt[:, None]
    z = torch.zeros(B, V, dtype=torch.float64, device="cuda")
    said = z.scatter_add(1, hist.long(), (there & ~asked).double())
    seen = z.scatter_add(1, hist.long(), there.double()) > 0
    c = lambda v: v.double()[:, None]  # noqa: E731
    y = x[:, 0].double()
    y = torch.where(seen, torch.where(y > 0, y / c(rep), y * c(rep)), y) - c(freq) * said - torch.where(said > 0, c(pres), 0.0)
    want = torch.softmax(y / c(T), -1)
    # as in _run: 5 roundings of magnitudes up to 60 (counts are small) over T >= 0.5, for the token, the largest and the sum;
    # the exponent's four; 102 more
    rel = 2.0 ** -24 * (3 * 5 * 60 / 0.5 + 8 * 60 / 0.5 + 102)
    assert ((out[:, 0].double() - want).abs() <= want * rel + 2.0 ** -126).all()


def test_streaming_shares_over_and_over():
    """More rows than fit at once, whose pieces go round a ring of few slots: a slot that is filled again before every warp
    has read it shows in some row of some run."""
    B, V, n = 1024, 131072, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(B, 1, V, device="cuda", generator=g) * 2.5).to(BF16)
    hist = (torch.rand(B, n, device="cuda", generator=g) ** 3 * V).int()
    lens = torch.randint(n // 2, n + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    out, first = torch.empty_like(x), None
    for _ in range(25):
        out.fill_(7)
        da.token_probs(x, out, history=hist, history_lens=lens)         # no penalties: the listed tokens keep their logits
        if first is None:
            first = out.clone()
            for lo in range(0, B, 128):
                want = torch.softmax(x[lo:lo + 128].double(), -1)
                # fp32 as in the tests above (magnitudes up to 20, T = 1), then bf16: half a step
                assert ((first[lo:lo + 128].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -24 * (3 * 5 * 40 + 8 * 40 + 102)) + 2.0 ** -126).all()
        assert torch.equal(out, first)


def test_rows_that_start_anywhere_and_results_in_place():
    for pad in (0, 1, 3, 5):
        c = _case(3, 2, 777, 6 + pad, hist=30, mask=0.8)
        for t in (F32, BF16, F16):
            _run(c, t, t, pad=pad)
            _run(c, t, t, pad=pad, in_place=True)
            _run(c, t, F32 if t != F32 else BF16, pad=pad)


def test_history_counts_and_marks():
    """A token thousands of times, in prompt and text both, outside the vocabulary; lengths past the row; long histories
    whose counts take 32 bits."""
    V = 200
    for cols in (3000, 16383, 16384, 40000):
        c = _case(3, 2, V, cols, hist=cols, temps=(1.0,))
        c["history"][0] = 7
        c["history"][1, ::2] = -1
        c["history"][1, 1::4] = V + 5
        c["lens"][:] = [cols, cols + 9, 5]
        c["prompt"][:] = [0, 17, 5000]
        c["frequency"][:] = [0.001, 0.0005, 0.1]
        _run(c)


def test_chains_end_at_a_negative_draft():
    c = _case(4, 5, 60, 8, hist=10, temps=(1.0, 0.5))
    c["drafts"] = np.array([[3, 3, 3, 3, 3], [1, -1, 1, 1, 1], [-1, 2, 2, 2, 2], [59, 60, 0, 1 << 30, 5]], np.int32)
    c["repetition"][:], c["frequency"][:], c["presence"][:] = 1.3, 0.4, 0.2
    _run(c)


def test_one_token_biased_many_times():
    c = _case(2, 0, 100, 9, temps=(1.0,))
    c["bias"] = (np.array([0, 200, 203], np.int32), np.concatenate([np.full(200, 42), [99, -3, 100]]).astype(np.int32),
                 np.concatenate([np.random.RandomState(1).randn(200), [-np.inf, 5.0, 5.0]]).astype(np.float32))
    _run(c)


@pytest.mark.parametrize("V,B,K", [(3000, 3, 1), (60000, 2, 0), (20000, 160, 0)])
def test_more_biases_than_a_list_has_room_for(V, B, K):
    """One request with thousands of biases beside others with few, in every way that a share is held, in place too."""
    c = _case(B, K, V, 17, hist=40, bias=3, mask=0.8, temps=(1.0, 0.7, 0.0))
    g = np.random.RandomState(4)
    starts, toks, vals = c["bias"]
    many = 2500
    c["temperature"][0], c["temperature"][-1] = 0.9, 0.0
    c["bias"] = (np.concatenate([[0], starts[1:] + many]).astype(np.int32), np.concatenate([g.randint(0, V, many), toks]).astype(np.int32),
                 np.concatenate([g.randn(many), vals]).astype(np.float32))
    _run(c)
    _run(c, F32, F32, in_place=True)
    if B < 10:                                            # all of them in the one greedy request
        n = int(c["bias"][0][-1])
        c["bias"] = (np.array([0] * B + [n], np.int32), *c["bias"][1:])
        _run(c, BF16, BF16)


def test_rows_that_nothing_is_left_of():
    c = _case(3, 1, 500, 10, temps=(1.0, 0.0))
    c["temperature"][:] = [1.0, 0.0, 1.0]
    c["allowed"] = np.ones((3, 2, 500), bool)
    c["allowed"][0, 1] = c["allowed"][1, 0] = False
    c["logits"][2, 0] = -np.inf
    out = _run(c, want_err=da.DA_DEV_BAD_PROBS)
    assert (out[0, 1] == 0).all() and (out[1, 0] == 0).all() and (out[2, 0] == 0).all()


def test_masked_places_may_hold_anything():
    c = _case(4, 0, 300, 11)
    c["temperature"][:] = [1.0, 0.0, 1.0, 0.0]
    c["allowed"] = np.random.RandomState(1).rand(4, 1, 300) < 0.6
    for v in (np.nan, np.inf, -np.inf, 3e38):
        c["logits"] = np.where(c["allowed"], c["logits"], v).astype(np.float32)
        _run(c)
    c["logits"] = np.where(c["allowed"], c["logits"], np.finfo(np.float32).min)
    c["allowed"] = None                                   # masks of the type's lowest value, in the logits themselves
    c["logits"][1, 0, :5] = -np.inf
    _run(c)


def test_nan_and_infinity_where_they_count():
    c = _case(4, 0, 5000, 12, temps=(1.0,))
    c["logits"][0, 0, 17], c["logits"][1, 0, 4999], c["logits"][2, 0, 3] = np.nan, np.inf, -np.inf
    c["logits"][3, 0, :100] = np.nan
    c["temperature"][3] = 0.0                             # greedy: the largest number
    out = _run(c)
    assert float(out[3].sum()) == 1


def test_ties_go_to_the_lowest_token():
    for V in (40, 5000, 131072):
        c = _case(3, 0, V, 13, temps=(0.0,))
        c["logits"] = np.zeros((3, 1, V), np.float32)
        c["logits"][1, 0, [V - 1, V // 2, V // 2 + 1]] = 1
        c["logits"][2] = -1
        c["logits"][2, 0, V - 1] = -0.5
        _run(c, BF16, F32)


def test_temperatures_at_the_ends():
    c = _case(5, 0, 1000, 14)
    c["temperature"][:] = [1e-30, 1e-45, 1e30, -1.0, np.nan]
    out = _run({**c, "repetition": np.ones(5, np.float32)})
    assert float(out[0].max()) == 1 and abs(float(out[2].sum()) - 1) < 1e-4


def test_nothing_but_a_softmax():
    x = torch.randn(3, 1, 1000, device="cuda")
    p = torch.empty_like(x)
    da.token_probs(x, p)
    assert torch.allclose(p, torch.softmax(x, -1), rtol=1e-5, atol=0)


def test_with_the_verification_that_draws_from_them():
    """Greedy requests of a chain: the drafts that are the row's largest are accepted, the next token is the next largest."""
    B, K, V = 6, 3, 4099
    c = _case(B, K, V, 15, hist=50, bias=4, mask=0.9, temps=(0.0,))
    rows = []
    for b in range(B):
        best, drafts = [], []
        for j in range(K + 1):
            lo, hi = c["bias"][0][b:b + 2]
            x = adjusted(c["logits"][b, j], np.float32, c["history"][b, :c["lens"][b]].tolist(), int(c["prompt"][b]), drafts, j,
                         c["repetition"][b], c["frequency"][b], c["presence"][b],
                         list(zip(c["bias"][1][lo:hi].tolist(), c["bias"][2][lo:hi].tolist())), V)
            best.append(int(np.argmax(np.where(c["allowed"][b, j], x, -np.inf))))
            if j < K:
                drafts.append(best[j] if j < b % (K + 1) else (best[j] + 1) % V)
        c["drafts"][b] = drafts
        rows.append(best)
    p = _run(c)
    acc, toks = _i32([0] * B), _i32([[0] * (K + 1)] * B)
    da.verify_drafts(p, None, torch.from_numpy(c["drafts"]).cuda(), torch.full((B, K + 1), 0.5, device="cuda"), acc, toks)
    for b in range(B):
        a = min(b % (K + 1), K)
        assert int(acc[b]) == a and toks[b, :a + 1].tolist() == rows[b][:a + 1]


def test_captured_on_another_stream():
    c = _case(8, 1, 3001, 16, hist=64)
    dev = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    out, again = torch.empty(8, 2, 3001, device="cuda"), torch.empty(8, 2, 3001, device="cuda")

    def call(o):
        da.token_probs(dev["logits"], o, temperature=dev["temperature"], repetition=dev["repetition"], frequency=dev["frequency"],
                       presence=dev["presence"], history=dev["history"], history_lens=dev["lens"], prompt_lens=dev["prompt"],
                       draft_tokens=dev["drafts"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call(out)
    for k in range(3):
        dev["logits"].copy_(torch.from_numpy(c["logits"]).cuda().roll(k, 2))
        graph.replay()
        call(again)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and math.isfinite(float(out.sum()))
