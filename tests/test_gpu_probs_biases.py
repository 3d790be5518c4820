"""Token probabilities of requests with very many biases: one or several on every
token, in the list's order, in every way that a row is held; with histories,
drafts and masks, in place, greedy."""
import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _dev(x, t=None):
    x = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return x if t is None else x.to(t)


def _check(x, tokens, values, tin=F32, hist=None, drafts=None, allowed=None, T=None, in_place=False):
    """x float32 [B, rows, V] (held in tin); tokens, values: lists of arrays, one per request. The biases are added in fp32 in their
    order (numpy's unbuffered add), so that what is left to bound is the exponentials and the sums."""
    B, rows, V = x.shape
    starts = np.concatenate([[0], np.cumsum([len(t) for t in tokens])]).astype(np.int32)
    toks, vals = np.concatenate(tokens).astype(np.int32), np.concatenate(values).astype(np.float32)
    rules = dict(bias=(_dev(starts), _dev(toks), _dev(vals)))
    freq = np.full(B, 0.25, np.float32)
    rep = np.full(B, 2.0, np.float32)                     # exact in fp32
    if hist is not None:
        rules.update(history=_dev(hist.astype(np.int32)), history_lens=_dev(np.full(B, hist.shape[1], np.int32)),
                     prompt_lens=_dev(np.full(B, hist.shape[1] // 2, np.int32)))
    if hist is not None or drafts is not None:
        rules.update(frequency=_dev(freq), repetition=_dev(rep))
    if drafts is not None:
        rules.update(draft_tokens=_dev(drafts.astype(np.int32)))
    if allowed is not None:
        pad = np.zeros((B, rows, -(-V // 32) * 32), bool)
        pad[..., :V] = allowed
        rules.update(allowed=_dev(np.packbits(pad, axis=-1, bitorder="little").view(np.int32)))
    if T is not None:
        rules.update(temperature=_dev(np.asarray(T, np.float32)))
    logits = _dev(x, tin)
    held = logits.float().cpu().numpy()
    out = logits if in_place else torch.empty(B, rows, V, dtype=F32, device="cuda")
    err = _dev(np.zeros(1, np.int32))
    da.token_probs(logits, out, device_error=err, **rules)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = out.double().cpu().numpy()
    eps = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[out.dtype]
    for b in range(B):
        for j in range(rows):
            y = held[b, j].copy()
            if hist is not None or drafts is not None:
                said = np.zeros(V, np.float32)
                seen = np.zeros(V, bool)
                if hist is not None:
                    half = hist.shape[1] // 2
                    np.add.at(said, hist[b, half:], 1)
                    seen[hist[b, :half]] = True
                if drafts is not None:
                    np.add.at(said, drafts[b, :j], 1)
                seen |= said > 0
                y = np.where(seen, np.where(y > 0, y / np.float32(2), y * np.float32(2)), y) - freq[b] * said
            ok = (tokens[b] >= 0) & (tokens[b] < V)
            np.add.at(y, tokens[b][ok], values[b][ok].astype(np.float32))
            y = y.astype(np.float64)
            if allowed is not None:
                y[~allowed[b, j]] = -np.inf
            t = 1.0 if T is None else float(T[b])
            if t == 0:
                want = np.zeros(V)
                want[y.argmax()] = 1
                assert np.array_equal(got[b, j], want)
                continue
            d = np.where(np.isneginf(y), 0.0, y.max() - y) / t
            p = np.exp(-d) * ~np.isneginf(y)
            p /= p.sum()
            # the exponent: x - max, its scale and their product, 4 u d, for the token and (averaged) for the total; ex2 2 ulp of the
            # value, of the correction of a part's sum and of log2's; a thread's values one behind the other (listed ones too), then 13
            u = 2.0 ** -24
            rel = 4 * u * (d + (p * d).sum()) + 12 * u + (-(-V // 512) + 16) * u
            assert (np.abs(got[b, j] - p) <= p * ((1 + rel) * (1 + eps) - 1) + 2.0 ** -126).all(), (b, j)
    return out


@pytest.mark.parametrize("tin", [F32, BF16])
@pytest.mark.parametrize("V,B", [(1500, 2), (5000, 3), (16001, 2), (70001, 1), (131072, 2), (20000, 170)])
def test_a_bias_on_every_token(V, B, tin):
    g = np.random.RandomState(V)
    x = (g.randn(B, 1, V) * 2.5).astype(np.float32)
    tokens, values = [g.permutation(V) for _ in range(B)], [g.randn(V) * 3 for _ in range(B)]
    _check(x, tokens, values, tin)


@pytest.mark.parametrize("V", [1500, 9000, 40000, 131072, (1 << 19) - 7])
def test_several_on_a_token_in_their_order(V):
    """Millions up and down: another order leaves other rounding errors, of 0.1 and more."""
    g = np.random.RandomState(V % 1000)
    n = 5 * V // 2
    half = g.randint(0, V, n // 2)
    big = (g.rand(n // 2) * 4e6).astype(np.float32)
    tokens, values = np.concatenate([half, half[::-1]]), np.concatenate([big, -big[::-1]])
    at = g.permutation(len(tokens) - len(tokens) // 3) + len(tokens) // 3          # some in pairs' order, the rest anywhere
    tokens[len(tokens) // 3:], values[len(tokens) // 3:] = tokens[at], values[at]
    x = (g.randn(1, 1, V) * 2).astype(np.float32)
    _check(x, [tokens], [values])


@pytest.mark.parametrize("V,B,in_place", [(131072, 180, False), (131072, 160, True), (250043, 104, True)])
def test_shares_with_more_touched_tokens_than_16_bits_count(V, B, in_place):
    """One or two CTAs a row; a few requests with a bias on nearly every token, beside some with few and none."""
    g = torch.Generator(device="cuda").manual_seed(V + B)
    x = (torch.randn(B, 1, V, device="cuda", generator=g) * 2.5).to(BF16)
    n = [V + 30000 if b in (0, 7, B - 1) else (0, 5, 300)[b % 3] for b in range(B)]
    starts = torch.tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32), device="cuda")
    tokens = torch.randint(0, V, (sum(n),), device="cuda", generator=g, dtype=torch.int32)
    values = torch.randn(sum(n), device="cuda", generator=g)
    tokens[:V] = torch.randperm(V, device="cuda", generator=g).int()       # all of them in the first
    request = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
    allowed = torch.randint(-2 ** 31, 2 ** 31, (B, 1, -(-V // 32)), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    v = torch.arange(V, device="cuda")
    wants, most = [], 0
    for b in range(B):
        mine = request == b
        y = x[b, 0].double().index_put_((tokens[mine].long(),), values[mine].double(), accumulate=True)
        most = max(most, int(torch.bincount(tokens[mine], minlength=1).max())) if n[b] else most
        wants.append(torch.softmax(torch.where((allowed[b, 0][v // 32] >> (v % 32)) & 1 == 1, y, -torch.inf), -1))
    out = x if in_place else torch.full((B, 1, V), 7.0, device="cuda")
    keep = x.clone()
    da.token_probs(x, out, bias=(starts, tokens, values), allowed=allowed)
    # x: `most` sums of magnitudes up to 30 (logits of 2.5 sigma, each sum of normal biases), for the token, the largest and the total;
    # the exponent's four; ex2 three times; a thread's values one behind the other, then 13
    u = 2.0 ** -24
    rel, eps = u * (3 * most * 30 + 8 * 30 + 12 + V // 512 + 16), {True: 2.0 ** -8, False: u}[in_place]
    for b in range(B):
        assert ((out[b, 0].double() - wants[b]).abs() <= wants[b] * ((1 + rel) * (1 + eps) - 1) + 2.0 ** -126).all(), b
    for _ in range(3):
        again = torch.full_like(out, 9.0)
        da.token_probs(keep, again, bias=(starts, tokens, values), allowed=allowed)
        assert torch.equal(again, out)


def test_one_token_tens_of_thousands_of_times():
    g = np.random.RandomState(1)
    V, n = 3001, 60000
    tokens = np.where(g.rand(n) < 0.9, 1777, g.randint(-5, V + 5, n))
    values = (g.randn(n) * 1000).astype(np.float32)
    values[np.flatnonzero(tokens == 1777)[-1]] -= values[tokens == 1777].sum(dtype=np.float64)
    _check((g.randn(1, 1, V) * 2).astype(np.float32), [tokens], [values])


@pytest.mark.parametrize("V,B,K", [(4000, 2, 3), (60000, 2, 1), (20000, 80, 1), (131072, 1, 3)])
def test_with_everything_else(V, B, K):
    """Histories, drafts, masks; some requests greedy, some with few biases or none; in place."""
    g = np.random.RandomState(V + B)
    x = (g.randn(B, K + 1, V) * 2.5).astype(np.float32)
    tokens, values = [], []
    for b in range(B):
        n = (3 * V // 2, 0, 7, 1500)[b % 4]
        tokens.append(g.randint(0, V, n))
        values.append((g.randn(n) * 3).astype(np.float32))
    hist, drafts = g.randint(0, V, (B, 3000)), g.randint(0, V, (B, K))
    drafts[:, 0] = tokens[0][0]
    T = g.choice([1.0, 0.5, 0.0], B)
    T[0] = 1.0
    allowed = g.rand(B, K + 1, V) < 0.7
    for in_place in (False, True):
        out = _check(x, tokens, values, F32, hist, drafts, allowed, T, in_place)
        assert float(out.sum()) == pytest.approx(B * (K + 1), rel=1e-3)
    _check(x, tokens, values, BF16, hist, drafts, allowed, T, True)


def test_again_and_again_the_same():
    g = np.random.RandomState(3)
    V, B = 131072, 6
    x = _dev((g.randn(B, 1, V) * 2.5).astype(np.float32))
    starts = _dev((np.arange(B + 1) * V).astype(np.int32))
    tokens, values = _dev(g.randint(0, V, B * V).astype(np.int32)), _dev(g.randn(B * V).astype(np.float32))
    first = None
    for _ in range(20):
        out = torch.full_like(x, 9.0)
        da.token_probs(x, out, bias=(starts, tokens, values))
        first = out if first is None else first
        assert torch.equal(out, first)
