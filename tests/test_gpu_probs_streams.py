"""Token probabilities of rows whose shares stream: in place, where pieces are
loaded again from rows that are being written; into rows that are aligned
otherwise than the logits; with lists as long as there is room for."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _padded(B, V, pad, dtype, fill=77.0):
    """Rows [B, 1, V] that start `pad` elements into a row of V + 2 pad + 1 (pad 0: packed), and what is around them."""
    width = V if pad == 0 else V + 2 * pad + 1
    store = torch.full((B, width), fill, dtype=dtype, device="cuda")
    return store[:, pad:pad + V].unflatten(1, (1, V)), store


def _rules(B, V, cols, seed, masks=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda: torch.rand(B, device="cuda", generator=g) + 0.5  # noqa: E731
    r = dict(temperature=rand(), repetition=rand(), frequency=rand(), presence=rand())
    r["history"] = torch.randint(0, V, (B, cols), device="cuda", generator=g, dtype=torch.int32)
    r["history_lens"] = torch.randint(0, cols + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    r["prompt_lens"] = r["history_lens"] // 3
    if masks:
        r["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (B, 1, -(-V // 32)), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)
    return r


def _want(x, r, V):
    """Float64, by the definition; x [B, V]."""
    B, cols = r["history"].shape
    i = torch.arange(cols, device="cuda")
    there, asked = i < r["history_lens"][:, None], i < r["prompt_lens"][:, None]
    z = torch.zeros(B, V, dtype=torch.float64, device="cuda")
    said = z.scatter_add(1, r["history"].long(), (there & ~asked).double())
    seen = z.scatter_add(1, r["history"].long(), there.double()) > 0
    c = lambda n: r[n].double()[:, None]  # noqa: E731
    y = x.double()
    y = torch.where(seen, torch.where(y > 0, y / c("repetition"), y * c("repetition")), y)
    y = y - c("frequency") * said - torch.where(said > 0, c("presence"), 0.0)
    if "allowed" in r:
        v = torch.arange(V, device="cuda")
        y = torch.where((r["allowed"][:, 0][:, v // 32] >> (v % 32)) & 1 == 1, y, -torch.inf)
    return torch.softmax(torch.where(torch.isneginf(y), y, y / c("temperature")), -1)


def _close(got, want, dtype, counts, V):
    """x: five roundings of magnitudes up to 30 + 1.5 counts (logits of 2.5 sigma, penalties up to 1.5 a count) over T >= 0.5,
    for the token, for the largest and for the total; the exponent's four, likewise for the token and the total; ex2 three times
    (2 ulp: 4 u each), and a thread's sum: its groups of eight one behind the other (3 additions in a group), then 9 over its
    CTA and 4 over a cluster. Then the rounding to the type."""
    u = 2.0 ** -24
    big = 30 + 1.5 * counts
    groups = -(-V // 8 // 512) + 1
    rel = u * (3 * 5 * big / 0.5 + 8 * big / 0.5 + 12 + groups + 3 + 13)
    assert ((got.double() - want).abs() <= want * ((1 + rel) * (1 + EPS[dtype]) - 1) + TINY[dtype]).all()


@pytest.mark.parametrize("pad", [0, 3, 5])
@pytest.mark.parametrize("dtype,B,V", [(BF16, 200, 130999), (F32, 160, 130999), (F16, 190, 128003)])
def test_rows_loaded_again_in_place_and_unaligned(dtype, B, V, pad):
    """One or two CTAs a row, each with more pieces than slots."""
    x = (torch.randn(B, 1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(pad)) * 2.5).to(dtype)
    for masks, greedy in ((True, False), (False, False), (True, True)):
        r = _rules(B, V, 3000, 7 + pad, masks)
        if greedy:
            r["temperature"] = torch.zeros(B, device="cuda")
        logits, around = _padded(B, V, pad, dtype)
        logits.copy_(x)
        same, _ = _padded(B, V, pad, dtype)               # aligned like the logits
        da.token_probs(logits, same, **r)
        other, beside = _padded(B, V, pad + 2, dtype)     # otherwise
        da.token_probs(logits, other, **r)
        assert torch.equal(other, same)
        assert (beside[:, :pad + 2] == 77).all() and (beside[:, pad + 2 + V:] == 77).all()
        wide, beside = _padded(B, V, pad + 1, F32)        # and in another type
        da.token_probs(logits, wide, **r)
        assert torch.equal(wide.to(dtype), same)
        assert (beside[:, :pad + 1] == 77).all() and (beside[:, pad + 1 + V:] == 77).all()
        assert torch.equal(logits, x)
        da.token_probs(logits, logits, **r)
        assert torch.equal(logits, same)
        if pad:
            assert (around[:, :pad] == 77).all() and (around[:, pad + V:] == 77).all()
        if greedy:
            assert ((same == 1).sum(-1) == 1).all() and ((same == 0).sum(-1) == V - 1).all()
            continue
        for lo in range(0, B, 40):
            s = {k: t[lo:lo + 40] for k, t in r.items()}
            want = _want(x[lo:lo + 40, 0], s, V)
            _close(same[lo:lo + 40, 0], want, dtype, 6, V)
            _close(wide[lo:lo + 40, 0], want, F32, 6, V)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [32768, 50000])
def test_long_lists_beside_a_short_ring(dtype, cols):
    """16 CTAs a row, each with a share of 32768 tokens and a list that leaves room for few pieces, or is too short itself."""
    B, V = 3, (1 << 19) - 7
    x = (torch.randn(B, 1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(cols)) * 2.5).to(dtype)
    r = _rules(B, V, cols, cols)
    r["history_lens"][:] = torch.tensor([cols, 7, cols // 2], device="cuda")
    r["history"][0, ::2] %= 20000                         # one share has most of them
    out = torch.empty_like(x)
    da.token_probs(x, out, **r)
    other, _ = _padded(B, V, 1, dtype)
    da.token_probs(x, other, **r)
    assert torch.equal(other, out)
    want = _want(x[:, 0], r, V)
    _close(out[:, 0], want, dtype, 20, V)
    keep = x.clone()
    da.token_probs(keep, keep, **r)
    assert torch.equal(keep, out)


def test_a_history_buffer_far_wider_than_what_is_used():
    """The same probabilities, but for the order of sums."""
    B, V = 170, 131072
    x = (torch.randn(B, 1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) * 2.5).to(BF16)
    narrow = _rules(B, V, 64, 5, masks=False)
    wide = dict(narrow, history=torch.cat([narrow["history"], torch.full((B, V - 64), 11, dtype=torch.int32, device="cuda")], 1))
    want = _want(x[:, 0], narrow, V)
    for r in (narrow, wide):
        out = torch.empty(B, 1, V, device="cuda")
        da.token_probs(x, out, **r)
        _close(out[:, 0], want, F32, 2, V)


@pytest.mark.parametrize("dtype,B,V,cols", [(BF16, 200, 130999, 20000), (F32, 160, 131072, 40000), (BF16, 320, 65000, 65000), (BF16, 70, 131072, 131072)])
def test_histories_longer_than_a_list(dtype, B, V, cols):
    """Shares whose touched tokens take one window (short texts in a wide buffer), two, or many; in place; again and again the
    same."""
    x = (torch.randn(B, 1, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(B)) * 2.5).to(dtype)
    r = _rules(B, V, cols, B)
    r["history_lens"][0], r["history_lens"][1], r["history_lens"][2] = cols, 0, 9345
    out = torch.empty_like(x)
    da.token_probs(x, out, **r)
    for lo in range(0, B, 40):
        s = {k: t[lo:lo + 40] for k, t in r.items()}
        # a token stands there 1 time in the mean at most: 14 times or more with a chance below 1e-11, of 1e7 tokens
        _close(out[lo:lo + 40, 0], _want(x[lo:lo + 40, 0], s, V), dtype, 14, V)
    for _ in range(5):
        same = torch.full_like(x, 7.0)
        da.token_probs(x, same, **r)
        assert torch.equal(same, out)
    da.token_probs(x, x, **r)
    assert torch.equal(x, out)
