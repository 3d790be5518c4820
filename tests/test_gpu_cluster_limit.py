"""Devices that have no room for clusters of 16 CTAs: the page operators and the
token probabilities with clusters of at most eight (a switch of the test build),
at the sizes that take 16 where there is room."""
import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import debug_build_library

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def tlib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib = debug_build_library()
    assert lib.decode_attn_debug_max_cluster(4) != 0
    assert lib.decode_attn_debug_max_cluster(8) == 0
    yield lib
    lib.decode_attn_debug_max_cluster(16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,B,cols,near", [(40000, 1, 0, 0), (128259, 1, 600, 0), ((1 << 19) - 7, 1, 0, 0), ((1 << 19) - 7, 2, 40000, 0),
                                           ((1 << 19) - 7, 2, 50000, 60000), (131072, 40, 131072, 0)])
def test_probabilities(tlib, dtype, V, B, cols, near):
    """Long rows, lists of every length; `near`: the history's tokens lie below it, so that one share has more of them than
    any list has room for (27904). Against float64."""
    g = torch.Generator(device="cuda").manual_seed(V % 101 + cols)
    x = (torch.randn(B, 1, V, device="cuda", generator=g) * 2.5).to(dtype)
    rand = lambda: torch.rand(B, device="cuda", generator=g) + 0.5  # noqa: E731
    T, rep, freq, pres = rand(), rand(), rand(), rand()
    rules = dict(temperature=T, repetition=rep, frequency=freq, presence=pres)
    y = x[:, 0].double()
    counts = 0
    if cols:
        hist = torch.randint(0, near or V, (B, cols), device="cuda", generator=g, dtype=torch.int32)
        if near:
            hist[0, :near * 3 // 4] = torch.randperm(near, device="cuda", generator=g)[:near * 3 // 4].int()
        lens = torch.full((B,), cols, dtype=torch.int32, device="cuda")
        lens[1:] //= 3
        prompt = lens // 4
        rules.update(history=hist, history_lens=lens, prompt_lens=prompt)
        i = torch.arange(cols, device="cuda")
        there, asked = i < lens[:, None], i < prompt[:, None]
        z = torch.zeros(B, V, dtype=torch.float64, device="cuda")
        said = z.scatter_add(1, hist.long(), (there & ~asked).double())
        seen = z.scatter_add(1, hist.long(), there.double()) > 0
        counts = float(said.max())
        if near:
            assert int(seen[0].sum()) > 27904
        c = lambda v: v.double()[:, None]  # noqa: E731
        y = torch.where(seen, torch.where(y > 0, y / c(rep), y * c(rep)), y) - c(freq) * said - torch.where(said > 0, c(pres), 0.0)
    want = torch.softmax(y / T.double()[:, None], -1)
    out, err = torch.empty(B, 1, V, device="cuda"), _i32([0])
    da.token_probs(x, out, device_error=err, lib=tlib, **rules)
    torch.cuda.synchronize()
    assert int(err) == 0
    # fp32: five roundings of magnitudes up to 30 + 1.5 counts over T >= 0.5 for the token, the largest and the total; the
    # exponent's four for the token and the total; ex2 three times (4 u each); a thread's groups of eight (a share has V / 64 / 512
    # of them for a thread at most, one behind the other), 3 additions in a group, 13 above
    u, big = 2.0 ** -24, 30 + 1.5 * counts
    rel = u * (3 * 5 * big / 0.5 + 8 * big / 0.5 + 12 + V // 64 // 512 + 2 + (1 if not cols else 1 + 65536 // 512) + 16)
    assert ((out[:, 0].double() - want).abs() <= want * rel + 2.0 ** -126).all()
    same = torch.empty_like(out)
    da.token_probs(x, same, device_error=err, lib=tlib, **rules)
    assert torch.equal(same, out)


@pytest.mark.parametrize("pages", [200000, 1 << 21, 1 << 23])
@pytest.mark.parametrize("B", [40, 8192])
def test_pages(tlib, pages, B):
    """Every entry as with the product's clusters (which other tests compare with the replica)."""
    P, cols = 16, 20
    g = np.random.RandomState(B)
    desc = da.Desc.make(B=B, H_kv=1, G=8, D_qk=64, D_v=64, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=da.KV_BF16)
    taken = torch.from_numpy((g.rand(pages) < 0.5).astype(np.int32)).cuda()
    asks = _i32(g.randint(0, P * 6, size=B).tolist())
    results = []
    for lib in (None, tlib):
        table, held, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, cols), (B,), (B,)))
        refs, copies, missing, err = taken.clone(), _i32([[0, 0]] * B), _i32([5]), _i32([0])
        da.reserve_pages(desc, lens, table, held, refs, copies, missing, new_tokens=asks, device_error=err, lib=lib)
        into, new_refs, new_page, counts = torch.zeros_like(table), torch.zeros_like(refs), torch.zeros_like(refs), _i32([0, 0])
        pairs = torch.zeros(pages // 2, 2, dtype=torch.int32, device="cuda")
        da.compact_pages(desc, table, held, refs, into, new_refs, new_page, pairs, counts, device_error=err, lib=lib)
        torch.cuda.synchronize()
        assert int(err) == 0 and int(missing) == 0 and int(counts[0]) == int((refs > 0).sum())
        results.append((table, held, refs, copies, into, new_refs, new_page, pairs, counts))
    assert all(torch.equal(a, b) for a, b in zip(*results))
