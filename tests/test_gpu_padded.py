"""A batch padded with rows that are no requests, as a captured step of a fixed
size has them: length 0, no drafts (-1), positions -1. They report nothing,
change nothing, keep the length 0, and the other rows come out as without them."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _step(kv, real, pad):
    """One step of `real` requests and `pad` rows behind them (one split each, so that no sum depends on the batch);
    everything it writes."""
    g = torch.Generator().manual_seed(7)
    latent = kv == da.KV_MLA656
    H, G, D, Dv, P, cols, s_q, V, budget = (1, 128, 576, 512, 16, 16, 3, 700, 90) if latent else (2, 8, 64, 64, 16, 16, 3, 700, 90)
    pages, B = 2 * real * cols, real + pad
    perm = torch.randperm(pages, generator=g).int()
    table, into = (torch.cat([t.view(real, cols), torch.full((pad, cols), -1, dtype=torch.int32)]).cuda() for t in perm.split(real * cols))
    more = lambda t, fill: torch.cat([t, torch.full((pad, *t.shape[1:]), fill, dtype=t.dtype)])  # noqa: E731
    lens = [20 + 61 * b for b in range(real)]
    full, before = _i32(lens + [0] * pad), _i32([n - s_q for n in lens] + [0] * pad)
    desc = da.Desc.make(B=B, H_kv=H, G=G, D_qk=D, D_v=Dv, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=kv, s_q=s_q,
                        splits=1)
    if latent:
        k, v = torch.randint(0, 96, (pages, P, 1, 656), generator=g, dtype=torch.uint8), None
        k[..., 512:528] = torch.full((pages, P, 1, 4), 0.02).view(torch.uint8)
        k[..., 528:] = torch.randn(pages, P, 1, 64, generator=g).to(torch.bfloat16).view(torch.uint8)
        k = k.cuda()
    else:
        k, v = (torch.randn(pages, P, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    weights = torch.rand(pages, H, P, generator=g).cuda()
    x = more(torch.randn(real, s_q, (G * H + (1 if latent else 2 * H)) * D, generator=g).to(torch.bfloat16), 1.0).cuda().flatten(0, 1)
    pos = more(torch.tensor([[n - s_q + j for j in range(s_q)] for n in lens], dtype=torch.int32), -1).cuda().flatten()
    drafts = more(torch.randint(0, V, (real, s_q - 1), generator=g).int(), -1).cuda()
    p = more(torch.softmax(torch.randn(real, s_q, V, generator=g), -1), 1.0 / V).cuda()
    u = more(torch.rand(real, s_q, generator=g), 0.5).cuda()
    q = torch.full((B * s_q, H * G, D), -3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(B, s_q, H * G, Dv, dtype=torch.bfloat16, device="cuda"), torch.empty(B, s_q, H * G, device="cuda")
    acc, toks, new, cut, err = _i32([9] * B), _i32([[9] * s_q] * B), _i32([9] * B), _i32([9] * B), _i32([0])
    kept = torch.full((B, H, budget), 9, dtype=torch.int32, device="cuda")
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    q_len, kv_len = G * H * D, H * D
    da.rope_append(desc, da.Rope.make(64), x[:, :q_len], x[:, q_len:q_len + kv_len], None if latent else x[:, q_len + kv_len:],
                   torch.ones(32, device="cuda"), pos.view(1, -1), pos, table, q, k, v, device_error=err)
    da.sched_meta(desc, full, meta)
    da.fwd(desc, q, k, v, None, None, table, full, meta, out, lse)
    da.verify_drafts(p, None, drafts, u, acc, toks, cache_seqlens=full, new_seqlens=new, device_error=err)
    da.accum_weights(desc, q, k, None, table, full, meta, lse, weights, num_accepted=acc, weighted_lens=before)
    da.evict(desc, budget, new, table, into, k, v, weights, kept, cut, keep_first=1, keep_last=4, device_error=err)
    meta2 = torch.empty_like(meta)
    da.sched_meta(desc, cut, meta2)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and da.get_error(meta) == 0 and da.get_error(meta2) == 0
    return dict(k=k, weights=weights, **({} if latent else dict(v=v))), dict(q=q.view(B, s_q, H * G, D), out=out, lse=lse, acc=acc, toks=toks,
                                                                             new=new, cut=cut, kept=kept)


@pytest.mark.parametrize("kv", [da.KV_BF16, da.KV_MLA656])
@pytest.mark.parametrize("pad", [1, 4])
def test_rows_that_are_no_requests(kv, pad):
    real = 4
    pools, rows = _step(kv, real, 0)
    pools2, rows2 = _step(kv, real, pad)
    for name, t in pools.items():
        assert torch.equal(pools2[name], t), name
    for name, t in rows.items():
        assert torch.equal(rows2[name][:real], t), name
    for name in ("acc", "new", "cut"):
        assert (rows2[name][real:] == 0).all(), name
    assert (rows2["kept"][real:] == -1).all() and (rows2["q"][real:] == -3.0).all() and torch.isneginf(rows2["lse"][real:]).all()


def test_lengths_shorter_than_the_chain():
    """A length that cannot hold the drafts gives 0, never less."""
    V, K = 50, 3
    p = torch.full((4, K + 1, V), 1.0 / V, device="cuda")
    x, u = _i32([[-1] * K, [-1] * K, [4, 5, -1], [4, 5, 6]]), torch.zeros(4, K + 1, device="cuda")
    acc, toks, new = _i32([0] * 4), torch.empty(4, K + 1, dtype=torch.int32, device="cuda"), _i32([9] * 4)
    da.verify_drafts(p, None, x, u, acc, toks, cache_seqlens=_i32([0, 2, 2, -(1 << 31)]), new_seqlens=new)
    assert acc.tolist() == [0, 0, 2, 3] and new.tolist() == [0, 0, 1, 0]
