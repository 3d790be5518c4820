"""Pools whose byte offsets pass 32 bits: the last pages of pools of more than
4 GB hold the tokens."""
import math

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


def test_rows_beyond_four_gigabytes():
    H, D, P, G = 8, 128, 64, 8
    num_pages = 20000                                     # 2.6 GB a pool in elements, 5.2 GB in bytes
    kp, vp = (torch.empty(num_pages, P, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights = torch.zeros(num_pages, H, P, device="cuda")
    table = torch.tensor([[num_pages - 1, 3, num_pages - 2, -1]], dtype=torch.int32, device="cuda")
    into = torch.tensor([[num_pages - 5, num_pages - 4, -1, -1]], dtype=torch.int32, device="cuda")
    L = 150
    desc = da.Desc.make(B=1, H_kv=H, G=G, D_qk=D, D_v=D, page_size=P, max_pages_per_seq=4, num_pages=num_pages)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(L, (G + 2) * H * D, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :G * H * D], x[:, G * H * D:(G + 1) * H * D], x[:, (G + 1) * H * D:]
    q_out, err = torch.empty(L, G * H, D, dtype=torch.bfloat16, device="cuda"), i32([0])
    at = torch.zeros(1, L, dtype=torch.int32, device="cuda")   # no rotation: plain copies to compare with
    da.rope_append(desc, da.Rope.make(D), q, k, v, torch.ones(D // 2, device="cuda"), at, torch.arange(L, device="cuda").int(), table,
                   q_out, kp, vp, requests=torch.zeros(L, dtype=torch.int32, device="cuda"), device_error=err)
    assert torch.equal(q_out.view(L, -1), q)
    rows = lambda pool, t: pool[t[0, :3].clamp(min=0).long()].reshape(-1, H, D)  # noqa: E731
    assert torch.equal(rows(kp, table)[:L], k.view(L, H, D)) and torch.equal(rows(vp, table)[:L], v.view(L, H, D))
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    lens = i32([L])
    out, lse = torch.empty(1, G * H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, G * H, device="cuda")
    qq = q_out[-1:].contiguous()
    da.sched_meta(desc, lens, meta)
    da.fwd(desc, qq, kp, vp, None, None, table, lens, meta, out, lse)
    da.accum_weights(desc, qq, kp, None, table, lens, meta, lse, weights, weighted_lens=i32([0]))
    s = torch.einsum("hgd,thd->hgt", qq.view(H, G, D).double(), k.view(L, H, D).double()) / math.sqrt(D)
    want = s.softmax(-1).sum(1)                             # [H, L]
    got = weights[table[0, :3].long()].permute(1, 0, 2).reshape(H, -1)[:, :L]
    assert torch.allclose(got.double(), want, rtol=1e-4, atol=0)
    kept, new = torch.empty(1, H, 100, dtype=torch.int32, device="cuda"), i32([0])
    da.evict(desc, 100, lens, table, into, kp, vp, weights, kept, new, keep_first=2, keep_last=10, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and new.tolist() == [100] and da.get_error(meta) == 0
    for h in range(H):
        keep = kept[0, h].long()
        assert (keep[1:] > keep[:-1]).all() and keep[0] == 0 and keep[-1] == L - 1
        assert torch.equal(kp[into[0, :2].long()].reshape(-1, H, D)[:100, h], k.view(L, H, D)[keep, h])
        assert torch.equal(vp[into[0, :2].long()].reshape(-1, H, D)[:100, h], v.view(L, H, D)[keep, h])
