"""Pools of more than 4 GiB whose last pages hold the tokens: byte offsets beyond
2^32 (and element indices beyond 2^31) in every operator and format. The same
calls on a pool of a few pages give the values to compare with, bit for bit."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16, FP8, MLA = da.KV_BF16, da.KV_FP8, da.KV_MLA656


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _loop(kv, H, D, P, num_pages, table, into):
    """Prompt, one more token by append_kv, attention, accumulation, eviction; what they leave, read through the tables."""
    G, Dv, row = (128, 512, 656) if kv == MLA else (8, D, D * (2 if kv == BF16 else 1))
    L, budget, B = [150, 40], 90, 2
    g = torch.Generator().manual_seed(D)
    desc = da.Desc.make(B=B, H_kv=H, G=G, D_qk=D, D_v=Dv, page_size=P, max_pages_per_seq=len(table[0]), num_pages=num_pages, kv_dtype=kv)
    pools = [torch.empty(num_pages, P, H, row, dtype=torch.uint8, device="cuda") for _ in range(1 if kv == MLA else 2)]
    k, v = pools[0], None if kv == MLA else pools[1]
    weights = torch.zeros(num_pages, H, P, device="cuda")
    scale = torch.full((H,), 1 / 64, device="cuda") if kv == FP8 else None
    table, into, lens, err = _i32(table), _i32(into), _i32(L), _i32([0])
    n, q_len, kv_len = sum(L) - B, G * H * D, H * D
    x = torch.randn(n + B, q_len + (1 if kv == MLA else 2) * kv_len, generator=g).to(torch.bfloat16).cuda()
    nk, nv = x[:, q_len:q_len + kv_len], None if kv == MLA else x[:, q_len + kv_len:]
    pos = _i32([t for m in L for t in range(m - 1)])
    q_out = torch.empty(n, G * H, D, dtype=torch.bfloat16, device="cuda")
    da.rope_append(desc, da.Rope.make(64), x[:n, :q_len], nk[:n], None if nv is None else nv[:n], torch.full((32,), 0.1, device="cuda"),
                   pos.view(1, -1), pos, table, q_out, k, v, scale, scale, requests=_i32([b for b, m in enumerate(L) for _ in range(m - 1)]),
                   device_error=err)
    da.append_kv(desc, nk[n:].contiguous(), None if nv is None else nv[n:].contiguous(), _i32([m - 1 for m in L]), table, k, v, scale,
                 scale, device_error=err)
    q = x[n:, :q_len].contiguous()
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(B, G * H, Dv, dtype=torch.bfloat16, device="cuda"), torch.empty(B, G * H, device="cuda")
    da.sched_meta(desc, lens, meta)
    da.fwd(desc, q, k, v, scale, scale, table, lens, meta, out, lse)
    da.accum_weights(desc, q, k, scale, table, lens, meta, lse, weights, weighted_lens=_i32([0, 0]))
    tokens = lambda t, pool, m: torch.cat([pool[t[b, :-(-m[b] // P)].long()].flatten(0, 1)[:m[b]] for b in range(B)])  # noqa: E731
    got = dict(q=q_out, out=out, lse=lse, w=tokens(table, weights.transpose(1, 2), L), k=tokens(table, k, L))
    kept, cut = torch.empty(B, H, budget, dtype=torch.int32, device="cuda"), _i32([0] * B)
    da.evict(desc, budget, lens, table, into, k, v, weights, kept, cut, keep_first=2, keep_last=8, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and da.get_error(meta) == 0 and cut.tolist() == [budget, 40]
    got.update(kept=kept, k2=tokens(into, k, [budget, 40]), w2=tokens(into, weights.transpose(1, 2), [budget, 40]))
    if v is not None:
        got.update(v=tokens(table, v, L), v2=tokens(into, v, [budget, 40]))
    return got


@pytest.mark.parametrize("kv,H,D,num_pages", [(BF16, 8, 128, 40000), (FP8, 8, 128, 70000), (MLA, 1, 576, 110000)])
def test_the_last_pages_of_a_large_pool(kv, H, D, num_pages):
    P = 64
    page_bytes = P * H * (656 if kv == MLA else D * (2 if kv == BF16 else 1))
    assert (num_pages - 10) * page_bytes > 1 << 32
    n = num_pages
    far = ([[n - 1, 3, n - 2, -1], [n - 6, -1, -1, -1]], [[n - 5, n - 4, -1, -1], [5, -1, -1, -1]])     # from far to far, and to near
    m = 16
    near = ([[m - 1, 3, m - 2, -1], [m - 6, -1, -1, -1]], [[m - 5, m - 4, -1, -1], [5, -1, -1, -1]])
    want, got = _loop(kv, H, D, P, m, *near), _loop(kv, H, D, P, num_pages, *far)
    for name, t in want.items():
        assert torch.equal(got[name], t), name
    rows = want["k"].view(torch.uint8).flatten(1)
    assert (rows != rows[:1]).any(1)[1:].all()             # rows that tell one token from another
