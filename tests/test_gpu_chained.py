"""Calls that read what the call before them wrote, on one stream with nothing
between them: each kernel may be resident while the one before it still writes
(programmatic dependent launch). The same calls with a synchronisation after
each give the values to compare with, bit for bit. Pages of 8 tokens put the
weights of four heads, which different SMs write, into one 128-byte line."""
import math

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


class Loop:
    """A chain of two drafts on filled caches: schedule, attention, verification, accumulation, eviction to other
    pages, then a new row (in the slot that the accepted count names, turned by the length that the eviction gave),
    schedule and attention behind it."""

    def __init__(self, kv, H, D, P, B, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.kv, self.H, self.D, self.B, self.s_q, self.budget = kv, H, D, B, 2, 600
        G, self.Dv = (128, 512) if kv == MLA else (8, D)
        lens = torch.randint(300, 1500, (B,), generator=r).tolist()
        self.cols = -(-1500 // P)
        pages = 2 * B * self.cols
        perm = torch.randperm(pages, generator=r).int().cuda()
        self.table, self.into = (t.clone().view(B, self.cols) for t in perm.split(B * self.cols))
        base = dict(B=B, H_kv=H, G=G, D_qk=D, D_v=self.Dv, page_size=P, max_pages_per_seq=self.cols, num_pages=pages, kv_dtype=kv)
        self.desc, self.one = da.Desc.make(**base, s_q=2), da.Desc.make(**base)
        self.scale = torch.full((H,), 0.03, device="cuda") if kv == FP8 else None
        if kv == MLA:
            x = torch.randint(0, 96, (pages, P, 1, 656), generator=g, device="cuda", dtype=torch.uint8)
            x[..., 512:528] = torch.full((pages, P, 1, 4), 0.02, device="cuda").view(torch.uint8)
            x[..., 528:] = rand(pages, P, 1, 64).to(torch.bfloat16).view(torch.uint8)
            self.pools = [x]
        elif kv == FP8:
            self.pools = [(rand(pages, P, H, D) / 0.03).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
        else:
            self.pools = [rand(pages, P, H, D).to(torch.bfloat16) for _ in range(2)]
        self.weights, self.lens, self.weighted = rand(pages, H, P).abs() * 1e-3, _i32(lens), _i32([n - 2 for n in lens])
        self.q = rand(B, 2, H * G, D).to(torch.bfloat16)
        self.p = torch.softmax(rand(B, 2, 3000) * 2, -1)
        self.x = torch.randint(0, 3000, (B, 1), generator=r).int().cuda()
        self.u = torch.rand(B, 2, generator=g, device="cuda")
        self.new = rand(B, (H * G + (1 if kv == MLA else 2 * H)) * D).to(torch.bfloat16)
        self.freq = (1000.0 ** (-torch.arange(32) / 32)).float().cuda()

    def run(self, sync):
        e = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        B, H, D, HG, scale = self.B, self.H, self.D, self.q.shape[2], self.scale
        pools, w = [p.clone() for p in self.pools], self.weights.clone()
        k, v = pools[0], pools[1] if len(pools) > 1 else None
        meta, meta2 = (e(da.sched_meta_bytes(d), dtype=torch.uint8) for d in (self.desc, self.one))
        out, lse = e(B, 2, HG, self.Dv, dtype=torch.bfloat16), e(B, 2, HG, dtype=torch.float32)
        out2, lse2 = e(B, HG, self.Dv, dtype=torch.bfloat16), e(B, HG, dtype=torch.float32)
        acc, tok, new, cut, err, kept = e(B), e(B, 2), e(B), e(B), e(1), e(B, H, self.budget)
        q_out, q_len, kv_len = e(B, HG, D, dtype=torch.bfloat16), HG * D, H * D
        nk, nv = self.new[:, q_len:q_len + kv_len], None if self.kv == MLA else self.new[:, q_len + kv_len:]
        wait = torch.cuda.synchronize if sync else (lambda: None)
        torch.cuda.synchronize()
        da.sched_meta(self.desc, self.lens, meta)
        wait()
        da.fwd(self.desc, self.q, k, v, scale, scale, self.table, self.lens, meta, out, lse)
        wait()
        da.verify_drafts(self.p, None, self.x, self.u, acc, tok, cache_seqlens=self.lens, new_seqlens=new, device_error=err)
        wait()
        da.accum_weights(self.desc, self.q, k, scale, self.table, self.lens, meta, lse, w, num_accepted=acc,
                         weighted_lens=self.weighted, decay=0.5)
        wait()
        da.evict(self.one, self.budget, new, self.table, self.into, k, v, w, kept, cut, keep_first=2, keep_last=16, device_error=err)
        wait()
        da.rope_append(self.one, da.Rope.make(64), self.new[:, :q_len], nk, nv, self.freq, cut.view(1, B), acc, self.into, q_out, k, v,
                       scale, scale, device_error=err)
        wait()
        da.sched_meta(self.one, cut, meta2)
        wait()
        da.fwd(self.one, q_out, k, v, scale, scale, self.into, cut, meta2, out2, lse2)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and da.get_error(meta) == 0 and da.get_error(meta2) == 0
        return dict(out=out, lse=lse, accepted=acc, tokens=tok, new=new, weights=w, kept=kept, cut=cut, q=q_out, out2=out2, lse2=lse2,
                    k=k, **({} if v is None else {"v": v}))


@pytest.mark.parametrize("kv,H,D,P", [(BF16, 4, 64, 8), (BF16, 8, 128, 16), (FP8, 4, 128, 8), (MLA, 1, 576, 8)])
def test_a_loop_without_a_synchronisation_in_it(kv, H, D, P):
    loop = Loop(kv, H, D, P, B=5, seed=H + D + P)
    want = loop.run(sync=True)
    assert (want["cut"] <= loop.budget).all() and (want["cut"] < loop.lens).any()
    assert not any(math.isnan(float(want[n].float().sum())) for n in ("out", "weights", "out2"))
    for rep in range(12):
        got = loop.run(sync=False)
        for name, t in want.items():
            assert torch.equal(got[name], t), (name, rep)
