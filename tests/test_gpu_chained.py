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

    def buffers(self):
        """What the calls write, and copies of what they change."""
        e = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        B, HG, bf16, f32 = self.B, self.q.shape[2], torch.bfloat16, torch.float32
        pools = [p.clone() for p in self.pools]
        return dict(k=pools[0], v=pools[1] if len(pools) > 1 else None, weights=self.weights.clone(),
                    meta=e(da.sched_meta_bytes(self.desc), dtype=torch.uint8), meta2=e(da.sched_meta_bytes(self.one), dtype=torch.uint8),
                    out=e(B, 2, HG, self.Dv, dtype=bf16), lse=e(B, 2, HG, dtype=f32), out2=e(B, HG, self.Dv, dtype=bf16),
                    lse2=e(B, HG, dtype=f32), accepted=e(B), tokens=e(B, 2), new=e(B), cut=e(B), err=e(1), kept=e(B, self.H, self.budget),
                    q=e(B, HG, self.D, dtype=bf16))

    def calls(self, s, wait=lambda: None):
        B, scale, k, v, err = self.B, self.scale, s["k"], s["v"], s["err"]
        q_len, kv_len = s["q"].shape[1] * self.D, self.H * self.D
        nk, nv = self.new[:, q_len:q_len + kv_len], None if self.kv == MLA else self.new[:, q_len + kv_len:]
        da.sched_meta(self.desc, self.lens, s["meta"])
        wait()
        da.fwd(self.desc, self.q, k, v, scale, scale, self.table, self.lens, s["meta"], s["out"], s["lse"])
        wait()
        da.verify_drafts(self.p, None, self.x, self.u, s["accepted"], s["tokens"], cache_seqlens=self.lens, new_seqlens=s["new"],
                         device_error=err)
        wait()
        da.accum_weights(self.desc, self.q, k, scale, self.table, self.lens, s["meta"], s["lse"], s["weights"],
                         num_accepted=s["accepted"], weighted_lens=self.weighted, decay=0.5)
        wait()
        da.evict(self.one, self.budget, s["new"], self.table, self.into, k, v, s["weights"], s["kept"], s["cut"], keep_first=2,
                 keep_last=16, device_error=err)
        wait()
        da.rope_append(self.one, da.Rope.make(64), self.new[:, :q_len], nk, nv, self.freq, s["cut"].view(1, B), s["accepted"], self.into,
                       s["q"], k, v, scale, scale, device_error=err)
        wait()
        da.sched_meta(self.one, s["cut"], s["meta2"])
        wait()
        da.fwd(self.one, s["q"], k, v, scale, scale, self.into, s["cut"], s["meta2"], s["out2"], s["lse2"])

    def results(self, s):
        assert int(s["err"].item()) == 0 and da.get_error(s["meta"]) == 0 and da.get_error(s["meta2"]) == 0
        return {n: t for n, t in s.items() if t is not None and not n.startswith("meta")}

    def run(self, sync):
        s = self.buffers()
        torch.cuda.synchronize()
        self.calls(s, torch.cuda.synchronize if sync else (lambda: None))
        torch.cuda.synchronize()
        return self.results(s)


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


def test_loops_of_three_formats_at_once():
    """The same loops on three streams, all of their calls enqueued behind one event before any of them can start, so
    that attention, accumulation, eviction and appends of different formats run beside each other."""
    loops = [Loop(kv, H, D, P, B=6, seed=3 + kv) for kv, H, D, P in ((BF16, 4, 64, 8), (FP8, 4, 128, 16), (MLA, 1, 576, 16))]
    want = [loop.run(sync=True) for loop in loops]
    reps = 4
    states = [[loop.buffers() for _ in range(reps)] for loop in loops]
    streams = [torch.cuda.Stream() for _ in loops]
    busy = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(60):                                   # about 20 ms, the time to enqueue everything else
        busy.copy_(busy.roll(1))
    start = torch.cuda.Event()
    start.record()
    for st in streams:
        st.wait_event(start)
    for rep in range(reps):
        for loop, st, state in zip(loops, streams, states):
            with torch.cuda.stream(st):
                loop.calls(state[rep])
    torch.cuda.synchronize()
    for loop, ref, state in zip(loops, want, states):
        for rep in range(reps):
            got = loop.results(state[rep])
            for name, t in ref.items():
                assert torch.equal(got[name], t), (name, loop.kv, rep)
