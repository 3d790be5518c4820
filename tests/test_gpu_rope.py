"""GPU parity of decode_attn_rope_append against the float64 oracle. Every
value is checked against the interval that its arithmetic allows:

* fp32 part: x cos - y sin with cos and sin each within 2^-22 of the exact
  ones (angle within 2^-32 of a turn, 2^-25 from its conversion, 2 ulp of the
  function), two products and a sum rounded to nearest (3 * 2^-24): together
  below 2^-20 (|x| + |y|).
* bf16: half a step of the value, 2^-8 relative.
* e4m3: rounding is monotonic, so the code's value lies between the codes of
  the ends of the fp32 interval divided by the scale.

V, the NoPE part of the latent token, values that pass through and every byte
outside the addressed rows are exact."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.append_ref import append_ref, e4m3_encode
from oracle.ops_ref import rope_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
BF16, FP8, MLA = da.KV_BF16, da.KV_FP8, da.KV_MLA656


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import oracle
    ensure_built()
    oracle.build_oracle()


class Case:
    def __init__(self, kv, B, N, H_kv, G, D, P, sections, rot, mix=0, adjacent=0, seed=0, far=1000, bad=True, stride_pad=0,
                 s_q=0):
        g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.__dict__.update(kv=kv, B=B, N=N, H_kv=H_kv, G=G, D=D, P=P, sections=sections, rot=rot, mix=mix, adjacent=adjacent)
        self.H_q = H_kv * G
        # tokens of the requests, distinct slots: consecutive positions from a start of each request's own
        req = np.sort(r.integers(0, B, N)) if not s_q else np.repeat(np.arange(B), s_q)
        start = r.integers(0, 3 * P, B)
        pos = np.array([start[b] + int((req[:i] == b).sum()) for i, b in enumerate(req)], dtype=np.int64)
        self.max_pages = int(-(-(pos.max() + 1) // P)) + 1
        self.num_pages = B * self.max_pages + 3
        table = r.permutation(self.num_pages)[:B * self.max_pages].reshape(B, self.max_pages)
        self.want_err = 0
        if bad and N > 6:
            pos[1] = -4                                    # skipped
            pos[2] = self.max_pages * P                    # past the table
            req[3], self.want_err = B, 128 | 2             # no such request
            table[req[4], pos[4] // P] = self.num_pages    # a page outside the pool (other tokens may be on it)
            self.want_err |= 1
        self.req, self.pos, self.table = req, pos, table
        self.at = r.integers(-far, far + 1, (len(sections), N))
        self.at[:, 0] = 0
        self.freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
        row = 576 if kv == MLA else H_kv * D
        wide = torch.randn(N, self.H_q * D + (1 if kv == MLA else 2) * row + stride_pad, generator=g).to(torch.bfloat16)
        self.wide, self.row, self.pad = wide, row, stride_pad
        q0 = stride_pad
        self.q, self.k = wide[:, q0:q0 + self.H_q * D], wide[:, q0 + self.H_q * D:q0 + self.H_q * D + row]
        self.v = None if kv == MLA else wide[:, q0 + self.H_q * D + row:]
        shape = (self.num_pages, P, H_kv, 656 if kv == MLA else D)
        dt = torch.bfloat16 if kv == BF16 else torch.uint8

        def pool():
            x = torch.randint(0, 256, (math.prod(shape) * (2 if kv == BF16 else 1),), generator=g, dtype=torch.uint8)
            return x.view(dt).view(shape)
        self.k_pool, self.v_pool = pool(), None if kv == MLA else pool()
        self.ks = torch.rand(H_kv, generator=g) * 0.02 + 0.004 if kv == FP8 else None
        self.vs = torch.rand(H_kv, generator=g) * 0.02 + 0.004 if kv == FP8 else None
        self.s_q = s_q

    def desc(self):
        return da.Desc.make(B=self.B, H_kv=self.H_kv, G=self.G, D_qk=self.D, D_v=512 if self.kv == MLA else self.D,
                            page_size=self.P, max_pages_per_seq=self.max_pages, num_pages=self.num_pages, kv_dtype=self.kv,
                            s_q=max(1, self.s_q))

    def run(self, in_place=False, stream=None):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
        wide, n = self.wide.cuda(), self.H_q * self.D
        q, k = wide[:, self.pad:self.pad + n], wide[:, self.pad + n:self.pad + n + self.row]
        v = None if self.v is None else wide[:, self.pad + n + self.row:]
        if in_place:
            q = q.contiguous().view(self.N, self.H_q, self.D)
        out = q if in_place else torch.full((self.N, self.H_q, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        kp, vp, err = c(self.k_pool), c(self.v_pool), torch.zeros(1, dtype=torch.int32, device="cuda")
        rope = da.Rope.make(self.rot, self.sections, interleaved=bool(self.mix), adjacent=bool(self.adjacent))
        da.rope_append(self.desc(), rope, q, k, v, torch.from_numpy(self.freq).cuda(), i32(self.at), i32(self.pos),
                       i32(self.table), out, kp, vp, c(self.ks), c(self.vs), requests=None if self.s_q else i32(self.req),
                       device_error=err, stream=stream)
        torch.cuda.synchronize()
        return out.cpu(), kp.cpu(), None if vp is None else vp.cpu(), int(err.item())

    def check(self, got, in_place=False):
        q_out, kp, vp, err = got
        assert err == self.want_err
        off = 512 if self.kv == MLA else 0
        args = (self.at, self.freq, self.sections, self.mix, self.adjacent, off)
        n, H, D = self.N, self.H_kv, self.D
        q = self.q.double().numpy().reshape(n, self.H_q, D)
        want, mag = rope_ref(q, *args)
        tol = mag * 2.0 ** -20 + np.where(mag > 0, np.abs(want) * 2.0 ** -8, 0)
        off_by = np.abs(q_out.double().numpy() - want)
        live = self.pos >= 0
        assert (off_by[live] <= tol[live]).all(), (off_by - tol)[live].max()
        rest = torch.full((), 7.0).to(torch.bfloat16) if not in_place else None
        if in_place:
            assert np.array_equal(q_out.double().numpy()[~live], q[~live])
        else:
            assert (q_out[torch.from_numpy(~live)] == rest).all()      # skipped tokens: left as they were
        # pools: as the append of the unrotated rows, but for the rotated values
        idx = [i for i in range(n) if live[i] and self.pos[i] < self.max_pages * self.P and self.req[i] < self.B
               and 0 <= self.table[self.req[i], self.pos[i] // self.P] < self.num_pages]
        t = torch.from_numpy
        ek, ev = self.k_pool, self.v_pool
        if idx:
            rows = self.table[self.req[idx], :]
            kr = self.k[idx].reshape(len(idx), H, -1)
            vr = None if self.v is None else self.v[idx].reshape(len(idx), H, D)
            bk, bv, e = append_ref(self.kv, self.P, self.k_pool, self.v_pool, kr, vr, t(self.pos[idx]), t(rows), self.ks, self.vs)
            assert e == 0
            ek = t(bk).view(self.k_pool.dtype).view(self.k_pool.shape)
            ev = None if bv is None else t(bv).view(self.v_pool.dtype).view(self.v_pool.shape)
        if ev is not None:
            assert torch.equal(vp.view(torch.uint8), ev.view(torch.uint8))
        page, slot = self.table[self.req[idx], self.pos[idx] // self.P], self.pos[idx] % self.P
        keep = torch.ones(kp.shape, dtype=torch.bool)
        kk = self.k.double().numpy().reshape(n, H, D)
        want, mag = rope_ref(kk, *args)
        want, mag = want[idx], mag[idx]
        turned = slice(0, self.rot)
        if self.kv == MLA:
            got_k = kp[page, slot][..., 528:].contiguous().view(torch.bfloat16).double().numpy()
            want, mag = want[..., 512:], mag[..., 512:]
            keep[page, slot, :, 528:528 + 2 * self.rot] = False
        else:
            keep[page, slot, :, :self.rot] = False
            got_k = kp[page, slot][..., turned]
            want, mag = want[..., turned], mag[..., turned]
        a, b = kp[keep].view(torch.uint8), ek[keep].view(torch.uint8)
        assert torch.equal(a, b)                                       # every other byte
        if self.kv == FP8:
            s = self.ks.double().numpy()[None, :, None]
            value = lambda c: t(c).view(torch.float8_e4m3fn).double().numpy()  # noqa: E731
            e = mag * 2.0 ** -20
            code = lambda x: value(e4m3_encode(np.float32(x)))  # noqa: E731
            # the quotient is rounded to fp32 before it is coded: 2^-23 of it covers that
            lo, hi = (want - e) / s, (want + e) / s
            lo, hi = lo - np.abs(lo) * 2.0 ** -23, hi + np.abs(hi) * 2.0 ** -23
            got_v = got_k.view(torch.float8_e4m3fn).double().numpy()
            assert ((got_v >= code(lo)) & (got_v <= code(hi))).all()
        else:
            got_v = got_k if isinstance(got_k, np.ndarray) else got_k.double().numpy()
            tol = mag * 2.0 ** -20 + np.abs(want) * 2.0 ** -8
            assert (np.abs(got_v - want) <= tol).all()


SHAPES = [
    # kv, B, N, H_kv, G, D, P, sections, rot
    (BF16, 1, 1, 1, 8, 64, 16, [32], 64),
    (BF16, 3, 50, 2, 8, 128, 8, [16, 24, 24], 128),
    (BF16, 5, 41, 3, 4, 96, 32, [8, 8, 8], 48),
    (BF16, 2, 9, 1, 1, 72, 64, [8], 16),
    (BF16, 2, 33, 1, 3, 256, 192, [40, 0, 24, 64], 256),
    (BF16, 4, 700, 1, 8, 64, 16, [10, 6], 32),
    (BF16, 2, 40, 2, 2, 64, 5, [32], 64),
    (BF16, 1, 9, 1, 2, 512, 16, [200, 56], 512),         # as many angles as a block has threads
    (BF16, 2, 7, 1, 1, 4096, 8, [256], 512),             # one row to a block
    (BF16, 1, 3, 1, 700, 16, 8, [4, 4], 16),
    (FP8, 3, 50, 4, 8, 128, 32, [24, 20, 20], 128),
    (FP8, 2, 31, 1, 2, 72, 16, [3, 2, 3], 16),
    (FP8, 2, 300, 2, 8, 64, 64, [16], 32),
    (MLA, 3, 50, 1, 128, 576, 64, [32], 64),
    (MLA, 1, 1, 1, 16, 576, 16, [4, 6, 6], 32),
    (MLA, 2, 90, 1, 3, 576, 8, [8], 16),
]


@pytest.mark.parametrize("adjacent", [0, 1])
@pytest.mark.parametrize("mix", [0, 1])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope_append(shape, mix, adjacent):
    c = Case(*shape, mix=mix, adjacent=adjacent, seed=sum(map(int, shape[:7])))
    c.check(c.run())


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[2], SHAPES[6], SHAPES[9], SHAPES[11]])
@pytest.mark.parametrize("adjacent", [0, 1])
def test_in_place_and_strided_rows(shape, adjacent):
    c = Case(*shape, adjacent=adjacent, seed=3)
    c.check(c.run(in_place=True), in_place=True)
    c = Case(*shape, adjacent=adjacent, seed=4, stride_pad=24)
    c.check(c.run())


def test_chain_without_request_indexes():
    c = Case(BF16, 9, 36, 2, 8, 64, 16, [32], 64, seed=5, bad=False, s_q=4)
    c.check(c.run())


@pytest.mark.parametrize("far", [(1 << 20), (1 << 28)])
def test_far_positions(far):
    """Positions whose fp32 angle would keep no digit: the tolerance is the same as for near ones."""
    c = Case(BF16, 2, 64, 1, 8, 64, 16, [16, 8, 8], 64, seed=6, far=far)
    c.check(c.run())


def test_grid_stride_and_many_heads():
    """More tiles than resident blocks, and heads that one pass of a block does not cover."""
    c = Case(BF16, 1, 3001, 1, 8, 64, 16, [32], 64, seed=7, bad=False)
    c.check(c.run())
    c = Case(BF16, 2, 1300, 16, 8, 128, 16, [32, 16, 16], 128, seed=8, bad=False)
    c.check(c.run())


def test_frequencies_at_the_ends():
    """Zero, tiny, subnormal, large and negative frequencies; an infinite one poisons its own pair only."""
    c = Case(BF16, 1, 20, 1, 8, 64, 16, [8], 16, seed=9, far=4000)
    c.freq = np.array([0.0, 1e-40, 1e-20, 3.0e-7, 1.0, 6.0, -0.5, 100.5], dtype=np.float32)
    c.check(c.run())
    c.freq = np.array([0.1, np.inf, np.nan, 0.2, 0.3, 0.4, 0.5, 0.6], dtype=np.float32)
    out = c.run()[0].float()
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[1, 2, 9, 10]] = True
    live = torch.from_numpy(c.pos >= 0)
    assert torch.isnan(out[live][..., bad]).all() and torch.isfinite(out[live][..., ~bad]).all()


def test_nothing_to_do_and_all_skipped():
    c = Case(FP8, 2, 12, 2, 8, 128, 16, [64], 128, seed=10, bad=False)
    c.pos[:] = -1
    out, kp, vp, err = c.run()
    assert (out == 7.0).all() and torch.equal(kp, c.k_pool) and torch.equal(vp, c.v_pool) and err == 0
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    i = torch.int32
    da.rope_append(c.desc(), da.Rope.make(128), e(0, 2048), e(0, 256), e(0, 256), torch.ones(64, device="cuda"), e(1, 0, dt=i),
                   e(0, dt=i), torch.from_numpy(c.table).int().cuda(), e(0, 16, 128), kp.cuda(), vp.cuda(),
                   torch.ones(2, device="cuda"), torch.ones(2, device="cuda"), requests=e(0, dt=i))


def test_captured_and_replayed_on_another_stream():
    c = Case(BF16, 3, 40, 2, 8, 128, 16, [64], 128, seed=11)
    want = c.run()
    s = torch.cuda.Stream()
    got = c.run(stream=s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1].view(torch.uint8), want[1].view(torch.uint8))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
    n = c.H_q * c.D
    wide, kp, vp = c.wide.cuda(), c.k_pool.cuda(), c.v_pool.cuda()
    args = (da.Rope.make(128), wide[:, :n], wide[:, n:n + c.row], wide[:, n + c.row:], torch.from_numpy(c.freq).cuda(), t(c.at),
            t(c.pos), t(c.table), torch.full((c.N, c.H_q, c.D), 7.0, dtype=torch.bfloat16, device="cuda"), kp, vp)
    kw = dict(requests=t(c.req), device_error=torch.zeros(1, dtype=torch.int32, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.rope_append(c.desc(), *args, **kw)
    args[8].fill_(7.0)
    kp.copy_(c.k_pool.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[8].cpu(), want[0]) and torch.equal(kp.cpu().view(torch.uint8), want[1].view(torch.uint8))
