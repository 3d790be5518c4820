"""The cache in 8 bits with a scale per block of 16 tokens and KV head: append
(bit for bit) and attention (within derived bounds) against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.serving_ref import T, append_block_ref, attend_ref, cached, codes_of, scale_for, values_of

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu
KIND = {da.KV_FP8_BLOCK: "fp8", da.KV_INT8_BLOCK: "int8"}
KINDS = [da.KV_FP8_BLOCK, da.KV_INT8_BLOCK]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(lens, P, cols, pages, seed):
    perm = np.random.RandomState(seed).permutation(pages)
    table, at = np.full((len(lens), cols), -7, np.int32), 0
    for b, L in enumerate(lens):
        n = -(-L // P)
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _filled(kind, pages, P, H, seed, spread=1.0, powers=True):
    """Codes and scales of a pool; every block has its own size."""
    g = np.random.RandomState(seed)
    x = g.randn(pages, P // T, T, H, 128) * np.exp(g.randn(pages, P // T, 1, H, 1) * spread)
    scale = np.abs(x).max((2, 4)) / (448 if kind == "fp8" else 127)
    scale = (np.exp2(np.ceil(np.log2(scale))) if powers else scale).astype(np.float32)
    codes = codes_of(x / scale[:, :, None, :, None].astype(np.float64), kind)
    return codes.reshape(pages, P, H, 128), np.ascontiguousarray(scale.transpose(0, 2, 1))


def _attend(kv, lens, H, P, s_q, splits=0, window=0, sinks=None, seed=0, spread=1.0, powers=True, q_scale=1.0, poison=True):
    """One call and its oracle; asserts the bounds."""
    kind, B = KIND[kv], len(lens)
    cols = max(1, -(-max(lens) // P)) + 1
    pages = sum(-(-L // P) for L in lens) + 2
    table = _table(lens, P, cols, pages, seed)
    (kc, ks), (vc, vs) = _filled(kind, pages, P, H, seed + 1, spread, powers), _filled(kind, pages, P, H, seed + 2, spread, powers)
    k_ref = [cached(kind, kc, ks, table[b], L) for b, L in enumerate(lens)]
    v_ref = [cached(kind, vc, vs, table[b], L) for b, L in enumerate(lens)]
    if poison:                      # whatever no token is on: codes of NaN (or the lowest), scales of NaN
        live = np.zeros((pages, P), bool)
        for b, L in enumerate(lens):
            for t in range(L):
                live[table[b, t // P], t % P] = True
        for c, s in ((kc, ks), (vc, vs)):
            c[~live] = 0x7F if kind == "fp8" else 0x80
            s.transpose(0, 2, 1)[~live.reshape(pages, P // T, T).any(-1)] = math.nan
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, s_q, 8 * H, 128, generator=g) * q_scale).to(torch.bfloat16)
    q = torch.where(q.abs() < 2.0 ** -14, 0, q)          # the others are exact in f16
    desc = da.Desc.make(B=B, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=kv,
                        s_q=s_q, splits=splits, window=window)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    out = torch.full((B, s_q, 8 * H, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, s_q, 8 * H), math.nan, device="cuda")
    dev = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs, table)]
    seq = _i32(lens)
    da.sched_meta(desc, seq, meta)
    da.fwd(desc, q.cuda(), *dev, seq, meta, out, lse, sinks=None if sinks is None else sinks.cuda())
    torch.cuda.synchronize()
    assert da.get_error(meta) == 0
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    sigma = 1 / math.sqrt(128)
    for b, L in enumerate(lens):
        o, l, big, pv, sv = attend_ref(q[b].double().numpy().reshape(s_q, H, 8, 128), k_ref[b], v_ref[b], s_q, sigma, window,
                                       None if sinks is None else sinks.double().numpy().reshape(H, 8))
        o, l, big, pv, sv = (x.reshape(s_q, 8 * H, *x.shape[3:]) for x in (o, l, big, pv, sv))
        # a score: up to 130 fp32 roundings of terms that add up to `big`
        eps = (130 + 2) * 2.0 ** -24 * big + 2.0 ** -22
        # the sum of weights: fp32, ex2 to 2 ulp; merging a few dozen partials
        sum_err = 2.0 ** -24 * (L / 8 + 256)
        assert np.array_equal(np.isneginf(l), np.isneginf(lse[b])), b
        fin = ~np.isneginf(l)
        assert (np.abs(lse[b] - l)[fin] <= (eps + sum_err + 2.0 ** -23 * np.abs(l))[fin]).all(), b
        # weights go to f16: half a step, 2^-11, or 2^-25 of the row's largest below 2^-14; then the sum in fp32 and bf16
        rel = 2.0 ** -11 + 2 * eps[..., None] + 2 * sum_err
        tol = np.abs(o) * 2.0 ** -8 * (1 + 2.0 ** -8) + pv * rel * 1.01 + sv * 2.0 ** -25 * 1.01 + 1e-38
        assert (np.abs(out[b] - o) <= tol).all(), (b, L, np.abs(out[b] - o).max(), (np.abs(out[b] - o) / tol).max())


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200, 333]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("P,H,s_q,splits", [(16, 1, 1, 0), (32, 3, 1, 1), (64, 2, 2, 0), (128, 1, 3, 3), (16, 2, 4, 8), (192, 1, 1, 2),
                                            (32, 1, 2, 5), (16, 3, 3, 0), (64, 1, 1, 0)])
def test_attention_matches_the_oracle(kv, P, H, s_q, splits):
    _attend(kv, LENS, H, P, s_q, splits, seed=P + s_q)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("P,s_q,window,sinks", [(16, 1, 40, True), (64, 2, 17, False), (32, 4, 100, True), (16, 3, 1, True), (128, 1, 0, True)])
def test_window_and_sinks(kv, P, s_q, window, sinks):
    g = torch.Generator().manual_seed(9)
    _attend(kv, LENS, 2, P, s_q, 0, window, torch.randn(16, generator=g) * 2 if sinks else None, seed=window + s_q)


@pytest.mark.parametrize("kv", KINDS)
def test_scales_that_are_no_powers_and_blocks_far_apart_in_size(kv):
    """Blocks of V whose scales are many orders apart: a large one with next to no weight must not cost the others their bits."""
    _attend(kv, [257, 64, 500], 2, 32, 1, seed=4, spread=4.0, powers=False, q_scale=0.05)
    _attend(kv, [257, 64, 500], 1, 16, 2, splits=3, seed=5, spread=6.0, powers=False, q_scale=0.01)


@pytest.mark.parametrize("kv", KINDS)
def test_longer_cache(kv):
    _attend(kv, [5000, 3001], 1, 64, 1, seed=6)
    _attend(kv, [5000, 3001], 1, 16, 4, seed=7)


def test_a_page_outside_the_pool_is_reported():
    desc = da.Desc.make(B=1, H_kv=1, G=8, D_qk=128, D_v=128, page_size=16, max_pages_per_seq=4, num_pages=4, kv_dtype=da.KV_FP8_BLOCK)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    pool, scale = z(4, 16, 1, 128, dtype=torch.uint8), z(4, 1, 1)
    out, lse = z(1, 8, 128, dtype=torch.bfloat16), z(1, 8)
    da.sched_meta(desc, _i32([40]), meta)
    da.fwd(desc, z(1, 8, 128, dtype=torch.bfloat16), pool, pool, scale, scale, _i32([[0, 4, 2, -1]]), _i32([40]), meta, out, lse)
    assert da.get_error(meta) == da.DA_DEV_BAD_PAGE
    err = _i32([0])
    row = z(40, 128, dtype=torch.bfloat16)
    da.append_block(desc, row, row, _i32([0]), _i32([[0, 4, 2, -1]]), pool, pool.clone(), scale, scale.clone(), token_starts=_i32([0, 40]),
                    device_error=err)
    assert int(err.item()) == da.DA_DEV_BAD_PAGE


# ------------------------------------------------------------------ append
def _append_case(kv, H, P, pages, cols, seed):
    g = np.random.RandomState(seed)
    kind = KIND[kv]
    (kc, ks), (vc, vs) = _filled(kind, pages, P, H, seed + 1), _filled(kind, pages, P, H, seed + 2)
    desc = da.Desc.make(B=1, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=kv)
    return g, kind, [kc, vc], [ks, vs], desc


def _check_append(desc, kind, pools, scales, k, v, starts, positions, table, err_want=0, packed=False, s_q=0):
    """Appends rows k, v (float32 torch [N, H, 128], exact in bf16) on the device and in the oracle: everything equal."""
    B = len(positions)
    d = da.Desc.make(B=B, H_kv=desc.H_kv, G=8, D_qk=128, D_v=128, page_size=desc.page_size, max_pages_per_seq=desc.max_pages_per_seq,
                     num_pages=desc.num_pages, kv_dtype=desc.kv_dtype, s_q=max(1, s_q))
    want = append_block_ref(kind, pools, scales, [k.double().numpy(), v.double().numpy()], starts, positions, table)
    dev = [torch.from_numpy(x).cuda() for x in pools + scales]
    n, H = k.shape[0], desc.H_kv
    if packed:
        kd, vd = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
    else:       # columns of one projection output
        x = torch.cat([torch.full((n, 8), 7.0), k.view(n, -1), v.view(n, -1)], 1).to(torch.bfloat16).cuda()
        kd, vd = x[:, 8:8 + 128 * H], x[:, 8 + 128 * H:]
    err = _i32([0])
    da.append_block(d, kd, vd, _i32(positions), torch.from_numpy(table).cuda(), *dev, token_starts=None if s_q else _i32(starts),
                    device_error=err)
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in dev]
    assert int(err.item()) == want[2] == err_want
    for a, b in zip(got, want[0] + want[1]):
        assert np.array_equal(a, b, equal_nan=a.dtype != np.uint8)
    return got[:2], got[2:]


def _rows(g, n, H, spread=1.0):
    x = g.randn(n, H, 128) * np.exp(g.randn(n, H, 1) * spread)
    return torch.from_numpy(x).to(torch.bfloat16).float()


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("P,H", [(16, 1), (32, 3), (64, 2), (192, 1)])
def test_ragged_prompts_are_appended_bit_for_bit(kv, P, H):
    counts, pos = [1, 0, 77, 16, 300, 3, 15, 33], [0, 5, 3, 16, 17, 14, 1, 48]
    cols, B = -(-330 // P) + 1, len(counts)
    pages = sum(-(-(p + c) // P) for p, c in zip(pos, counts)) + 3
    table = _table([p + c for p, c in zip(pos, counts)], P, cols, pages, P)
    g, kind, pools, scales, desc = _append_case(kv, H, P, pages, cols, P)
    starts = np.concatenate([[0], np.cumsum(counts)]).tolist()
    for packed in (False, True):
        _check_append(desc, kind, pools, scales, _rows(g, starts[-1], H), _rows(g, starts[-1], H), starts, pos, table, packed=packed)
    assert B == len(pos)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("s_q", [1, 2, 4, 17])
def test_tokens_step_by_step_grow_their_blocks(kv, s_q):
    """s_q tokens a request and step, without row bounds, across block and page ends; one request sits out."""
    B, P, H, cols = 4, 32, 2, 6
    table = _table([cols * P] * B, P, cols, B * cols, 3)
    g, kind, pools, scales, desc = _append_case(kv, H, P, B * cols, cols, 3)
    pos = [0, 13, 31, -1]
    for step in range(60 // s_q):
        n = B * s_q
        pools, scales = _check_append(desc, kind, pools, scales, _rows(g, n, H, 2.0), _rows(g, n, H, 2.0), [b * s_q for b in range(B + 1)],
                                      pos, table, s_q=s_q)
        pos = [p + s_q if p >= 0 else p for p in pos]


@pytest.mark.parametrize("kv", KINDS)
def test_values_that_are_not_ordinary(kv):
    """NaN and infinities, zeros, the smallest and the largest magnitudes, blocks of maxima at a scale's border; after rows
    of ordinary ones, so that their codes go down many steps at once."""
    P, H, cols = 32, 2, 8
    table = _table([cols * P], P, cols, cols, 1)
    g, kind, pools, scales, desc = _append_case(kv, H, P, cols, cols, 1)
    q = 448.0 if kind == "fp8" else 127.0
    n = 100
    x = _rows(g, n, H)
    x[0:20] = 0
    x[20, 0, 5], x[21, 1, 7], x[22, 0, 9] = math.nan, math.inf, -math.inf
    x[32:48] = 0
    x[33] = torch.where(torch.arange(128) % 2 == 0, q, -q / 2)
    x[50, 0, 3] = 3e38
    x[64:80] *= 2.0 ** -130
    x[80:96] = 2.0 ** -133
    x = x.to(torch.bfloat16).float()
    for pos in (0, 3, 16, 29):
        p, s = _check_append(desc, kind, pools, scales, x, x.flip(0), [0, n], [pos], table)
        for k in range(3):       # and on behind it, token by token
            y = _rows(g, 1, H, 20.0)
            p, s = _check_append(desc, kind, p, s, y, -y, [0, 1], [pos + n + k], table)


@pytest.mark.parametrize("kv", KINDS)
def test_scales_of_a_users_own_and_tokens_that_do_not_fit(kv):
    P, H, cols = 16, 1, 3
    table = _table([cols * P] * 2, P, cols, 2 * cols, 1)
    table[1, 1] = 99
    g, kind, pools, scales, desc = _append_case(kv, H, P, 2 * cols, cols, 1)
    scales = [(s * np.float32(1.37)) for s in scales]     # no powers of two
    # request 0 runs past its table, request 1 over a page outside the pool
    _check_append(desc, kind, pools, scales, _rows(g, 80, H, 0.1), _rows(g, 80, H, 0.1), [0, 40, 80], [20, 4], table, err_want=3)


def test_appends_and_attention_captured_and_replayed():
    """A captured step (append of one token, schedule, attention) replayed along a growing cache, against eager calls."""
    B, P, H, cols, dev = 3, 16, 2, 8, "cuda"
    desc = da.Desc.make(B=B, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=B * cols, kv_dtype=da.KV_INT8_BLOCK)
    table = torch.from_numpy(_table([cols * P] * B, P, cols, B * cols, 8)).cuda()
    g = torch.Generator().manual_seed(8)
    qkv = torch.randn(40, B, 10 * H * 128, generator=g).to(torch.bfloat16).cuda()

    def state():
        pools = [torch.zeros(B * cols, P, H, 128, dtype=torch.uint8, device=dev) for _ in range(2)]
        scales = [torch.zeros(B * cols, H, P // 16, device=dev) for _ in range(2)]
        return dict(pools=pools, scales=scales, x=torch.empty_like(qkv[0]), pos=_i32([0, 3, 17]), seq=_i32([1, 4, 18]),
                    meta=torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device=dev),
                    out=torch.zeros(B, 8 * H, 128, dtype=torch.bfloat16, device=dev), lse=torch.zeros(B, 8 * H, device=dev))

    def step(s):
        x = s["x"]
        da.append_block(desc, x[:, 8 * H * 128:9 * H * 128], x[:, 9 * H * 128:], s["pos"], table, *s["pools"], *s["scales"])
        da.sched_meta(desc, s["seq"], s["meta"])
        da.fwd(desc, x[:, :8 * H * 128].contiguous().view(B, 8 * H, 128), *s["pools"], *s["scales"], table, s["seq"], s["meta"], s["out"], s["lse"])
        s["pos"].add_(1)
        s["seq"].add_(1)
    a, b = state(), state()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(a)
    for t in range(40):
        a["x"].copy_(qkv[t])
        b["x"].copy_(qkv[t])
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    assert all(torch.equal(x, y) for x, y in zip(a["pools"] + a["scales"], b["pools"] + b["scales"]))


def test_scale_for_is_the_kernels_rule():
    """Every border between two scales, both sides of it, as one block's largest value."""
    for kv in KINDS:
        kind = KIND[kv]
        q = 448.0 if kind == "fp8" else 127.0
        vals = []
        for e in (-120, -30, -1, 0, 3, 100):
            for f in (q, q * (1 + 2.0 ** -7), q * (1 - 2.0 ** -7)):
                vals.append(f * 2.0 ** e)
        x = torch.tensor(vals).to(torch.bfloat16).float()
        n = len(vals)
        rows = torch.zeros(16 * n, 1, 128)
        rows[::16, 0, 77] = x
        pools = [np.zeros((n, 16, 1, 128), np.uint8) for _ in range(2)]
        scales = [np.zeros((n, 1, 1), np.float32) for _ in range(2)]
        table = np.arange(n, dtype=np.int32)[None]
        desc = da.Desc.make(B=1, H_kv=1, G=8, D_qk=128, D_v=128, page_size=16, max_pages_per_seq=n, num_pages=n, kv_dtype=kv)
        _, s = _check_append(desc, kind, pools, scales, rows, rows, [0, 16 * n], [0], table)
        assert [float(v) for v in s[0][:, 0, 0]] == [scale_for(float(v), kind) for v in x]
        assert values_of(np.array([0x7E], np.uint8), "fp8") == 448


def test_pools_beyond_4_gib():
    """Pages whose codes lie past 2^32 bytes, whose scales' indexes stay apart: append, copy and attention there."""
    P, H, kv = 64, 8, da.KV_INT8_BLOCK
    pages = (1 << 32) // (P * H * 128) + 40
    kp, vp = (torch.empty(pages, P, H, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, H, P // 16, device="cuda") for _ in range(2))
    desc = da.Desc.make(B=2, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=4, num_pages=pages, kv_dtype=kv)
    table = _i32([[pages - 1, 3, pages - 2, pages - 3], [5, pages - 4, 7, pages - 5]])
    g = np.random.RandomState(2)
    x, y = _rows(g, 400, H), _rows(g, 400, H)
    da.append_block(desc, x.to(torch.bfloat16).cuda(), y.to(torch.bfloat16).cuda(), _i32([0, 0]), table, kp, vp, ks, vs, token_starts=_i32([0, 200, 400]))
    moved = _i32([[pages - 1, pages - 10], [3, pages - 11], [pages - 2, 9], [pages - 3, 11]])
    da.copy_pages(desc, moved, kp, vp, k_scale=ks, v_scale=vs)
    q = torch.randn(2, 8 * H, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    seq, outs = _i32([200, 200]), []
    for t in (table, torch.cat([moved[:, 1][None], table[1:]]).contiguous()):
        out, lse = torch.empty(2, 8 * H, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8 * H, device="cuda")
        da.sched_meta(desc, seq, meta)
        da.fwd(desc, q, kp, vp, ks, vs, t, seq, meta, out, lse)
        outs.append((out, lse))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for b in range(2):
        # int8 with power-of-two scales of whole blocks: at most half a step of up to 2 max / 127
        for pool, scale, v in ((kp, ks, x), (vp, vs, y)):
            rows = pool[table[b].long()].view(torch.int8).double().view(256, H, 128)[:200]
            sc = scale[table[b].long()].double().transpose(1, 2).reshape(16, H).repeat_interleave(16, 0)[:200]
            assert ((rows * sc[..., None]).cpu() - v[200 * b:200 * b + 200].double()).abs().max() <= 0.5 * sc.max().cpu()
    assert torch.isfinite(outs[0][0].float()).all()


def test_without_a_caller_s_scratch():
    """The allocation-free call takes the block formats too, with the same bits."""
    B, P, H, cols, kv = 2, 16, 1, 8, da.KV_FP8_BLOCK
    kind = "fp8"
    (kc, ks), (vc, vs) = _filled(kind, B * cols, P, H, 1), _filled(kind, B * cols, P, H, 2)
    dev = [torch.from_numpy(x).cuda() for x in (kc, vc, ks, vs)]
    table, seq = torch.from_numpy(_table([cols * P] * B, P, cols, B * cols, 4)).cuda(), _i32([100, 37])
    desc = da.Desc.make(B=B, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=B * cols, kv_dtype=kv, splits=4)
    q = torch.randn(B, 8, 128, device="cuda").to(torch.bfloat16)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    o = [torch.empty(B, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    l = [torch.empty(B, 8, device="cuda") for _ in range(2)]
    da.sched_meta(desc, seq, meta)
    da.fwd(desc, q, *dev, table, seq, meta, o[0], l[0])
    da.fwd_static_scratch(desc, q, *dev, table, seq, o[1], l[1])
    assert torch.equal(o[0], o[1]) and torch.equal(l[0], l[1])
