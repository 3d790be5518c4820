"""The operators as a serving loop runs them, on one stream without a
synchronisation between them: rotary append of a prompt, then steps of rotary
append of a draft chain, schedule, attention, verification of the chain,
accumulation with the accepted rows, and an eviction onto other pages with the
loop going on behind it. Every step is checked against a float64 replica kept
on the host from the device's own values, so that nothing drifts."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.ops_ref import accum_ref, evict_select, rope_ref, verify_ref

from gpu_util import LSE_TOL, OUT_TOL, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _read(pool, table, L, P):
    return pool[table[:-(-L // P)].long()].flatten(0, 1)[:L].double().cpu()


@pytest.mark.parametrize("H_kv,D,P,s_q", [(2, 64, 16, 3), (1, 128, 32, 2)])
def test_steps_with_verification_accumulation_and_eviction(H_kv, D, P, s_q):
    B, G, V, budget = 3, 8, 500, 40
    H_q, cols, dev = H_kv * G, 8, "cuda"
    g = torch.Generator().manual_seed(D)
    num_pages = 2 * B * cols
    perm = torch.randperm(num_pages, generator=g).int()
    table, spare = perm[:B * cols].view(B, cols).clone().cuda(), perm[B * cols:].view(B, cols).clone().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    kp = torch.full((num_pages, P, H_kv, D), math.nan, dtype=torch.bfloat16, device=dev)
    vp = torch.full_like(kp, math.nan)
    weights = torch.full((num_pages, H_kv, P), math.nan, device=dev)
    sections = [D // 4, D // 8, D // 8]
    rope = da.Rope.make(D, sections)
    freq = (1000.0 ** (-torch.arange(D // 2) / (D // 2))).float()
    base = dict(B=B, H_kv=H_kv, G=G, D_qk=D, D_v=D, page_size=P, max_pages_per_seq=cols, num_pages=num_pages)
    desc = da.Desc.make(**base, s_q=s_q)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device=dev)
    err = i32([0])

    def append(req, pos, where):
        """Rotary append of tokens (request, slot, position in the text); returns the rotated q."""
        n = len(req)
        qkv = torch.randn(n, (H_q + 2 * H_kv) * D, generator=g).to(torch.bfloat16)
        at = torch.tensor([where, [w // 3 for w in where], [w % 3 for w in where]], dtype=torch.int32)
        x, q_out = qkv.cuda(), torch.empty(n, H_q, D, dtype=torch.bfloat16, device=dev)
        da.rope_append(desc, rope, x[:, :H_q * D], x[:, H_q * D:(H_q + H_kv) * D], x[:, (H_q + H_kv) * D:], freq.cuda(), at.cuda(),
                       i32(pos), table, q_out, kp, vp, requests=i32(req), device_error=err)
        want, mag = rope_ref(qkv[:, :H_q * D].double().numpy().reshape(n, H_q, D), at.numpy(), freq.numpy(), sections, 0, 0)
        assert (np.abs(q_out.cpu().double().numpy() - want) <= mag * 2.0 ** -20 + np.abs(want) * 2.0 ** -8).all()
        return q_out

    lens = [29, 3, 61]                                    # prompts, ragged, in one call
    append([b for b in range(B) for _ in range(lens[b])], [t for b in range(B) for t in range(lens[b])],
           [t for b in range(B) for t in range(lens[b])])
    text, weighted, chosen = list(lens), [0] * B, 0
    for step in range(4):
        drafts = torch.randint(0, V, (B, s_q - 1), generator=g).int()
        q = append([b for b in range(B) for _ in range(s_q)], [lens[b] + j for b in range(B) for j in range(s_q)],
                   [text[b] + j for b in range(B) for j in range(s_q)]).view(B, s_q, H_q, D)
        full = [n + s_q for n in lens]
        seq, before = i32(full), weights.cpu().double()
        out, lse = torch.empty(B, s_q, H_q, D, dtype=torch.bfloat16, device=dev), torch.empty(B, s_q, H_q, device=dev)
        p = torch.softmax(torch.randn(B, s_q, V, generator=g) * 2, -1)
        p.scatter_(2, torch.cat([drafts, drafts[:, :1]], 1).long()[..., None], 0.4)
        u, acc, toks, new = torch.rand(B, s_q, generator=g), i32([0] * B), torch.empty(B, s_q, dtype=torch.int32, device=dev), i32([0] * B)
        da.sched_meta(desc, seq, meta)
        da.fwd(desc, q, kp, vp, None, None, table, seq, meta, out, lse)
        da.verify_drafts(p.cuda(), None, drafts.cuda(), u.cuda(), acc, toks, cache_seqlens=seq, new_seqlens=new, device_error=err)
        da.accum_weights(desc, q, kp, None, table, seq, meta, lse, weights, num_accepted=acc, weighted_lens=i32(weighted))
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and da.get_error(meta) == 0
        ks = [_read(kp, table[b], full[b], P) for b in range(B)]
        vs = [_read(vp, table[b], full[b], P) for b in range(B)]
        for b in range(B):                                # the attention itself
            for j in range(s_q):
                n = full[b] - s_q + 1 + j
                s = torch.einsum("hgd,thd->hgt", q[b, j].double().cpu().view(H_kv, G, D), ks[b][:n]) / math.sqrt(D)
                assert (lse[b, j].cpu().double() - s.logsumexp(-1).flatten()).abs().max() <= LSE_TOL
                o = torch.einsum("hgt,thd->hgd", s.softmax(-1), vs[b][:n]).reshape(H_q, D)
                assert (out[b, j].cpu().double() - o).abs().max() <= OUT_TOL
            a, want, _ = verify_ref(p[b].numpy(), None, drafts[b].tolist(), u[b].numpy(), V)
            assert int(acc[b]) == a and toks[b].tolist() == want and int(new[b]) == full[b] - s_q + 1 + a
        add, _ = accum_ref(q.double().cpu().numpy().reshape(B, s_q, H_kv, G, D), lambda b: ks[b].numpy(), full,
                           lse.cpu().double().numpy().reshape(B, s_q, H_kv, G), 1 / math.sqrt(D), s_q, acc.tolist())
        for b in range(B):
            for t in range(full[b]):
                at = (int(table[b, t // P]), slice(None), t % P)
                old = before[at] if t < weighted[b] else 0.0
                assert torch.allclose(weights[at].cpu().double(), old + torch.from_numpy(add[b][t]), rtol=1e-4, atol=0)
        lens = new.tolist()
        text = [text[b] + lens[b] - full[b] + s_q for b in range(B)]
        weighted = lens
        if step in (1, 2):                                # cut back, and go on behind it
            kept, cut = torch.empty(B, H_kv, budget, dtype=torch.int32, device=dev), i32([0] * B)
            was = [[w for w in weights.cpu()[table[b].cpu().long()].transpose(1, 2).flatten(0, 1)[:lens[b]].T] for b in range(B)]
            old_k = [_read(kp, table[b], lens[b], P) for b in range(B)]
            da.evict(desc, budget, new, table, spare, kp, vp, weights, kept, cut, keep_first=2, keep_last=6, device_error=err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0 and cut.tolist() == [min(n, budget) for n in lens]
            for b in range(B):
                now = _read(kp, spare[b], int(cut[b]), P)
                for h in range(H_kv):
                    want = evict_select(was[b][h].numpy(), budget, 2, 6)
                    assert kept[b, h, :len(want)].tolist() == want
                    assert torch.equal(now[:, h], old_k[b][want, h])
                    chosen += lens[b] > budget
            table, spare = spare, table
            lens = cut.tolist()
            weighted = lens
    assert chosen                                         # some request was over its budget


def test_latent_steps_with_accumulation_and_eviction():
    """The same on the 656-byte format: the weights that its eviction goes by come from its own attention."""
    B, P, cols, s_q, budget, dev = 2, 16, 12, 2, 100, "cuda"
    g = torch.Generator().manual_seed(5)
    num_pages = 2 * B * cols
    perm = torch.randperm(num_pages, generator=g).int()
    table, spare = perm[:B * cols].view(B, cols).clone().cuda(), perm[B * cols:].view(B, cols).clone().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    pool = torch.full((num_pages, P, 1, 656), 0xFF, dtype=torch.uint8, device=dev)
    weights = torch.full((num_pages, 1, P), math.nan, device=dev)
    rope, freq = da.Rope.make(64), (1000.0 ** (-torch.arange(32) / 32)).float().cuda()
    desc = da.Desc.make(B=B, H_kv=1, G=128, D_qk=576, D_v=512, page_size=P, max_pages_per_seq=cols, num_pages=num_pages,
                        kv_dtype=da.KV_MLA656, s_q=s_q)
    meta, err = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device=dev), i32([0])

    def append(req, pos):
        n = len(req)
        x = torch.randn(n, 129 * 576, generator=g).to(torch.bfloat16).cuda()
        q_out = torch.empty(n, 128, 576, dtype=torch.bfloat16, device=dev)
        da.rope_append(desc, rope, x[:, :128 * 576], x[:, 128 * 576:], None, freq, i32([pos]), i32(pos), table, q_out, pool,
                       None, requests=i32(req), device_error=err)
        return q_out

    def rows(tab, L):
        raw = pool[tab[:-(-L // P)].long()].flatten(0, 2)[:L].cpu()
        scale = raw[:, 512:528].contiguous().view(torch.float32).repeat_interleave(128, -1)
        nope = (raw[:, :512].contiguous().view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16).double()
        return torch.cat([nope, raw[:, 528:].contiguous().view(torch.bfloat16).double()], -1), raw

    lens, weighted = [150, 61], [0, 0]
    append([b for b in range(B) for _ in range(lens[b])], [t for b in range(B) for t in range(lens[b])])
    for step in range(3):
        q = append([b for b in range(B) for _ in range(s_q)], [lens[b] + j for b in range(B) for j in range(s_q)])
        q = q.view(B, s_q, 128, 576)
        lens = [n + s_q for n in lens]
        seq, before = i32(lens), weights.cpu().double()
        out, lse = torch.empty(B, s_q, 128, 512, dtype=torch.bfloat16, device=dev), torch.empty(B, s_q, 128, device=dev)
        da.sched_meta(desc, seq, meta)
        da.fwd(desc, q, pool, None, None, None, table, seq, meta, out, lse)
        da.accum_weights(desc, q, pool, None, table, seq, meta, lse, weights, weighted_lens=i32(weighted), decay=0.5)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and da.get_error(meta) == 0
        for b in range(B):
            k, _ = rows(table[b], lens[b])
            add = torch.zeros(lens[b], dtype=torch.float64)
            for j in range(s_q):
                n = lens[b] - s_q + 1 + j
                s = q[b, j].double().cpu() @ k[:n].T / 24.0
                assert (lse[b, j].cpu().double() - s.logsumexp(-1)).abs().max() <= LSE_TOL
                assert (out[b, j].cpu().double() - s.softmax(-1) @ k[:n, :512]).abs().max() <= OUT_TOL
                add[:n] += (s - lse[b, j].cpu().double()[:, None]).exp().sum(0)
            for t in range(lens[b]):
                at = (int(table[b, t // P]), 0, t % P)
                old = float(before[at]) / 2 if t < weighted[b] else 0.0
                assert math.isclose(float(weights[at]), old + float(add[t]), rel_tol=1e-4)
        weighted = lens
        if step == 1:
            kept, cut = torch.empty(B, 1, budget, dtype=torch.int32, device=dev), i32([0] * B)
            was = [weights.cpu()[table[b].cpu().long(), 0].flatten()[:lens[b]] for b in range(B)]
            old = [rows(table[b], lens[b])[1] for b in range(B)]
            da.evict(desc, budget, seq, table, spare, pool, None, weights, kept, cut, keep_first=2, keep_last=6, device_error=err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0 and cut.tolist() == [min(n, budget) for n in lens]
            for b in range(B):
                want = evict_select(was[b].numpy(), budget, 2, 6)
                assert kept[b, 0, :len(want)].tolist() == want
                assert torch.equal(rows(spare[b], int(cut[b]))[1], old[b][want])
            table, spare, lens, weighted = spare, table, cut.tolist(), cut.tolist()
