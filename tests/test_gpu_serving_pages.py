"""A beam search over drafts as a serving loop runs it on the device: fork, reserve,
copy, block append, schedule, attention, token probabilities, verification, with
nothing between the calls of a step; and each step checked against a float64
replica and the rows' own earlier contents."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from oracle.ops_ref import verify_ref
from oracle.serving_ref import adjusted, attend_ref, cached, probs_ref

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kv,kind,P,s_q,B", [(da.KV_FP8_BLOCK, "fp8", 16, 3, 5), (da.KV_INT8_BLOCK, "int8", 32, 2, 4), (da.KV_INT8_BLOCK, "int8", 64, 1, 3)])
def test_beams_with_drafts(kv, kind, P, s_q, B):
    H, V, cols, dev, K = 2, 400, 12, "cuda", s_q - 1
    pages = B * cols
    g = torch.Generator().manual_seed(P)
    desc = da.Desc.make(B=B, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=kv, s_q=s_q)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device=dev)
    poison = 0x7F if kind == "fp8" else 0x80
    kp, vp = (torch.full((pages, P, H, 128), poison, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.full((pages, H, P // 16), math.nan, device=dev) for _ in range(2))
    tables, held, lens = [torch.full((B, cols), -1, dtype=torch.int32, device=dev) for _ in range(2)], [_i32([0] * B) for _ in range(2)], [_i32([0] * B) for _ in range(2)]
    refs, copies, missing, err = _i32([0] * pages), _i32([[0, 0]] * B), _i32([0]), _i32([0])

    def append(n_rows, starts, table, pos):
        kv_new = torch.randn(n_rows, 2 * H * 128, generator=g).to(torch.bfloat16).cuda()
        da.append_block(desc, kv_new[:, :H * 128], kv_new[:, H * 128:], pos, table, kp, vp, ks, vs, token_starts=starts, device_error=err)
    # prompts: all rows of one prompt, taken in by row 0 and handed to the others by a fork
    n = 2 * P + 5
    da.reserve_pages(desc, lens[0], tables[0], held[0], refs, copies, missing, new_tokens=_i32([n] + [0] * (B - 1)), device_error=err)
    append(n, _i32([0] + [n] * B), tables[0], _i32([0] + [-1] * (B - 1)))
    lens[0][0] = n
    parents, now = [0] * B, 0
    texts = [torch.randint(0, V, (n,), generator=g).tolist()] * B
    prompt = [n] * B

    def contents(table, length):
        t, k, v, a, b = table.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(), ks.cpu().numpy(), vs.cpu().numpy()
        return [(cached(kind, k, a, t[r], L), cached(kind, v, b, t[r], L)) for r, L in enumerate(length)]
    for step in range(7):
        was = contents(tables[now], lens[now].tolist())
        then = 1 - now
        drafts = torch.randint(0, V, (B, K), generator=g).int()
        logits = torch.randn(B, s_q, V, generator=g) * 2
        if K:
            logits.scatter_(2, torch.cat([drafts, drafts[:, :1]], 1).long()[..., None], 6.0)
        texts, prompt = [texts[r] for r in parents], [prompt[r] for r in parents]
        hist = np.zeros((B, 200), np.int32)
        for b in range(B):
            hist[b, :len(texts[b])] = texts[b]
        u = torch.rand(B, s_q, generator=g)
        allowed = torch.randint(-2 ** 31, 2 ** 31, (B, s_q, (V + 31) // 32), generator=g).int() | torch.randint(-2 ** 31, 2 ** 31, (B, s_q, (V + 31) // 32), generator=g).int()
        q = torch.randn(B, s_q, 8 * H, 128, generator=g).to(torch.bfloat16)
        out, lse = torch.empty(B, s_q, 8 * H, 128, dtype=torch.bfloat16, device=dev), torch.empty(B, s_q, 8 * H, device=dev)
        probs, acc, toks = torch.empty(B, s_q, V, device=dev), _i32([0] * B), torch.empty(B, s_q, dtype=torch.int32, device=dev)
        temp, rep, pres = torch.full((B,), 0.8), torch.full((B,), 1.2), torch.full((B,), 0.3)
        dl, du, dd, dh, dn, dp, da_ = logits.cuda(), u.cuda(), drafts.cuda(), torch.from_numpy(hist).cuda(), _i32([len(t) for t in texts]), _i32(prompt), allowed.cuda()
        dt, dr, dpr, dq, par = temp.cuda(), rep.cuda(), pres.cuda(), q.cuda(), _i32(parents)
        torch.cuda.synchronize()
        # the step: nothing waits in it
        da.fork_pages(desc, par, lens[now], tables[now], held[now], refs, tables[then], held[then], lens[then], device_error=err)
        da.reserve_pages(desc, lens[then], tables[then], held[then], refs, copies, missing, device_error=err)
        da.copy_pages(desc, copies, kp, vp, k_scale=ks, v_scale=vs, device_error=err)
        append(B * s_q, None, tables[then], lens[then])
        seq = lens[then] + s_q
        da.sched_meta(desc, seq, meta)
        da.fwd(desc, dq, kp, vp, ks, vs, tables[then], seq, meta, out, lse)
        da.token_probs(dl, probs, temperature=dt, repetition=dr, presence=dpr, history=dh, history_lens=dn, prompt_lens=dp,
                       draft_tokens=dd if K else None, allowed=da_, device_error=err)
        da.verify_drafts(probs, None, dd if K else None, du, acc, toks, cache_seqlens=seq, new_seqlens=lens[then], device_error=err)
        torch.cuda.synchronize()
        assert int(err) == 0 and int(missing) == 0 and da.get_error(meta) == 0
        full = seq.tolist()
        got = contents(tables[then], full)
        t, r = tables[then].cpu().numpy(), refs.cpu().numpy()
        for b in range(B):
            L0 = full[b] - s_q
            a, c = was[parents[b]], got[b]
            assert len(a[0]) == L0
            # what the row had: its parent's, less a rounding where a block grew
            for x, y, scale in ((a[0], c[0], ks), (a[1], c[1], vs)):
                same = x == y[:L0]
                assert same[:L0 // 16 * 16].all()                        # whole blocks are as they were
                step_of = scale.cpu().numpy()[t[b, max(L0 - 1, 0) // P], :, max(L0 - 1, 0) % P // 16].astype(np.float64)
                assert (np.abs(x - y[:L0]) <= (step_of[:, None] * (0.5 if kind == "int8" else 16))).all()
            for j in range(L0 // P, -(-full[b] // P)):
                assert r[t[b, j]] == 1                                   # nobody else holds what was written to
            o, l, big, pv, sv = attend_ref(q[b].double().numpy().reshape(s_q, H, 8, 128), *c, s_q, 1 / math.sqrt(128))
            assert np.abs(lse[b].cpu().double().numpy().reshape(s_q, H, 8) - l).max() <= 1e-4
            tol = np.abs(o) * 2.0 ** -8 + pv * 2.0 ** -10 + sv * 2.0 ** -24 + 1e-30
            assert (np.abs(out[b].cpu().double().numpy().reshape(s_q, H, 8, 128) - o) <= tol).all()
            bits = np.unpackbits(allowed[b].numpy().view(np.uint8).reshape(s_q, -1), axis=-1, bitorder="little")[:, :V].astype(bool)
            for j in range(s_q):
                x = adjusted(logits[b, j].numpy(), np.float64, texts[b], prompt[b], drafts[b].tolist(), j, float(rep[b]), 0.0, float(pres[b]), [], V)
                p, _ = probs_ref(x, bits[j], float(temp[b]))
                assert np.abs(probs[b, j].cpu().double().numpy() - p).max() <= 1e-6
            n_acc, want, _ = verify_ref(probs[b].cpu().numpy(), None, drafts[b].tolist(), u[b].numpy(), V)
            assert int(acc[b]) == n_acc and toks[b].tolist() == want
            assert int(lens[then][b]) == L0 + 1 + n_acc
            texts[b] = texts[b] + want[:n_acc + 1]
        parents = torch.randint(0, B, (B,), generator=g).tolist()
        now = then


def test_calls_at_once_on_several_streams():
    """Appends, copies, probabilities and reservations of separate states on four streams, against the same in turn."""
    g = torch.Generator().manual_seed(1)
    B, P, H, cols = 6, 16, 2, 8
    desc = da.Desc.make(B=B, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=B * cols, kv_dtype=da.KV_INT8_BLOCK)
    x, logits = torch.randn(B * 40, 2 * H * 128, generator=g).to(torch.bfloat16).cuda(), torch.randn(64, 1, 70001, generator=g).cuda()

    def state():
        return dict(kp=torch.zeros(B * cols, P, H, 128, dtype=torch.uint8, device="cuda"), vp=torch.zeros(B * cols, P, H, 128, dtype=torch.uint8, device="cuda"),
                    ks=torch.zeros(B * cols, H, 1, device="cuda"), vs=torch.zeros(B * cols, H, 1, device="cuda"), table=torch.full((B, cols), -1, dtype=torch.int32, device="cuda"),
                    held=_i32([0] * B), refs=_i32([0] * (B * cols)), copies=_i32([[0, 0]] * B), missing=_i32([0]), probs=torch.empty_like(logits))

    zero, starts, need = _i32([0] * B), _i32([40 * b for b in range(B + 1)]), _i32([40] * B)

    def work(s, stream):
        for _ in range(5):
            da.reserve_pages(desc, zero, s["table"], s["held"], s["refs"], s["copies"], s["missing"], new_tokens=need, stream=stream)
            da.append_block(desc, x[:, :H * 128], x[:, H * 128:], zero, s["table"], s["kp"], s["vp"], s["ks"], s["vs"], token_starts=starts, stream=stream)
            da.copy_pages(desc, s["copies"], s["kp"], s["vp"], k_scale=s["ks"], v_scale=s["vs"], stream=stream)
            da.token_probs(logits, s["probs"], stream=stream)
    want, states, streams = state(), [state() for _ in range(4)], [torch.cuda.Stream() for _ in range(4)]
    work(want, None)
    torch.cuda.synchronize()
    for s, st in zip(states, streams):
        work(s, st)
    torch.cuda.synchronize()
    for s in states:
        assert all(torch.equal(s[k], want[k]) for k in want)
