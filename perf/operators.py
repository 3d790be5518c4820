"""What the operators around the paged decode attention cost: rotary positions
with several axes fused with the KV append, the attention weight that each
cached token has gathered, eviction by that weight, and the verification of
drafted tokens.

``own`` false: the plain form of each in elementary torch operations. ``own``
true: the library's entry points, called as a serving loop calls them.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
NOPE, ROPE, TOKEN = 512, 64, 656      # the latent token: 512 e4m3 | 4 fp32 scales | 64 bf16
STEP = 2.0 ** 44                      # verification weighs probabilities in steps of 2^-44


# --------------------------------------------------------------------- cases
# kv: bf16, fp8 (e4m3, one scale per head) or latent (656-byte tokens).
def listed():
    return [
        # rotary + append: one new token of one request (the smallest call: latency)
        dict(name="rope_step", op="rope", kv="bf16", B=1, tokens=1, H_q=8, H_kv=1, D=64, P=16, rot=64,
             axes="12,10,10", mix=0, adjacent=0, far=256),
        # a chain of four drafts of each of 64 requests into an e4m3 cache, far positions, half of each head rotated
        dict(name="rope_chain_fp8", op="rope", kv="fp8", B=64, tokens=256, H_q=32, H_kv=4, D=128, P=32, rot=64,
             axes="12,10,10", mix=1, adjacent=1, far=32768),
        # two drafts a request on the latent format: 128 heads' RoPE part and the shared token
        dict(name="rope_chain_latent", op="rope", kv="latent", B=32, tokens=64, H_q=128, H_kv=1, D=576, P=64, rot=64,
             axes="32", mix=0, adjacent=1, far=131072),
        # ragged prompts (text, images, video) of 8 requests appended in one call: bandwidth
        dict(name="rope_prompts", op="rope", kv="bf16", B=8, tokens=32771, H_q=64, H_kv=8, D=128, P=64, rot=128,
             axes="16,24,24", mix=0, adjacent=0, far=8192),
        # weights gathered by one new token over a short cache (latency)
        dict(name="accum_step", op="accum", kv="bf16", B=1, H_q=8, H_kv=1, D=64, P=16, lo=256, hi=256, s_q=1, decay=1.0, splits=1),
        # a chain of two drafts, part of them accepted, over mixed lengths
        dict(name="accum_mixed_chain", op="accum", kv="bf16", B=32, H_q=64, H_kv=8, D=128, P=64, lo=1024, hi=8192, s_q=2,
             decay=1.0, splits=0),
        # a large batch of long e4m3 caches: bandwidth
        dict(name="accum_fp8_long", op="accum", kv="fp8", B=64, H_q=32, H_kv=4, D=128, P=32, lo=32768, hi=32768, s_q=1,
             decay=0.96875, splits=0),
        # eviction: a few short caches cut to a third (latency)
        dict(name="evict_short", op="evict", kv="bf16", B=8, H_kv=4, D=64, P=256, lo=1536, hi=1536, budget=512, first=4, last=64),
        # mixed lengths, some under the budget, cut in the middle of a page
        dict(name="evict_mixed", op="evict", kv="bf16", B=32, H_kv=8, D=128, P=64, lo=1024, hi=8192, budget=2047, first=4, last=256),
        # two long latent caches: few rows, long selection
        dict(name="evict_latent_long", op="evict", kv="latent", B=2, H_kv=1, D=576, P=64, lo=100003, hi=131072, budget=32768, first=1,
             last=1024),
        # verification of one request's drafts (latency)
        dict(name="verify_one", op="verify", dtype="f32", B=1, drafts=3, V=32000, has_q=1),
        # a batch with an odd vocabulary
        dict(name="verify_batch", op="verify", dtype="f32", B=128, drafts=3, V=128259, has_q=1),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "accum", "evict", "verify"])
    if op == "rope":
        kv = rng.choice(["bf16", "fp8", "latent"])
        B = _spread(rng, 1, 64)
        tokens = max(B, _spread(rng, 1, 2048 if kv == "latent" else 16384))
        if kv == "latent":
            H_q, H_kv, D, rot = 128, 1, 576, 64
        else:
            H_kv = rng.choice([1, 2, 3, 4, 8])
            H_q, D = 8 * H_kv, rng.choice([64, 96, 128])
            rot = rng.choice([D, D // 2])
        n = rot // 2
        if rng.random() < 0.5:
            axes = str(n)
        else:
            b, c = rng.randint(1, n // 3), rng.randint(1, n // 3)
            axes = "%d,%d,%d" % (n - b - c, b, c)
        return dict(op=op, kv=kv, B=B, tokens=tokens, H_q=H_q, H_kv=H_kv, D=D, P=rng.choice([8, 16, 32, 64, 256]), rot=rot,
                    axes=axes, mix=rng.randint(0, 1), adjacent=rng.randint(0, 1), far=_spread(rng, 16, 1 << 20))
    if op == "accum":
        kv = rng.choice(["bf16", "fp8"])
        H_kv = rng.choice([1, 2, 3, 4, 8])
        hi = _spread(rng, 1, 32768)
        B = _spread(rng, 1, max(1, min(64, (1 << 21) // (hi * H_kv))))
        return dict(op=op, kv=kv, B=B, H_q=8 * H_kv, H_kv=H_kv, D=128 if kv == "fp8" else rng.choice([64, 128]),
                    P=rng.choice([8, 16, 32, 64, 128]), lo=max(1, int(hi * rng.uniform(0.1, 1))), hi=hi, s_q=rng.randint(1, 4),
                    decay=rng.choice([1.0, 0.5, 0.96875]), splits=rng.choice([0, 0, 1, 3, 8]))
    if op == "evict":
        kv = rng.choice(["bf16", "fp8", "latent"])
        H_kv = 1 if kv == "latent" else rng.choice([1, 2, 3, 4, 8])
        hi = _spread(rng, 16, 65536)
        B = _spread(rng, 1, max(1, min(64, (1 << 20) // (hi * H_kv))))
        budget = max(2, int(hi * rng.uniform(0.05, 1)))
        first = rng.randint(0, budget // 4)
        return dict(op=op, kv=kv, B=B, H_kv=H_kv, D=576 if kv == "latent" else rng.choice([64, 96, 128]),
                    P=rng.choice([8, 16, 32, 64, 256]), lo=max(1, int(hi * rng.uniform(0.1, 1))), hi=hi, budget=budget, first=first,
                    last=rng.randint(0, budget - first))
    return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), B=_spread(rng, 1, 128), drafts=rng.choice([0, 1, 2, 3, 5, 7]),
                V=_spread(rng, 1000, 131072), has_q=rng.randint(0, 1))


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, seed):
    r = random.Random(seed * 7919 + 1)
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _pages(lens, P, seed, columns, lo, hi):
    """A block table of shuffled pages out of [lo, hi) for these lengths."""
    need = [-(-n // P) for n in lens]
    perm = np.random.RandomState(seed % (1 << 31)).permutation(hi - lo) + lo
    table = np.full((len(lens), columns), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _quant(x, scale):
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(g, kv, pages, P, H, D):
    """A filled cache: K, V and their scales."""
    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    if kv == "bf16":
        return [torch.randn(pages, P, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)] + [None, None]
    if kv == "fp8":
        scale = [torch.rand(H, generator=g, device="cuda") * 0.004 + 0.01 for _ in range(2)]
        out = []
        for s in scale:
            pool = torch.empty(pages, P, H, D, device="cuda", dtype=torch.uint8)
            for lo in range(0, pages, 4096):
                hi = min(pages, lo + 4096)
                pool[lo:hi] = _quant(normal(hi - lo, P, H, D), s.view(H, 1))
            out.append(pool)
        return out + scale
    pool = torch.empty(pages, P, 1, TOKEN, device="cuda", dtype=torch.uint8)
    x = normal(pages, P, 1, NOPE + ROPE)
    block = x[..., :NOPE].reshape(pages, P, 1, 4, 128)
    scale = block.abs().amax(-1) / E4M3_MAX
    pool[..., :NOPE] = _quant(block, scale[..., None]).reshape(pages, P, 1, NOPE)
    pool[..., NOPE:NOPE + 16] = scale.view(torch.uint8)
    pool[..., NOPE + 16:] = x[..., NOPE:].to(torch.bfloat16).view(torch.uint8)
    return [pool, None, None, None]


def _axis_of_pair(case):
    sections = [int(x) for x in case["axes"].split(",")]
    n, A = case["rot"] // 2, len(sections)
    if case["mix"]:
        return [i % A if i // A < sections[i % A] else 0 for i in range(n)], sections
    return [a for a, m in enumerate(sections) for _ in range(m)], sections


def _prepare_rope(case, seed):
    g, r = _gen(seed), random.Random(seed)
    B, N, H_q, H_kv, D, P = (case[k] for k in ("B", "tokens", "H_q", "H_kv", "D", "P"))
    latent = case["kv"] == "latent"
    cuts = [0] + sorted(r.sample(range(1, N), B - 1)) + [N]
    counts = [b - a for a, b in zip(cuts, cuts[1:])]                 # new tokens of each request, ragged
    history = [r.randint(0, max(0, min(case["far"], 4096))) for _ in range(B)]
    pages = -(-(N + B * min(case["far"], 4096)) // P) + B            # room for whatever the seed gives
    table = _pages([h + c for h, c in zip(history, counts)], P, seed, -(-(N + 4096) // P), 0, pages)
    req = np.repeat(np.arange(B), counts)
    pos = np.concatenate([h + np.arange(c) for h, c in zip(history, counts)])
    axis, sections = _axis_of_pair(case)
    at = r.randint(0, case["far"]) + torch.from_numpy(pos)[None, :].repeat(len(sections), 1)
    for a in range(1, len(sections)):                                # rows and columns of images between the text
        at[a] = at[a] // 16 + at[a] % (8 * a + 5)
    width = D if latent else H_kv * D
    qkv = torch.randn(N, H_q * D + (1 if latent else 2) * width, generator=g, device="cuda", dtype=torch.bfloat16)
    k_pool, v_pool, k_scale, v_scale = _pool(g, case["kv"], pages, P, H_kv, D)
    n = case["rot"] // 2
    inv_freq = (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda()
    s = dict(case=case, q=qkv[:, :H_q * D], k=qkv[:, H_q * D:H_q * D + width], v=None if latent else qkv[:, H_q * D + width:],
             stride=qkv.shape[1], inv_freq=inv_freq, at=at.int().contiguous().cuda(), req=torch.from_numpy(req).int().cuda(),
             pos=torch.from_numpy(pos).int().cuda(), axis=torch.tensor(axis, device="cuda"), sections=sections,
             table=torch.from_numpy(table).cuda(), k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale,
             q_out=torch.empty(N, H_q, D, device="cuda", dtype=torch.bfloat16))
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, table.shape[1], pages)
        s["rope"] = da.Rope.make(case["rot"], sections, interleaved=bool(case["mix"]), adjacent=bool(case["adjacent"]))
    return s


def _desc(da, case, columns, pages, **more):
    latent = case["kv"] == "latent"
    return da.Desc.make(B=case["B"], H_kv=case["H_kv"], G=128 if latent else 8, D_qk=case["D"], D_v=NOPE if latent else case["D"],
                        page_size=case["P"], max_pages_per_seq=columns, num_pages=pages,
                        kv_dtype=dict(bf16=da.KV_BF16, fp8=da.KV_FP8, latent=da.KV_MLA656)[case["kv"]], **more)


def _values(pool, scale):
    return pool.float() if scale is None else pool.view(torch.float8_e4m3fn).float() * scale.view(-1, 1)


def _prepare_accum(case, seed):
    g, r = _gen(seed), random.Random(seed)
    B, H_kv, D, P, s_q = (case[k] for k in ("B", "H_kv", "D", "P", "s_q"))
    lens = _lengths(case, seed)
    pages = B * -(-case["hi"] // P) + 1                              # the last one is no one's
    table = _pages(lens, P, seed, -(-case["hi"] // P), 0, pages - 1)
    k_pool, _, k_scale, _ = _pool(g, case["kv"], pages, P, H_kv, D)
    q = torch.randn(B, s_q, 8 * H_kv, D, generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.empty(B, s_q, 8 * H_kv, device="cuda")
    on = torch.from_numpy(table).cuda()
    for b, L in enumerate(lens):                                     # what the attention call of this step left
        k = _values(k_pool[on[b, :-(-L // P)].long()].reshape(-1, H_kv, D)[:L], k_scale)
        s = torch.einsum("jhgd,thd->jhgt", q[b].float().view(s_q, H_kv, 8, D), k) / math.sqrt(D)
        late = torch.arange(L, device="cuda") > torch.arange(L - s_q, L, device="cuda")[:, None]
        lse[b] = s.masked_fill(late[:, None, None, :], -math.inf).logsumexp(-1).view(s_q, -1)
    weighted = [max(0, L - s_q) for L in lens]                       # the last s_q tokens are this step's
    s = dict(case=case, q=q, k_pool=k_pool, k_scale=k_scale, lse=lse, table=on, lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
             weighted=torch.tensor(weighted, device="cuda", dtype=torch.int32), longest=max(lens),
             accepted=torch.tensor([r.randint(0, s_q - 1) for _ in lens], device="cuda", dtype=torch.int32) if s_q > 1 else None,
             weights=torch.rand(pages, H_kv, P, generator=g, device="cuda") * 0.1)
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, table.shape[1], pages, s_q=s_q, splits=case["splits"])
        s["meta"] = torch.empty(da.sched_meta_bytes(s["desc"]), dtype=torch.uint8, device="cuda")
        da.sched_meta(s["desc"], s["lens"], s["meta"])               # the one that this step's attention call used
    return s


def _prepare_evict(case, seed):
    g = _gen(seed)
    H_kv, P = case["H_kv"], case["P"]
    lens = _lengths(case, seed)
    kept = [min(L, case["budget"]) for L in lens]
    columns, used = -(-case["hi"] // P), case["B"] * -(-case["hi"] // P)
    pages = used + case["B"] * -(-case["budget"] // P) + 1           # the last one is no one's
    table = _pages(lens, P, seed, columns, 0, used)
    into = _pages(kept, P, seed + 1, columns, used, pages - 1)
    k_pool, v_pool, k_scale, v_scale = _pool(g, case["kv"], pages, P, H_kv, case["D"])
    # gathered attention weight: heavy-tailed, many tokens with next to none
    weights = torch.exp(torch.randn(pages, H_kv, P, generator=g, device="cuda") * 2.5 - 6.0)
    s = dict(case=case, k_pool=k_pool, v_pool=v_pool, weights=weights, lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
             table=torch.from_numpy(table).cuda(), into=torch.from_numpy(into).cuda(), longest=max(lens),
             kept=torch.empty(case["B"], H_kv, case["budget"], device="cuda", dtype=torch.int32),
             new_lens=torch.empty(case["B"], device="cuda", dtype=torch.int32))
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, table.shape[1], pages)
    return s


def _dtype(case):
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[case["dtype"]]


def _prepare_verify(case, seed):
    g = _gen(seed)
    B, K, V = case["B"], case["drafts"], case["V"]
    def probs(rows):
        return torch.softmax(torch.randn(B, rows, V, generator=g, device="cuda") * 2.5, -1)
    p = probs(K + 1)
    s = dict(case=case, u=torch.rand(B, K + 1, generator=g, device="cuda"), q=None, tokens=None,
             lens=torch.randint(K + 1, 8192, (B,), generator=g, device="cuda", dtype=torch.int32),
             accepted=torch.empty(B, device="cuda", dtype=torch.int32), out=torch.empty(B, K + 1, device="cuda", dtype=torch.int32),
             new_lens=torch.empty(B, device="cuda", dtype=torch.int32))
    if K:
        q = 0.7 * p[:, :K] + 0.3 * probs(K)                          # a draft model that is mostly right
        s["tokens"] = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).int()
        if case["has_q"]:
            s["q"] = q.to(_dtype(case))
    s["p"] = p.to(_dtype(case))
    return s


def prepare(case, seed):
    return dict(rope=_prepare_rope, accum=_prepare_accum, evict=_prepare_evict, verify=_prepare_verify)[case["op"]](case, seed)


# --------------------------------------------------------------------- plain
def _pool_views(kv, k_pool, v_pool):
    """The pools as the values that they hold."""
    if kv == "bf16":
        return dict(k=k_pool, v=v_pool)
    if kv == "fp8":
        return dict(k=k_pool.view(torch.float8_e4m3fn), v=v_pool.view(torch.float8_e4m3fn))
    return dict(nope=k_pool[..., :NOPE].view(torch.float8_e4m3fn), scale=k_pool[..., NOPE:NOPE + 16].view(torch.float32),
                rope=k_pool[..., NOPE + 16:].view(torch.bfloat16))


def _turn(x, cos, sin, off, rot, adjacent):
    n = rot // 2
    ia = torch.arange(n, device=x.device) * (2 if adjacent else 1) + off
    ib = ia + (1 if adjacent else n)
    a, b = x[..., ia], x[..., ib]
    out = x.clone()
    out[..., ia] = a * cos - b * sin
    out[..., ib] = a * sin + b * cos
    return out


def _plain_rope(s):
    case = s["case"]
    N, H_q, H_kv, D, P, rot = (case[k] for k in ("tokens", "H_q", "H_kv", "D", "P", "rot"))
    latent = case["kv"] == "latent"
    angle = s["at"][s["axis"]].double() * s["inv_freq"].double()[:, None]        # far positions: 64 bits
    cos, sin = angle.cos().float().t()[:, None, :], angle.sin().float().t()[:, None, :]
    off = NOPE if latent else 0
    q = _turn(s["q"].view(N, H_q, D).float(), cos, sin, off, rot, case["adjacent"])
    s["q_out"].copy_(q)
    k = _turn(s["k"].view(N, -1, D).float(), cos, sin, off, rot, case["adjacent"])
    pos = s["pos"].long()
    page, slot = s["table"][s["req"].long(), pos // P].long(), pos % P
    if latent:
        block = k[..., :NOPE].view(N, 1, 4, 128)
        amax = block.abs().amax(-1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        row = torch.cat([_quant(block, scale[..., None]).view(N, 1, NOPE), scale.view(torch.uint8),
                         k[..., NOPE:].to(torch.bfloat16).view(torch.uint8)], -1)
        s["k_pool"][page, slot] = row
    else:
        v = s["v"].view(N, H_kv, D).float()
        if case["kv"] == "fp8":
            s["k_pool"][page, slot] = _quant(k, s["k_scale"].view(H_kv, 1))
            s["v_pool"][page, slot] = _quant(v, s["v_scale"].view(H_kv, 1))
        else:
            s["k_pool"][page, slot] = k.to(torch.bfloat16)
            s["v_pool"][page, slot] = v.to(torch.bfloat16)


def _plain_accum(s):
    case = s["case"]
    B, H_kv, D, P, s_q = (case[k] for k in ("B", "H_kv", "D", "P", "s_q"))
    T = s["longest"]
    t = torch.arange(T, device="cuda")
    spare = s["k_pool"].shape[0] - 1
    lens, there = s["lens"].long(), t < s["lens"][:, None]
    page = torch.where(there, s["table"][:, t // P].long(), spare)               # [B, T]
    slot = torch.where(there, t % P, 0)
    k = _values(s["k_pool"][page, slot], s["k_scale"])                           # [B, T, H, D]
    q = s["q"].view(B, s_q, H_kv, 8, D).permute(0, 2, 1, 3, 4).reshape(B, H_kv, s_q * 8, D).float()
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, H_kv, s_q, 8, T) / math.sqrt(D)
    lse = s["lse"].view(B, s_q, H_kv, 8).permute(0, 2, 1, 3)[..., None]
    j = torch.arange(s_q, device="cuda")
    seen = t <= (lens[:, None] - s_q + j)[..., None]                             # [B, s_q, T]
    if s["accepted"] is not None:
        seen = seen & (j <= s["accepted"][:, None])[..., None]
    new = torch.where(seen[:, None, :, None], torch.exp(score - lse), 0.0).sum((2, 3))      # [B, H, T]
    old = s["weights"][page, :, slot]                                            # [B, T, H]
    kept = torch.where(t < s["weighted"][:, None], 1.0, 0.0)[..., None] * case["decay"] * old
    s["weights"][page, :, slot] = torch.where(there[..., None], kept + new.transpose(1, 2), old)


def _plain_evict(s):
    case = s["case"]
    B, H_kv, P, budget, first, last = (case[k] for k in ("B", "H_kv", "P", "budget", "first", "last"))
    T = s["longest"]
    t = torch.arange(T, device="cuda")
    lens = s["lens"].long()
    there = t < lens[:, None]
    spare = s["k_pool"].shape[0] - 1
    w = s["weights"][torch.where(there, s["table"][:, t // P].long(), spare), :, torch.where(there, t % P, 0)].transpose(1, 2)
    always = (t < first) | (t >= lens[:, None] - last)
    w = torch.where(there[:, None], torch.where(always[:, None], math.inf, w), -math.inf)
    n = min(budget, T)
    at = w.sort(dim=-1, descending=True, stable=True).indices[..., :n]           # equal weights: the lower index first
    at = torch.where(at < lens[:, None, None], at, T).sort(-1).values
    ok = at < T                                                                  # [B, H, n]
    s["kept"].fill_(-1)
    s["kept"][..., :n] = torch.where(ok, at, -1)
    torch.minimum(s["lens"], torch.tensor(budget, device="cuda", dtype=torch.int32), out=s["new_lens"])
    b, h, i = torch.arange(B, device="cuda")[:, None, None], torch.arange(H_kv, device="cuda")[:, None], torch.arange(n, device="cuda")
    at = torch.where(ok, at, 0)
    src, src_slot = torch.where(ok, s["table"][b, at // P].long(), spare), torch.where(ok, at % P, 0)
    dst, dst_slot = torch.where(ok, s["into"][b, i // P].long(), spare), torch.where(ok, i % P, 0)
    s["k_pool"][dst, dst_slot, h] = s["k_pool"][src, src_slot, h]
    if s["v_pool"] is not None:
        s["v_pool"][dst, dst_slot, h] = s["v_pool"][src, src_slot, h]
    s["weights"][dst, h, dst_slot] = s["weights"][src, h, src_slot]


def _plain_verify(s):
    case = s["case"]
    B, K, V = case["B"], case["drafts"], case["V"]
    rows = torch.arange(B, device="cuda")
    a = torch.zeros(B, device="cuda", dtype=torch.long)
    if K:
        x = s["tokens"].long()[..., None]
        p = s["p"][:, :K].gather(2, x)[..., 0].double()
        q = s["q"].gather(2, x)[..., 0].double() if s["q"] is not None else 1.0
        a = (s["u"][:, :K].double() * q < p).long().cumprod(1).sum(1)            # next to a border: 64 bits
    w = s["p"][rows, a].float()
    if K:
        at = a.clamp(max=K - 1)
        if s["q"] is not None:
            q = s["q"][rows, at].float()
        else:
            q = (torch.arange(V, device="cuda") == s["tokens"][rows, at][:, None]).float()
        w = torch.where((a < K)[:, None], (w - q).clamp(min=0.0), w)
    cum = (w.double() * STEP).round().long().cumsum(1)
    until = (s["u"][:, K].double() * cum[:, -1].double()).floor().long()
    token = (cum <= until[:, None]).sum(1)
    i = torch.arange(K + 1, device="cuda")
    chain = torch.cat([s["tokens"].long(), token[:, None]], 1) if K else token[:, None]
    s["out"].copy_(torch.where(i < a[:, None], chain, torch.where(i == a[:, None], token[:, None], -1)))
    s["accepted"].copy_(a)
    s["new_lens"].copy_(s["lens"] - K + a)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        _own(s)
    else:
        dict(rope=_plain_rope, accum=_plain_accum, evict=_plain_evict, verify=_plain_verify)[op](s)
    if op == "rope":
        return dict(q=s["q_out"], **_pool_views(s["case"]["kv"], s["k_pool"], s["v_pool"]))
    if op == "accum":
        return s["weights"]
    if op == "evict":
        return dict(kept=s["kept"], lens=s["new_lens"], weights=s["weights"], **_pool_views(s["case"]["kv"], s["k_pool"], s["v_pool"]))
    return dict(accepted=s["accepted"], tokens=s["out"], lens=s["new_lens"])


def _own(s):
    import paged_kv_cache_60_gb300 as da
    case = s["case"]
    if case["op"] == "rope":
        da.rope_append(s["desc"], s["rope"], s["q"], s["k"], s["v"], s["inv_freq"], s["at"], s["pos"], s["table"], s["q_out"],
                       s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], requests=s["req"])
    elif case["op"] == "accum":
        da.accum_weights(s["desc"], s["q"], s["k_pool"], s["k_scale"], s["table"], s["lens"], s["meta"], s["lse"], s["weights"],
                         num_accepted=s["accepted"], weighted_lens=s["weighted"], decay=case["decay"])
    elif case["op"] == "evict":
        da.evict(s["desc"], case["budget"], s["lens"], s["table"], s["into"], s["k_pool"], s["v_pool"], s["weights"], s["kept"],
                 s["new_lens"], keep_first=case["first"], keep_last=case["last"])
    else:
        da.verify_drafts(s["p"], s["q"], s["tokens"], s["u"], s["accepted"], s["out"], cache_seqlens=s["lens"], new_seqlens=s["new_lens"])


# ---------------------------------------------------------------------- work
def _tokens(case):
    """Cached tokens that such a case has: its mean."""
    return case["B"] * (case["lo"] + case["hi"]) / 2


def work(case):
    op = case["op"]
    if op == "rope":
        N, D, rot = case["tokens"], case["D"], case["rot"]
        heads = case["H_q"] + case["H_kv"]
        if case["kv"] == "latent":
            cache = 2 * D + TOKEN
        else:
            cache = 2 * case["H_kv"] * D * (2 + (1 if case["kv"] == "fp8" else 2))
        places = 4 * (3 + len(case["axes"].split(",")))
        return dict(bytes=N * (4 * case["H_q"] * D + cache + places), flops=3 * N * heads * rot)
    if op == "accum":
        n = _tokens(case) * case["H_kv"]
        es = 1 if case["kv"] == "fp8" else 2
        rows = case["B"] * case["s_q"] * case["H_q"]
        return dict(bytes=n * (case["D"] * es + 8) + rows * (2 * case["D"] + 4), flops=2 * n * 8 * case["s_q"] * case["D"])
    if op == "evict":
        lo, hi, budget = case["lo"], case["hi"], case["budget"]
        span = range(lo, hi + 1, max(1, (hi - lo) // 256))
        kept = case["B"] * case["H_kv"] * sum(min(L, budget) for L in span) / len(span)
        row = TOKEN if case["kv"] == "latent" else 2 * case["D"] * (1 if case["kv"] == "fp8" else 2)
        return dict(bytes=4 * _tokens(case) * case["H_kv"] + kept * (2 * row + 8), flops=0)
    # one row of p, and one of q where a draft is refused (about 0.27 of the drafts are)
    refused = 1 - 0.73 ** case["drafts"] if case["has_q"] else 0.0
    n = case["B"] * case["V"]
    return dict(bytes=n * (1 + refused) * (4 if case["dtype"] == "f32" else 2), flops=3 * n)


# --------------------------------------------------------------------- exact
def _e4m3_nearest(x):
    """The e4m3 value nearest to each of these doubles (ties to the even code), from the format's definition."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    ulp = torch.exp2(torch.frexp(x).exponent.clamp(min=-5).double() - 4)         # 3 mantissa bits; subnormals below 2^-6
    return torch.round(x / ulp) * ulp


def _exact_rope(case, s):
    N, H_q, H_kv, D, P, rot = (case[k] for k in ("tokens", "H_q", "H_kv", "D", "P", "rot"))
    latent = case["kv"] == "latent"
    off = NOPE if latent else 0
    axis = s["axis"].tolist()
    where = torch.stack([s["at"][a] for a in axis], 1).double() * s["inv_freq"].double()     # [N, pairs]
    z = torch.polar(torch.ones_like(where), where)[:, None]
    pairs = lambda x: (x[..., 0::2], x[..., 1::2]) if case["adjacent"] else (x[..., :rot // 2], x[..., rot // 2:])  # noqa: E731

    def turned(x):
        x = x.double()
        a, b = pairs(x[..., off:off + rot])
        w = torch.complex(a, b) * z
        new = torch.stack([w.real, w.imag], -1).flatten(-2) if case["adjacent"] else torch.cat([w.real, w.imag], -1)
        return torch.cat([x[..., :off], new, x[..., off + rot:]], -1)

    q, k = turned(s["q"].reshape(N, H_q, D)), turned(s["k"].reshape(N, -1, D))
    row = s["table"].long().reshape(-1)[s["req"].long() * s["table"].shape[1] + s["pos"].long() // P] * P + s["pos"].long() % P
    out = {name: v.double() for name, v in _pool_views(case["kv"], s["k_pool"], s["v_pool"]).items()}
    flat = {name: v.view(-1, *v.shape[2:]) for name, v in out.items()}
    if latent:
        block = k[..., :NOPE].reshape(N, 1, 4, 128)
        scale = block.abs().amax(-1) / E4M3_MAX
        flat["nope"][row] = _e4m3_nearest(block / scale[..., None]).reshape(N, 1, NOPE)
        flat["scale"][row] = scale
        flat["rope"][row] = k[..., NOPE:]
    else:
        v = s["v"].reshape(N, H_kv, D).double()
        if case["kv"] == "fp8":
            k = _e4m3_nearest(k / s["k_scale"].double().view(H_kv, 1))
            v = _e4m3_nearest(v / s["v_scale"].double().view(H_kv, 1))
        flat["k"][row], flat["v"][row] = k, v
    return dict(q=q, **out)


def _exact_accum(case, s):
    H_kv, D, P, s_q = (case[k] for k in ("H_kv", "D", "P", "s_q"))
    out = s["weights"].double()
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-L // P)].long()
        k = s["k_pool"][pages]
        k = k.double() if s["k_scale"] is None else k.view(torch.float8_e4m3fn).double() * s["k_scale"].double().view(H_kv, 1)
        k = k.reshape(-1, H_kv, D)[:L]
        w = out[pages].transpose(1, 2).reshape(-1, H_kv)                          # [slots, H]
        new = torch.zeros(L, H_kv, dtype=torch.float64, device="cuda")
        for j in range(s_q if s["accepted"] is None else int(s["accepted"][b]) + 1):
            n = L - s_q + j + 1
            if n > 0:
                q = s["q"][b, j].double().view(H_kv, 8, D)
                e = torch.einsum("thd,hgd->thg", k[:n], q) / math.sqrt(D) - s["lse"][b, j].double().view(H_kv, 8)
                new[:n] += e.exp().sum(-1)
        m = int(s["weighted"][b])
        w[m:L] = 0
        w[:m] *= case["decay"]
        w[:L] += new
        out[pages] = w.view(-1, P, H_kv).transpose(1, 2)
    return out


def _exact_evict(case, s):
    P, budget, first, last = (case[k] for k in ("P", "budget", "first", "last"))
    pools = {name: v.double() for name, v in _pool_views(case["kv"], s["k_pool"], s["v_pool"]).items()}
    weights = s["weights"].double()
    for b, L in enumerate(s["lens"].tolist()):
        src, dst = s["table"][b].long(), s["into"][b].long()
        for h in range(case["H_kv"]):
            w = weights[src[:-(-L // P)], h].reshape(-1)[:L].cpu().numpy()
            stay = np.arange(L)
            if L > budget:
                mid = stay[first:L - last]
                best = mid[np.lexsort((mid, -w[mid]))[:budget - first - last]]
                stay = np.sort(np.concatenate([stay[:first], best, stay[L - last:]]))
            at, to = torch.from_numpy(stay).cuda(), torch.arange(len(stay), device="cuda")
            for v in pools.values():
                v[dst[to // P], to % P, h] = v[src[at // P], at % P, h]
            weights[dst[to // P], h, to % P] = weights[src[at // P], h, at % P]
    return dict(kept=None, lens=None, weights=weights, **pools)


def exact(case, seed):
    if case["op"] == "verify":                                                   # whole numbers throughout
        return None
    s = prepare(case, seed)
    return dict(rope=_exact_rope, accum=_exact_accum, evict=_exact_evict)[case["op"]](case, s)
