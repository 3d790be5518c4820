"""What further operators of a serving loop cost: attention over a cache in 8
bits with a scale for each block of 16 tokens and KV head and the append that
writes it, forking, reserving, compacting and copying the pages of a cache, and
the probabilities that a verification draws from, out of logits with penalties,
biases and grammar masks.

``own`` false: the plain form of each in elementary torch operations. ``own``
true: the library's entry points, called as a serving loop calls them.
"""
import math
import random

import numpy as np
import torch

own = False

T = 16                                   # tokens of a block that shares a scale
QMAX = dict(fp8=448.0, int8=127.0)       # the largest code


# --------------------------------------------------------------------- cases
# kv: bf16 (two bytes a value), fp8 or int8 (e4m3 or int8 codes, one scale per block of 16 tokens and KV head).
def listed():
    return [
        # one new token over one short cache (latency)
        dict(name="attend_step", op="attend", kv="fp8", B=1, H_kv=1, P=16, lo=512, hi=512, s_q=1, splits=1),
        # chains of two drafts over mixed lengths, ends inside a page and a block
        dict(name="attend_mixed_chain", op="attend", kv="int8", B=32, H_kv=8, P=64, lo=1024, hi=8192, s_q=2, splits=0),
        # a large batch of long caches: bandwidth
        dict(name="attend_long", op="attend", kv="fp8", B=64, H_kv=4, P=32, lo=32768, hi=32768, s_q=1, splits=0),
        # one new token of each of 64 requests, somewhere in its block (latency)
        dict(name="append_step", op="append", kv="fp8", B=64, tokens=64, H_kv=8, P=32, far=4096),
        # ragged prompts of 8 requests appended in one call: bandwidth
        dict(name="append_prompts", op="append", kv="int8", B=8, tokens=32771, H_kv=8, P=64, far=1024),
        # a step of a small beam search: rows follow their parents, get room for a token, shared ends are copied (latency)
        dict(name="fork_beams", op="fork", kv="bf16", B=8, beams=4, H_kv=2, D=64, P=16, lo=256, hi=1024, room=1),
        # sampling in parallel over long shared prompts: 512 rows, room for a chain of four
        dict(name="fork_many", op="fork", kv="fp8", B=512, beams=8, H_kv=2, D=128, P=16, lo=2048, hi=16384, room=4),
        # a small pool with holes, packed to its front (latency)
        dict(name="compact_small", op="compact", kv="bf16", B=8, H_kv=2, D=64, P=16, lo=64, hi=640, holes=0.3),
        # a pool of half a million tokens after most of its long requests have ended: bandwidth
        dict(name="compact_large", op="compact", kv="fp8", B=64, H_kv=8, D=128, P=16, lo=1024, hi=16384, holes=0.5),
        # one request's next token (latency)
        dict(name="probs_one", op="probs", logits="f32", probs="f32", B=1, drafts=0, V=32000, lo=64, hi=512, bias=4, mask=0, greedy=0.0),
        # a batch with drafts, grammars and an odd vocabulary
        dict(name="probs_grammar", op="probs", logits="bf16", probs="f32", B=32, drafts=3, V=128259, lo=256, hi=4096, bias=32, mask=1, greedy=0.25),
        # many rows, long histories: bandwidth
        dict(name="probs_batch", op="probs", logits="bf16", probs="bf16", B=256, drafts=3, V=131072, lo=1024, hi=8192, bias=0, mask=0, greedy=0.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "append", "fork", "compact", "probs"])
    kv = rng.choice(["fp8", "int8"])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    if op == "attend":
        hi = _spread(rng, 1, 32768)
        B = _spread(rng, 1, max(1, min(64, (1 << 21) // (hi * H_kv))))
        return dict(op=op, kv=kv, B=B, H_kv=H_kv, P=rng.choice([16, 32, 64, 128]), lo=max(1, int(hi * rng.uniform(0.1, 1))), hi=hi,
                    s_q=rng.randint(1, 4), splits=rng.choice([0, 0, 1, 3, 8]))
    if op == "append":
        B = _spread(rng, 1, 64)
        return dict(op=op, kv=kv, B=B, tokens=max(B, _spread(rng, 1, 16384)), H_kv=H_kv, P=rng.choice([16, 32, 64, 128, 256]),
                    far=_spread(rng, 16, 4096))
    paged = dict(kv=rng.choice(["bf16", "fp8", "int8"]), H_kv=H_kv, P=rng.choice([16, 32, 64]))
    paged["D"] = rng.choice([64, 128]) if paged["kv"] == "bf16" else 128
    if op == "fork":
        hi = _spread(rng, 16, 16384)
        beams = rng.choice([1, 2, 4, 8])
        return dict(op=op, B=beams * _spread(rng, 1, max(1, min(32, (1 << 18) // (hi * H_kv)))), beams=beams,
                    lo=max(1, int(hi * rng.uniform(0.1, 1))), hi=hi, room=rng.choice([1, 1, 2, 4, 100]), **paged)
    if op == "compact":
        hi = _spread(rng, 16, 16384)
        return dict(op=op, B=_spread(rng, 1, max(1, min(64, (1 << 20) // (hi * H_kv)))), lo=max(1, int(hi * rng.uniform(0.1, 1))),
                    hi=hi, holes=rng.choice([0.0, 0.1, 0.5, 0.8]), **paged)
    types = ["f32", "bf16", "f16"]
    hi = _spread(rng, 1, 8192)
    return dict(op=op, logits=rng.choice(types), probs=rng.choice(types), B=_spread(rng, 1, 96), drafts=rng.choice([0, 1, 3, 5]),
                V=_spread(rng, 1000, 131072), lo=max(1, hi // 4), hi=hi, bias=rng.choice([0, 1, 32, 300]), mask=rng.randint(0, 1),
                greedy=rng.choice([0.0, 0.25]))


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, seed):
    r = random.Random(seed * 7919 + 1)
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _scale_for(amax, kind):
    """The smallest power of two, at least 2^-126, by which values up to amax have codes."""
    m, e = torch.frexp(amax.double() / QMAX[kind])
    return torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-126)).float()


def _codes(x, scale, kind):
    x = x / scale
    if kind == "fp8":
        return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _numbers(codes, kind):
    return codes.view(torch.float8_e4m3fn if kind == "fp8" else torch.int8).float()


def _block_pool(g, kind, pages, P, H, D=128):
    """A filled pool in 8 bits and the scales of its blocks; tokens and heads differ in size."""
    pool = torch.empty(pages, P, H, D, device="cuda", dtype=torch.uint8)
    scale = torch.empty(pages, H, P // T, device="cuda")
    step = max(1, (1 << 26) // (P * H * D))
    for lo in range(0, pages, step):
        n = min(pages, lo + step) - lo
        x = torch.randn(n, P // T, T, H, D, generator=g, device="cuda")
        x *= torch.exp(torch.randn(n, P // T, T, H, 1, generator=g, device="cuda") * 0.5)
        s = _scale_for(x.abs().amax((2, 4)), kind)                               # [n, P / T, H]
        scale[lo:lo + n] = s.transpose(1, 2)
        pool[lo:lo + n] = _codes(x, s[:, :, None, :, None], kind).view(n, P, H, D)
    return pool, scale


def _pools(g, case, pages):
    """K and V pools and their scales (None for bf16)."""
    if case["kv"] == "bf16":
        shape = (pages, case["P"], case["H_kv"], case["D"])
        return [torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)] + [None, None]
    (k, ks), (v, vs) = (_block_pool(g, case["kv"], pages, case["P"], case["H_kv"]) for _ in range(2))
    return [k, v, ks, vs]


def _page_table(lens, P, seed, columns, pages):
    """A block table of shuffled pages for these lengths."""
    perm = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((len(lens), columns), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        n = -(-n // P)
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def _desc(da, case, columns, pages, **more):
    D = case.get("D", 128)
    return da.Desc.make(B=case["B"], H_kv=case["H_kv"], G=8, D_qk=D, D_v=D, page_size=case["P"], max_pages_per_seq=columns,
                        num_pages=pages, kv_dtype=dict(bf16=da.KV_BF16, fp8=da.KV_FP8_BLOCK, int8=da.KV_INT8_BLOCK)[case["kv"]], **more)


def _prepare_attend(case, seed):
    g = _gen(seed)
    B, H, P, s_q = (case[k] for k in ("B", "H_kv", "P", "s_q"))
    lens = _lengths(case, seed)
    columns = -(-case["hi"] // P)
    pages = B * columns + 1
    k, v, ks, vs = _pools(g, case, pages)
    s = dict(case=case, k=k, v=v, ks=ks, vs=vs, q=torch.randn(B, s_q, 8 * H, 128, generator=g, device="cuda").to(torch.bfloat16),
             table=torch.from_numpy(_page_table(lens, P, seed, columns, pages)).cuda(), lens=_i32(lens), longest=max(lens),
             out=torch.empty(B, s_q, 8 * H, 128, device="cuda", dtype=torch.bfloat16), lse=torch.empty(B, s_q, 8 * H, device="cuda"))
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, columns, pages, s_q=s_q, splits=case["splits"])
        s["meta"] = torch.empty(da.sched_meta_bytes(s["desc"]), dtype=torch.uint8, device="cuda")
        da.sched_meta(s["desc"], s["lens"], s["meta"])                           # one schedule serves a step's layers
    return s


def _prepare_append(case, seed):
    g, r = _gen(seed), random.Random(seed)
    B, N, H, P, far = (case[k] for k in ("B", "tokens", "H_kv", "P", "far"))
    cuts = [0] + sorted(r.sample(range(1, N), B - 1)) + [N]
    counts = [b - a for a, b in zip(cuts, cuts[1:])]
    history = [r.randint(0, far) for _ in range(B)]
    pages = -(-(N + B * far) // P) + B + 1                                       # room for whatever the seed gives; the last is no one's
    columns = -(-(N + far) // P)
    k, v, ks, vs = _pools(g, case, pages)
    # rows of one projection output: q, K and V side by side
    qkv = torch.randn(N, 10 * H * 128, generator=g, device="cuda")
    qkv *= torch.exp(torch.randn(N, 1, generator=g, device="cuda") * 0.5)
    qkv = qkv.to(torch.bfloat16)
    s = dict(case=case, k=k, v=v, ks=ks, vs=vs, k_new=qkv[:, 8 * H * 128:9 * H * 128], v_new=qkv[:, 9 * H * 128:],
             starts=None if N == B else _i32(cuts), positions=_i32(history),
             req=torch.from_numpy(np.repeat(np.arange(B), counts)).cuda(), first=torch.tensor(cuts[:-1], device="cuda"),
             table=torch.from_numpy(_page_table([h + c for h, c in zip(history, counts)], P, seed, columns, pages - 1)).cuda())
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, columns, pages)
    return s


def _prepare_fork(case, seed):
    g, r = _gen(seed), random.Random(seed)
    B, P, beams = case["B"], case["P"], case["beams"]
    lens, shared = [], []
    for _ in range(B // beams):                                                  # a prompt's rows share its first part
        L = r.randint(case["lo"], case["hi"])
        lens += [L] * beams
        shared += [r.randint(L // 2, L) // P] * beams
    used = [-(-L // P) for L in lens]
    most = -(-case["hi"] // P)
    columns = most + -(-case["room"] // P) + 1
    pages = B * (columns - most // 2) + (B // beams) * most + 8                  # room for whatever the seed gives
    perm = np.random.RandomState(seed % (1 << 31)).permutation(pages).astype(np.int32)
    table, at = np.full((B, columns), -1, dtype=np.int32), 0
    for b in range(B):
        mine = 0
        if b % beams:
            mine = shared[b]
            table[b, :mine] = table[b - b % beams, :mine]
        n = used[b] - mine
        table[b, mine:used[b]] = perm[at:at + n]
        at += n
    refs = np.zeros(pages, dtype=np.int32)
    for b in range(B):
        np.add.at(refs, table[b, :used[b]], 1)
    # rows stay with their prompt, some twice, some not at all
    parents = [b - b % beams + r.randrange(beams) for b in range(B)]
    k, v, ks, vs = _pools(g, case, pages)
    s = dict(case=case, k=k, v=v, ks=ks, vs=vs, refs=torch.from_numpy(refs).cuda(), parents=_i32(parents),
             now=dict(table=torch.from_numpy(table).cuda(), held=_i32(used), lens=_i32(lens)),
             then=dict(table=torch.full((B, columns), -1, device="cuda", dtype=torch.int32), held=_i32([0] * B), lens=_i32([0] * B)),
             room=_i32([case["room"]] * B), copies=torch.empty(B, 2, device="cuda", dtype=torch.int32), missing=_i32([0]))
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, columns, pages)
    return s


def _prepare_compact(case, seed):
    g = _gen(seed)
    B, P = case["B"], case["P"]
    lens = _lengths(case, seed)
    columns = -(-case["hi"] // P)
    pages = int(B * columns / (1 - case["holes"])) + 1
    table = _page_table(lens, P, seed, columns, pages)
    refs = np.zeros(pages, dtype=np.int32)
    refs[table[table >= 0]] = 1
    live = int((refs > 0).sum())
    k, v, ks, vs = _pools(g, case, pages)
    s = dict(case=case, k=k, v=v, ks=ks, vs=vs, refs=torch.from_numpy(refs).cuda(), table=torch.from_numpy(table).cuda(),
             held=_i32([-(-L // P) for L in lens]), into=torch.full((B, columns), -1, device="cuda", dtype=torch.int32),
             new_refs=torch.empty(pages, device="cuda", dtype=torch.int32), new_page=torch.empty(pages, device="cuda", dtype=torch.int32),
             copies=torch.empty(pages // 2, 2, device="cuda", dtype=torch.int32), counts=_i32([0, 0]), moves=int((refs[live:] > 0).sum()))
    if own:
        import paged_kv_cache_60_gb300 as da
        s["desc"] = _desc(da, case, columns, pages)
    return s


def _dtype(name):
    return dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[name]


def _prepare_probs(case, seed):
    g, r = _gen(seed), random.Random(seed)
    B, K, V = case["B"], case["drafts"], case["V"]
    lens = _lengths(case, seed)
    logits = torch.randn(B, K + 1, V, generator=g, device="cuda") * 2.5
    # a text repeats itself: tokens are drawn from the lower end of the vocabulary
    history = (torch.rand(B, case["hi"], generator=g, device="cuda") ** 3 * V).int().clamp(max=V - 1)
    per = lambda values: torch.tensor([r.choice(values) for _ in range(B)], device="cuda")  # noqa: E731
    s = dict(case=case, logits=logits.to(_dtype(case["logits"])), history=history, lens=_i32(lens),
             prompt=_i32([r.randint(0, n) for n in lens]), repetition=per([1.0, 1.1, 1.3]), frequency=per([0.0, 0.2, 0.5]),
             presence=per([0.0, 0.5]), drafts=None, bias=None, allowed=None,
             temperature=torch.tensor([0.0 if r.random() < case["greedy"] else r.choice([0.6, 0.8, 1.0]) for _ in range(B)], device="cuda"),
             probs=torch.empty(B, K + 1, V, device="cuda", dtype=_dtype(case["probs"])))
    if K:
        s["drafts"] = torch.randint(0, V, (B, K), generator=g, device="cuda", dtype=torch.int32)
    if case["bias"]:
        n = [r.randint(0, case["bias"]) for _ in range(B)]
        cuts = np.concatenate([[0], np.cumsum(n)])
        s["bias_req"] = torch.from_numpy(np.repeat(np.arange(B), n)).cuda()
        s["bias"] = (_i32(cuts.tolist()), torch.randint(0, V, (int(cuts[-1]),), generator=g, device="cuda", dtype=torch.int32),
                     torch.randn(int(cuts[-1]), generator=g, device="cuda") * 4)
    if case["mask"]:
        # a grammar leaves a few words of bits in one place, most of them in another
        dense = torch.rand(B, K + 1, 1, generator=g, device="cuda") < 0.5
        bits = [torch.randint(-2 ** 31, 2 ** 31, (B, K + 1, -(-V // 32)), generator=g, device="cuda").int() for _ in range(5)]
        few = bits[0] & bits[1] & bits[2] & bits[3] & bits[4]
        s["allowed"] = torch.where(dense, bits[0] | bits[1], few)
    return s


def prepare(case, seed):
    return dict(attend=_prepare_attend, append=_prepare_append, fork=_prepare_fork, compact=_prepare_compact,
                probs=_prepare_probs)[case["op"]](case, seed)


# --------------------------------------------------------------------- plain
def _plain_attend(s):
    case = s["case"]
    B, H, P, s_q, kind = (case[k] for k in ("B", "H_kv", "P", "s_q", "kv"))
    n = -(-s["longest"] // P)
    page = s["table"][:, :n].clamp(min=0).long()                                 # columns past a request's end are masked below
    lens, t, j = s["lens"].long(), torch.arange(n * P, device="cuda"), torch.arange(s_q, device="cuda")
    late = t > (lens[:, None] - s_q + j)[..., None]                              # [B, s_q, T]
    q = s["q"].view(B, s_q, H, 8, 128).permute(0, 2, 1, 3, 4).reshape(B, H, s_q * 8, 128).float()

    def values(pool, scale):
        by_token = scale[page].repeat_interleave(T, -1)                          # [B, n, H, P]
        x = _numbers(pool[page], kind) * by_token.transpose(2, 3)[..., None]     # [B, n, P, H, 128]
        return x.flatten(1, 2).permute(0, 2, 1, 3)
    x = torch.matmul(q, values(s["k"], s["ks"]).transpose(2, 3)).view(B, H, s_q, 8, n * P) / math.sqrt(128)
    x = x.masked_fill(late[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)                                # a row that sees no token
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    seen = torch.where(late.transpose(1, 2)[:, None].all(-1), 0.0, 1.0)          # [B, 1, T]: tokens that no row sees hold anything
    v = torch.where(seen[..., None] > 0, values(s["v"], s["vs"]), 0.0)
    o = torch.matmul(e.view(B, H, s_q * 8, -1), v).view(B, H, s_q, 8, 128)
    o = torch.where(total > 0, o / total, 0.0)
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, s_q, 8 * H, 128))
    s["lse"].copy_((top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B, s_q, 8 * H))


def _plain_append(s):
    case = s["case"]
    N, H, P, kind = (case[k] for k in ("tokens", "H_kv", "P", "kv"))
    at = s["positions"].long()[s["req"]] + torch.arange(N, device="cuda") - s["first"][s["req"]]
    page, slot = s["table"][s["req"], at // P].long(), at % P
    block = page * (P // T) + slot // T                                          # of the whole pool
    # each request's first block may hold tokens already
    pos = s["positions"].long()
    was = s["table"].gather(1, pos[:, None] // P)[:, 0].long() * (P // T) + pos % P // T
    filled = pos % T                                                             # tokens before the new ones
    was = torch.where(filled > 0, was, len(s["k"]) * (P // T) - 1)               # else a block that is no one's
    i = torch.arange(T, device="cuda")
    for new, pool, scale in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        x = new.reshape(N, H, 128).float()
        blocks = pool.view(-1, P // T, T, H, 128).view(-1, T, H, 128)
        sc = scale.transpose(1, 2).reshape(-1, H)                                # [blocks, H]
        amax = torch.zeros_like(sc).index_reduce_(0, block, x.abs().amax(-1), "amax")
        need = _scale_for(amax, kind)
        touched = torch.zeros(len(sc), device="cuda").index_fill_(0, block, 1.0)[:, None] > 0
        old = sc[was]                                                            # [B, H]
        kept = torch.maximum(need[was], old)
        to = torch.where(touched, need, sc)
        to[was] = torch.where(filled[:, None] > 0, kept, to[was])
        mine = blocks[was]                                                       # [B, T, H, 128]
        again = _codes(_numbers(mine, kind) * old[:, None, :, None], kept[:, None, :, None], kind)
        grows = (i < filled[:, None])[:, :, None, None] & (kept > old)[:, None, :, None]
        blocks[was] = torch.where(grows, again, mine)
        scale.copy_(to.view(-1, P // T, H).transpose(1, 2))
        blocks[block, slot % T] = _codes(x, to[block][..., None], kind)


def _plain_copy(s, src, dst):
    for pool in (s["k"], s["v"], s["ks"], s["vs"]):
        if pool is not None:
            pool[dst] = pool[src]


def _plain_fork(s):
    case = s["case"]
    P, refs, now, then = case["P"], s["refs"], s["now"], s["then"]
    B, columns = now["table"].shape
    rows, j = torch.arange(B, device="cuda"), torch.arange(columns, device="cuda")
    # every old row lets its pages go, every new one takes those that its parent's tokens are on
    parents = s["parents"].long()
    pages = now["table"].long()
    held = j < now["held"][:, None]
    refs.scatter_add_(0, torch.where(held, pages, 0).view(-1), torch.where(held, -1, 0).int().view(-1))
    used = ((now["lens"] + P - 1) // P)[parents]
    held = j < used[:, None]
    pages = pages[parents]
    refs.scatter_add_(0, torch.where(held, pages, 0).view(-1), held.int().view(-1))
    then["table"].copy_(torch.where(held, pages.int(), then["table"]))
    then["held"].copy_(used)
    then["lens"].copy_(now["lens"][parents])
    # room: pages that others hold are not written, the last one's tokens go along
    L, n, table = then["lens"].long(), s["room"].long(), then["table"]
    last, partial = L // P, (L % P > 0) & (n > 0)
    page = torch.where(partial, table.gather(1, last[:, None])[:, 0].long(), 0)
    count = torch.zeros_like(refs).scatter_add_(0, page, partial.int())
    lowest = torch.full_like(refs, B).scatter_reduce_(0, page, torch.where(partial, rows, B).int(), "amin")
    copied = partial & (refs[page] > 1) & ~((count[page] == refs[page]) & (lowest[page] == rows))
    need = torch.where(n > 0, (L + n + P - 1) // P, used.long())
    fresh = (copied[:, None] & (j == last[:, None])) | ((j >= used[:, None]) & (j < need[:, None]))
    refs.scatter_add_(0, page, -copied.int())
    there = (refs == 0).cumsum(0)
    rank = fresh.view(-1).cumsum(0)
    new = torch.searchsorted(there, rank).view(B, columns)                       # the rank-th free page, lowest first
    refs.scatter_add_(0, torch.where(fresh, new, 0).view(-1), fresh.int().view(-1))
    table.copy_(torch.where(fresh, new.int(), table))
    then["held"].copy_(need)
    to = table.gather(1, last[:, None])[:, 0]
    s["copies"].copy_(torch.where(copied[:, None], torch.stack([page.int(), to], 1), -1))
    s["missing"].zero_()
    # a row without a copy: the page that it has, onto itself
    to = torch.where(partial, to.long(), table[:, 0].long())
    _plain_copy(s, torch.where(copied, page, to), to)
    s["now"], s["then"] = then, now


def _plain_compact(s):
    refs = s["refs"]
    n = len(refs)
    p = torch.arange(n, device="cuda")
    live = refs > 0
    count = live.sum()
    far, gap = live & (p >= count), ~live & (p < count)
    places = torch.full((n + 1,), -1, device="cuda", dtype=torch.long)
    places.scatter_(0, torch.where(gap, gap.cumsum(0) - 1, n), p)                # the i-th gap
    to = torch.where(far, places[(far.cumsum(0) - 1).clamp(min=0)], p)
    s["new_page"].copy_(torch.where(live, to, -1))
    s["new_refs"].zero_().scatter_add_(0, torch.where(live, to, 0), torch.where(live, refs, 0))
    held = torch.arange(s["table"].shape[1], device="cuda") < s["held"][:, None]
    s["into"].copy_(torch.where(held, s["new_page"][s["table"].clamp(min=0).long()], s["into"]))
    m = s["moves"]
    src = torch.full((n + 1,), -1, device="cuda", dtype=torch.long)
    src.scatter_(0, torch.where(far, far.cumsum(0) - 1, n), p)
    s["copies"].fill_(-1)
    s["copies"][:m] = torch.stack([src[:m], places[:m]], 1)
    s["counts"].copy_(torch.stack([count, far.sum()]))
    _plain_copy(s, src[:m], places[:m])


def _plain_probs(s):
    case = s["case"]
    B, K, V = case["B"], case["drafts"], case["V"]
    i = torch.arange(s["history"].shape[1], device="cuda")
    there, prompt = i < s["lens"][:, None], i < s["prompt"][:, None]
    token = s["history"].long()
    said = torch.zeros(B, V, device="cuda").scatter_add_(1, token, (there & ~prompt).float())
    asked = torch.zeros(B, V, device="cuda").scatter_add_(1, token, (there & prompt).float())
    of = lambda name: s[name][:, None]  # noqa: E731
    for j in range(K + 1):
        x = s["logits"][:, j].float()
        x = torch.where((said > 0) | (asked > 0), torch.where(x > 0, x / of("repetition"), x * of("repetition")), x)
        x = x - of("frequency") * said - torch.where(said > 0, of("presence"), 0.0)
        if s["bias"] is not None:
            x = x.index_put((s["bias_req"], s["bias"][1].long()), s["bias"][2], accumulate=True)
        if s["allowed"] is not None:
            v = torch.arange(V, device="cuda")
            x = x.masked_fill((s["allowed"][:, j, v // 32] >> (v % 32)) & 1 == 0, -math.inf)
        top, best = x.max(-1, keepdim=True)                                      # the lowest of equals, below
        best = (x == top).float().argmax(-1, keepdim=True)
        warm = of("temperature") > 0
        e = torch.exp((x - torch.where(top == -math.inf, 0.0, top)) / torch.where(warm, of("temperature"), 1.0))
        total = e.sum(-1, keepdim=True)
        p = torch.where(warm, e / torch.where(total > 0, total, 1.0), torch.zeros_like(x).scatter_(1, best, 1.0))
        s["probs"][:, j] = torch.where(top == -math.inf, 0.0, p)
        if j < K:
            said.scatter_add_(1, s["drafts"][:, j:j + 1].long(), torch.ones(B, 1, device="cuda"))


# ----------------------------------------------------------------------- run
def _as_numbers(case, pool):
    return pool if case["kv"] == "bf16" else pool.view(torch.float8_e4m3fn if case["kv"] == "fp8" else torch.int8)


def _cache(s):
    out = dict(k=_as_numbers(s["case"], s["k"]), v=_as_numbers(s["case"], s["v"]))
    return out if s["ks"] is None else dict(out, ks=s["ks"], vs=s["vs"])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        dict(attend=_own_attend, append=_own_append, fork=_own_fork, compact=_own_compact, probs=_own_probs)[op](s)
    else:
        dict(attend=_plain_attend, append=_plain_append, fork=_plain_fork, compact=_plain_compact, probs=_plain_probs)[op](s)
    if op == "attend":
        return dict(out=s["out"], lse=s["lse"])
    if op == "append":
        return _cache(s)
    if op == "fork":
        return dict(refs=s["refs"], copies=s["copies"], missing=s["missing"], **s["now"], **_cache(s))
    if op == "compact":
        return dict(table=s["into"], refs=s["new_refs"], pages=s["new_page"], counts=s["counts"], **_cache(s))
    return s["probs"]


def _own_attend(s):
    import paged_kv_cache_60_gb300 as da
    da.fwd(s["desc"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], s["meta"], s["out"], s["lse"])


def _own_append(s):
    import paged_kv_cache_60_gb300 as da
    da.append_block(s["desc"], s["k_new"], s["v_new"], s["positions"], s["table"], s["k"], s["v"], s["ks"], s["vs"],
                    token_starts=s["starts"])


def _own_fork(s):
    import paged_kv_cache_60_gb300 as da
    now, then = s["now"], s["then"]
    da.fork_pages(s["desc"], s["parents"], now["lens"], now["table"], now["held"], s["refs"], then["table"], then["held"], then["lens"])
    da.reserve_pages(s["desc"], then["lens"], then["table"], then["held"], s["refs"], s["copies"], s["missing"], new_tokens=s["room"])
    da.copy_pages(s["desc"], s["copies"], s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"])
    s["now"], s["then"] = then, now


def _own_compact(s):
    import paged_kv_cache_60_gb300 as da
    da.compact_pages(s["desc"], s["table"], s["held"], s["refs"], s["into"], s["new_refs"], s["new_page"], s["copies"], s["counts"])
    da.copy_pages(s["desc"], s["copies"], s["k"], s["v"], k_scale=s["ks"], v_scale=s["vs"], num_copies=s["counts"][1:])


def _own_probs(s):
    import paged_kv_cache_60_gb300 as da
    da.token_probs(s["logits"], s["probs"], temperature=s["temperature"], repetition=s["repetition"], frequency=s["frequency"],
                   presence=s["presence"], history=s["history"], history_lens=s["lens"], prompt_lens=s["prompt"],
                   draft_tokens=s["drafts"], bias=s["bias"], allowed=s["allowed"])


# ---------------------------------------------------------------------- work
def _page_bytes(case):
    es = 2 if case["kv"] == "bf16" else 1
    rows = case["P"] * case["H_kv"]
    return 2 * rows * case.get("D", 128) * es + (0 if es == 2 else 8 * rows // T)


def work(case):
    op, B = case["op"], case["B"]
    if op == "probs":
        rows, es = B * (case["drafts"] + 1), dict(f32=4, bf16=2, f16=2)
        row = case["V"] * (es[case["logits"]] + es[case["probs"]] + (0.125 if case["mask"] else 0))
        return dict(bytes=rows * row + B * (4 * (case["lo"] + case["hi"]) / 2 + 4 * case["bias"]), flops=6 * rows * case["V"])
    if op == "append":
        N, H = case["tokens"], case["H_kv"]
        return dict(bytes=N * H * 2 * 128 * 3 + 8 * H * (N / T + B), flops=4 * N * H * 2 * 128)
    tokens = B * (case["lo"] + case["hi"]) / 2
    if op == "attend":
        H, rows = case["H_kv"], B * case["s_q"] * 8 * case["H_kv"]
        return dict(bytes=tokens * H * 2 * (128 + 4 / T) + rows * (4 * 128 + 4) + 4 * tokens / case["P"], flops=4 * tokens * rows / B * 128)
    in_table = tokens / case["P"]
    if op == "fork":
        # tables read and written, counts of pages changed; of n rows of a prompt n (1 - (1 - 1/n)^n) are no one's second child
        n = case["beams"]
        again = B * (1 - 1 / case["P"]) * (1 - 1 / n) ** n
        return dict(bytes=8 * in_table + 8 * in_table + again * 2 * _page_bytes(case) + 24 * B, flops=0)
    columns = -(-case["hi"] // case["P"])
    pages = int(B * columns / (1 - case["holes"])) + 1
    live = in_table
    moved = live * (1 - live / pages)
    return dict(bytes=12 * pages + 8 * in_table + moved * (2 * _page_bytes(case) + 8), flops=0)


# --------------------------------------------------------------------- exact
def _exact_attend(case, s):
    H, P, s_q, kind = (case[k] for k in ("H_kv", "P", "s_q", "kv"))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-L // P)].long()

        def tokens(pool, scale):
            codes = pool[pages].view(torch.float8_e4m3fn if kind == "fp8" else torch.int8)
            return torch.einsum("pbthd,phb->pbthd", codes.double().view(-1, P // T, T, H, 128), scale[pages].double()).flatten(0, 2)
        k, v = tokens(s["k"], s["ks"]), tokens(s["v"], s["vs"])
        for j in range(s_q):
            n = L - s_q + j + 1
            if n > 0:
                x = torch.einsum("hgd,thd->hgt", s["q"][b, j].double().view(H, 8, 128), k[:n]) / math.sqrt(128)
                lse[b, j] = x.logsumexp(-1).view(-1)
                out[b, j] = torch.einsum("hgt,thd->hgd", x.softmax(-1), v[:n]).reshape(8 * H, 128)
    return dict(out=out, lse=lse)


def _round_code(x, kind):
    """The code's value nearest to each of these doubles (ties to even)."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    x = x.clamp(-448.0, 448.0)
    ulp = torch.exp2(torch.frexp(x).exponent.clamp(min=-5).double() - 4)         # 3 mantissa bits; subnormals below 2^-6
    return torch.round(x / ulp) * ulp


def _exact_append(case, s):
    H, P, kind = case["H_kv"], case["P"], case["kv"]
    starts = s["first"].tolist() + [case["tokens"]]
    out = dict(k=_as_numbers(case, s["k"]).double(), v=_as_numbers(case, s["v"]).double(), ks=s["ks"].double(), vs=s["vs"].double())
    table = s["table"].cpu()
    for b, pos in enumerate(s["positions"].tolist()):
        lo, hi = starts[b], starts[b + 1]
        first, last = pos // T, (pos + hi - lo - 1) // T
        where = [(int(table[b, i * T // P]), i * T % P) for i in range(first, last + 1)]
        page, off = torch.tensor([w[0] for w in where], device="cuda"), torch.tensor([w[1] for w in where], device="cuda")
        slots = off[:, None] + torch.arange(T, device="cuda")
        filled, n = pos % T, len(where)
        for name, scales, new in (("k", "ks", s["k_new"]), ("v", "vs", s["v_new"])):
            x = torch.full((n * T, H, 128), math.nan, dtype=torch.float64, device="cuda")
            x[filled:filled + hi - lo] = new[lo:hi].reshape(-1, H, 128).double()
            x = x.view(n, T, H, 128)
            amax = x.abs().nan_to_num(nan=0.0).amax((1, 3))                      # [n, H]
            # (a power of two itself is not pushed up by log2's last bit: bf16 maxima above one are 2^-8 above it at least)
            up = torch.ceil(torch.log2(amax / QMAX[kind]) - 1e-6).clamp(min=-126)
            scale = torch.ldexp(torch.ones_like(up), up.int())
            had = out[scales][page[0], :, off[0] // T]
            was = out[name][page[0], off[0]:off[0] + T]                          # [T, H, 128]
            if filled:
                scale[0] = torch.maximum(scale[0], had)
            code = _round_code(x / scale[:, None, :, None], kind)
            if filled:
                more = (scale[0] > had)[None, :, None]
                code[0, :filled] = torch.where(more, _round_code(was * (had / scale[0])[None, :, None], kind), was)[:filled]
            keep = out[name][page[:, None], slots]
            out[name][page[:, None], slots] = torch.where(code.isnan(), keep, code)
            out[scales][page[:, None], torch.arange(H, device="cuda"), off[:, None] // T] = scale
    return out


def _exact_probs(case, s):
    B, K, V = case["B"], case["drafts"], case["V"]
    out = torch.zeros(B, K + 1, V, dtype=torch.float64, device="cuda")
    rep, freq, pres, temp = (s[n].double().tolist() for n in ("repetition", "frequency", "presence", "temperature"))
    ids = torch.arange(V, device="cuda")
    for b in range(B):
        n, m = int(s["lens"][b]), int(s["prompt"][b])
        text = s["history"][b, :n].long()
        for j in range(K + 1):
            gone = text[m:] if j == 0 else torch.cat([text[m:], s["drafts"][b, :j].long()])
            said = torch.bincount(gone, minlength=V).double()
            known = (said > 0) | (torch.bincount(text[:m], minlength=V) > 0)
            x = s["logits"][b, j].double()
            x = torch.where(known, torch.where(x > 0, x / rep[b], x * rep[b]), x) - freq[b] * said - pres[b] * (said > 0)
            if s["bias"] is not None:
                lo, hi = s["bias"][0][b:b + 2].tolist()
                x = x + torch.zeros_like(x).index_put_((s["bias"][1][lo:hi].long(),), s["bias"][2][lo:hi].double(), accumulate=True)
            if s["allowed"] is not None:
                words = s["allowed"][b, j].long() & 0xFFFFFFFF
                x = torch.where((words[ids >> 5] >> (ids & 31)) % 2 == 1, x, -math.inf)
            if float(x.max()) == -math.inf:
                continue
            if temp[b] > 0:
                out[b, j] = torch.softmax(x / temp[b], -1)
            else:
                out[b, j, int((x == x.max()).nonzero()[0])] = 1.0
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):                                        # whole numbers and copies throughout
        return None
    s = prepare(case, seed)
    return dict(attend=_exact_attend, append=_exact_append, probs=_exact_probs)[case["op"]](case, s)
