"""CPU oracle for the cache in 8 bits with a scale per block of 16 tokens and
head, for the pages of a cache and for the probabilities made of logits. TEST
INFRASTRUCTURE ONLY (see oracle/__init__.py). numpy float64 and Python integers,
request by request; nothing is shared with the library.
"""
import math

import numpy as np

T = 16
QMAX = {"fp8": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ e4m3 and int8 codes
def _e4m3_table():
    """Value of each code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.nan if e == 15 and m == 7 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = -v if c & 128 else v
    return out


E4M3 = _e4m3_table()


def values_of(codes, kind):
    """uint8 codes -> float64 values, without the scale."""
    return E4M3[codes] if kind == "fp8" else codes.view(np.int8).astype(np.float64)


def codes_of(x, kind):
    """Nearest codes (ties to even), saturating; NaN -> 0x7F (e4m3), 0 (int8)."""
    if kind == "int8":
        return np.clip(np.rint(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e9, neginf=-1e9)), 448.0)
    pos = E4M3[:127]                                       # ascending, code = index
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == pos[hi], hi, code).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax, kind):
    """Smallest power of two s >= 2^-126 with amax <= QMAX s."""
    s = 2.0 ** -126
    while amax > QMAX[kind] * s:
        s *= 2
    return s


# ------------------------------------------------------------------ append
def append_block_ref(kind, pools, scales, new, starts, positions, table):
    """One append. pools: [k, v] uint8 [num_pages, P, H, 128]; scales: [k, v] float32 [num_pages, H, P / 16]; new: [k, v]
    float64 [N, H, 128]. Returns new pools, scales, error bits (1 bad page, 2 behind the table); positions in a block behind
    the last new one keep their codes."""
    pools, scales = [p.copy() for p in pools], [s.copy() for s in scales]
    num_pages, P, H, _ = pools[0].shape
    err = 0
    for b, pos in enumerate(positions):
        rows = range(starts[b], starts[b + 1])
        if pos < 0 or not rows:
            continue
        for blk in range(pos // T, (pos + len(rows) - 1) // T + 1):
            t0, t1 = max(pos, blk * T), min(pos + len(rows), blk * T + T)
            if t1 > table.shape[1] * P:
                err |= 2
                continue
            page, off = int(table[b, blk * T // P]), blk * T % P
            if not 0 <= page < num_pages:
                err |= 1
                continue
            for pool, scale, x in zip(pools, scales, new):
                for h in range(H):
                    vals = x[rows[0] + t0 - pos:rows[0] + t1 - pos, h]
                    fin = np.abs(vals[np.isfinite(vals)])
                    s, filled = scale_for(fin.max() if fin.size else 0.0, kind), t0 - blk * T
                    if filled:
                        had = float(scale[page, h, off // T])
                        if had >= s:
                            s = had
                        else:
                            old = values_of(pool[page, off:off + filled, h], kind) * had
                            pool[page, off:off + filled, h] = codes_of(old / s, kind)
                    with np.errstate(over="ignore", invalid="ignore"):
                        pool[page, off + t0 - blk * T:off + t1 - blk * T, h] = codes_of(vals / s, kind)
                    scale[page, h, off // T] = s
    return pools, scales, err


def cached(kind, pool, scale, table_row, L):
    """Values of a request's first L tokens, float64 [L, H, 128]."""
    P, H = pool.shape[1], pool.shape[2]
    out = np.zeros((L, H, 128))
    for t in range(L):
        page, slot = int(table_row[t // P]), t % P
        out[t] = values_of(pool[page, slot], kind) * scale[page, :, slot // T].astype(np.float64)[:, None]
    return out


# ------------------------------------------------------------------ attention, with what bounds its errors
def attend_ref(q, k, v, s_q, sigma, window=0, sinks=None):
    """One request: q [s_q, H, G, D], k, v [L, H, D], all float64. Returns out [s_q, H, G, D], lse [s_q, H, G], the largest
    sigma sum |q||k| of a row, sum p |v| per output value, and sum |v| over the tokens that the row sees."""
    L, H, D = k.shape
    G = q.shape[2]
    out, lse = np.zeros((s_q, H, G, D)), np.full((s_q, H, G), -math.inf)
    big, pv, sv = np.zeros((s_q, H, G)), np.zeros((s_q, H, G, D)), np.zeros((s_q, H, G, D))
    for j in range(s_q):
        n = L - s_q + 1 + j
        lo = max(0, n - window) if window else 0
        for h in range(H):
            for g in range(G):
                m, z = -math.inf, 0.0
                if n > lo:
                    s = sigma * (k[lo:n, h] @ q[j, h, g])
                    big[j, h, g] = (sigma * (np.abs(k[lo:n, h]) @ np.abs(q[j, h, g]))).max()
                    m = s.max()
                    e = np.exp(s - m)
                    z = e.sum()
                    lse[j, h, g] = m + math.log(z)
                    p = e / z
                    if sinks is not None:
                        tot = np.logaddexp(lse[j, h, g], sinks[h, g])
                        p = p * math.exp(lse[j, h, g] - tot)
                        lse[j, h, g] = tot
                    out[j, h, g] = p @ v[lo:n, h]
                    pv[j, h, g] = p @ np.abs(v[lo:n, h])
                    sv[j, h, g] = np.abs(v[lo:n, h]).sum(0)
                elif sinks is not None:
                    lse[j, h, g] = sinks[h, g]
    return out, lse, big, pv, sv


# ------------------------------------------------------------------ pages
def fork_ref(parents, lens, table, held, refs, new_table, P):
    """-> new table, held, lens, refs, error bits (1 bad page, 4 negative length, 128 bad parent)."""
    B, cols = table.shape
    refs, new_table, err = refs.copy(), new_table.copy(), 0
    new_held, new_lens = np.zeros(B, np.int32), np.zeros(B, np.int32)
    ok = lambda page: 0 <= page < len(refs)  # noqa: E731
    for b in range(B):
        for j in range(min(max(held[b], 0), cols)):
            if ok(table[b, j]):
                refs[table[b, j]] -= 1
    for i, r in enumerate(parents):
        if r >= B:
            err |= 128
        if not 0 <= r < B:
            continue
        err |= 4 if lens[r] < 0 else 0
        L = max(lens[r], 0)
        n = min(-(-L // P), min(max(held[r], 0), cols))
        for j in range(n):
            new_table[i, j] = table[r, j]
            if ok(table[r, j]):
                refs[table[r, j]] += 1
        new_held[i], new_lens[i] = n, L
    return new_table, new_held, new_lens, refs, err


def reserve_ref(new_tokens, lens, table, held, refs, P):
    """-> table, held, refs, copies, missing, error bits (2 too long, 4 negative length, 256 too few pages)."""
    B, cols = table.shape
    before = (table.copy(), held.copy(), refs.copy())
    table, held, refs = table.copy(), held.copy(), refs.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    copies, err = np.full((B, 2), -1, np.int32), 0
    asks, was = {}, refs.copy()
    for b in range(B):
        L, n = max(lens[b], 0), new_tokens[b]
        err |= 4 if lens[b] < 0 else 0
        if n <= 0:
            continue
        if L + n > cols * P:
            err |= 2
            continue
        asks[b] = (L, -(-(L + n) // P))
    writers = {}                                           # shared last pages with tokens on them
    for b, (L, need) in asks.items():
        if L % P and L // P < held[b] and was[table[b, L // P]] > 1:
            writers.setdefault(int(table[b, L // P]), []).append(b)
    copied = {}
    for page, rows in writers.items():
        movers = rows[1:] if len(rows) == was[page] else rows
        for b in movers:
            copied[b] = page
            refs[page] -= 1
    fresh = []                                             # (row, entry)
    for b, (L, need) in asks.items():
        first, start = -(-L // P), held[b]
        if any(was[table[b, j]] > 1 for j in range(first, min(held[b], need))):
            for j in range(first, held[b]):
                refs[table[b, j]] -= 1
            start = held[b] = first
        if b in copied:
            fresh.append((b, L // P))
        fresh += [(b, j) for j in range(start, need)]
        held[b] = max(held[b], need)
    if len(fresh) > len(free):
        return (*before, np.full((B, 2), -1, np.int32), len(fresh) - len(free), err | 256)
    for (b, j), page in zip(fresh, free):
        table[b, j] = page
        refs[page] = 1
    for b, page in copied.items():
        copies[b] = page, table[b, asks[b][0] // P]
    return table, held, refs, copies, 0, err


def compact_ref(table, held, refs, into):
    """-> new table, new refs, new_page, pairs, pages in use."""
    live = [p for p in range(len(refs)) if refs[p] > 0]
    N = len(live)
    far, gap = [p for p in live if p >= N], [p for p in range(N) if refs[p] <= 0]
    new_page = np.full(len(refs), -1, np.int32)
    new_page[live] = live
    new_page[far] = gap
    new_refs = np.zeros_like(refs)
    new_refs[new_page[live]] = refs[live]
    into = into.copy()
    for b in range(len(held)):
        into[b, :held[b]] = new_page[table[b, :held[b]]]
    return into, new_refs, new_page, list(zip(far, gap)), N


# ------------------------------------------------------------------ probabilities out of logits
def adjusted(logits, dtype, text, prompt, drafts, j, rep, freq, pres, bias, V):
    """x of row j in `dtype` (float32: each step rounded as the header says; float64: the formula). logits [V], text: the
    request's tokens, prompt: how many of them are the prompt's, bias: list of (token, value) in order."""
    f = dtype
    x = logits.astype(f)
    said, asked = np.zeros(V, np.int64), np.zeros(V, bool)
    for i, t in enumerate(text):
        if 0 <= t < V:
            if i < prompt:
                asked[t] = True
            else:
                said[t] += 1
    for t in drafts[:j]:
        if t < 0:
            break
        if t < V:
            said[t] += 1
    seen = asked | (said > 0)
    with np.errstate(all="ignore"):
        x = np.where(seen, np.where(x > 0, x / f(rep), x * f(rep)), x)
        x = np.where(said > 0, x - f(freq) * said.astype(f) - f(pres), x)
        for t, v in bias:
            if 0 <= t < V:
                x[t] = x[t] + f(v)
    return x


def probs_ref(x, allowed, T):
    """p (float64) of adjusted logits (float64); allowed: bool [V]. With T > 0 also |x - max| (0 where nothing is)."""
    V = len(x)
    ok = allowed & ~(np.isneginf(x))
    if not T > 0:
        p = np.zeros(V)
        cand = ok & ~np.isnan(x)
        if cand.any():
            p[int(np.argmax(np.where(cand, x, -np.inf)))] = 1
        return p, np.zeros(V)
    if not ok.any():
        return np.zeros(V), np.zeros(V)
    if np.isnan(x[ok]).any() or np.isposinf(x[ok]).any():
        return np.full(V, np.nan), np.zeros(V)
    d = np.where(ok, x - x[ok].max(), 0.0)
    e = np.where(ok, np.exp(d / T), 0.0)
    return e / e.sum(), np.abs(d)
