"""CPU oracle for the operators around decode attention: rotary positions with
several axes, the attention weight gathered by cached tokens, eviction by that
weight, and the verification of drafted tokens. TEST INFRASTRUCTURE ONLY (see
oracle/__init__.py). numpy float64 and Python integers, token by token through
the block table; nothing is shared with the library.
"""
import math
from fractions import Fraction

import numpy as np

from .append_ref import E4M3_MAX  # noqa: F401  (the quantiser's range, for tests)


# ------------------------------------------------------------------ rotary positions
def axis_of_pairs(sections, interleaved):
    """The axis that each pair follows, from the definition."""
    n, A = sum(sections), len(sections)
    if not interleaved:
        out = []
        for a, m in enumerate(sections):
            out += [a] * m
        return out
    return [(i % A) if (i // A) < sections[i % A] else 0 for i in range(n)]


def rope_ref(x, rope_positions, inv_freq, sections, interleaved, adjacent, offset=0):
    """x float64 [N, H, D] -> rotated, and the sum of magnitudes |a| + |b| of each value's pair (0 where it
    passes through): the measure of the rounding errors. rope_positions int [A, N]; inv_freq fp32 [pairs]."""
    N, H, D = x.shape
    axes = axis_of_pairs(sections, interleaved)
    R = 2 * len(axes)
    out, mag = x.copy(), np.zeros_like(x)
    for i, a in enumerate(axes):
        # the angle modulo a turn, exactly as far as float64 goes: fp32 frequency times integer is exact in 53 bits
        # for |position| < 2^29
        theta = rope_positions[a].astype(np.float64) * float(inv_freq[i])
        c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
        u, v = (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)
        u, v = u + offset, v + offset
        p, q = x[:, :, u], x[:, :, v]
        out[:, :, u], out[:, :, v] = p * c - q * s, p * s + q * c
        mag[:, :, u] = mag[:, :, v] = np.abs(p) + np.abs(q)
    return out, mag


# ------------------------------------------------------------------ gathered attention weight
def accum_ref(q, k_of, lens, lse, sigma, s_q, accepted=None):
    """What one step adds to each token's weight: list over requests of float64 [L_b, H_kv], and a bound on the
    magnitude of the scores' terms, sigma * sum |q| |k| + |lse| of the rows, weighted the same way (for error bounds).
    q float64 [B, s_q, H_kv, G, D]; k_of(b) -> float64 [L_b, H_kv, D]; lse float64 [B, s_q, H_kv, G]."""
    add, err = [], []
    for b, L in enumerate(lens):
        k = k_of(b)
        H = k.shape[1] if L else q.shape[2]
        w, e = np.zeros((L, H)), np.zeros((L, H))
        for j in range(s_q):
            if accepted is not None and j > accepted[b]:
                continue
            n = L - s_q + 1 + j
            for h in range(H):
                for g in range(q.shape[3]):
                    ls = lse[b, j, h, g]
                    if n <= 0 or ls == -math.inf:
                        continue
                    row = q[b, j, h, g]
                    s = sigma * (k[:n, h] @ row)
                    t = np.exp(s - ls)
                    w[:n, h] += t
                    if ls != math.inf:          # (a row of zeros has no error to bound)
                        e[:n, h] += t * (sigma * (np.abs(k[:n, h]) @ np.abs(row)) + abs(ls))
        add.append(w)
        err.append(e)
    return add, err


# ------------------------------------------------------------------ eviction
def evict_select(weights, budget, keep_first, keep_last):
    """Positions kept of one request and head; weights: its tokens' weights in order (float32)."""
    L = len(weights)
    if L <= budget:
        return list(range(L))
    mid = list(range(keep_first, L - keep_last))
    # heaviest first, NaN above everything, the lower position on equality
    rank = sorted(mid, key=lambda t: (0, 0.0, t) if math.isnan(weights[t]) else (1, -float(weights[t]), t))
    chosen = rank[:budget - keep_first - keep_last]
    return sorted(list(range(keep_first)) + chosen + list(range(L - keep_last, L)))


def evict_ref(lens, table, into, pools, weights, budget, keep_first, keep_last):
    """Expected (kept [B, H, budget], new lengths, pools, weights, error bits) after an eviction. pools: uint8
    arrays [num_pages, P, H, row]; weights float32 [num_pages, H, P]; all copied. Bits: 1 bad page, 2 length over
    the table (clamped), 4 negative length (0)."""
    num_pages, P, H = pools[0].shape[:3]
    src_pools, src_w = pools, weights
    pools, weights = [p.copy() for p in pools], weights.copy()
    B, err = len(lens), 0
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    new = np.zeros(B, dtype=np.int32)
    ok = lambda page: 0 <= page < num_pages  # noqa: E731
    for b, L in enumerate(lens):
        if L < 0:
            L, err = 0, err | 4
        if L > table.shape[1] * P:
            L, err = table.shape[1] * P, err | 2
        new[b] = min(L, budget)
        for h in range(H):
            w = np.full(L, -math.inf)
            bad = set()
            for t in range(L):
                page = int(table[b, t // P])
                if ok(page):
                    w[t] = src_w[page, h, t % P]
                else:
                    bad.add(t)
            # a token on a bad page weighs less than any other, -inf among them
            if bad and L > budget:
                mid = [t for t in range(keep_first, L - keep_last)]
                rank = sorted(mid, key=lambda t: (2, 0.0, t) if t in bad else
                              ((0, 0.0, t) if math.isnan(w[t]) else (1, -float(w[t]), t)))
                stay = sorted(list(range(keep_first)) + rank[:budget - keep_first - keep_last] +
                              list(range(L - keep_last, L)))
                err |= 1 if any(t in bad for t in mid) and budget > keep_first + keep_last else 0
            else:
                stay = evict_select(w, budget, keep_first, keep_last)
            kept[b, h, :len(stay)] = stay
            for i, t in enumerate(stay):
                sp, dp = int(table[b, t // P]), int(into[b, i // P])
                if not (ok(sp) and ok(dp)):
                    err |= 1
                    continue
                for p, s in zip(pools, src_pools):
                    p[dp, i % P, h] = s[sp, t % P, h]
                weights[dp, h, i % P] = src_w[sp, h, t % P]
    return kept, new, pools, weights, err


# ------------------------------------------------------------------ verification of drafts
def _steps(w):
    """Weights in whole steps of 2^-44, to nearest, ties to even, each within [0, 1]; NaN and negative: 0. Scaling by
    a power of two is exact in float64 and the counts stay below 2^53, so rint is the rule itself."""
    w = np.asarray(w, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        w = np.where(w > 0, np.minimum(w, 1.0), 0.0)
    return np.rint(w * 2.0 ** 44).astype(np.uint64)


def draw_ref(weights, u):
    """First v whose running sum of steps exceeds floor(u * total); -1 without any weight. Exact: fewer than 2^20
    weights of at most 2^44 steps fit 64 bits."""
    run = np.cumsum(_steps(weights), dtype=np.uint64)
    total = int(run[-1])
    if total == 0:
        return -1
    u = 0.0 if not u > 0 else min(float(np.float32(u)), float(np.float32(1) - np.float32(2.0 ** -24)))
    until = math.floor(Fraction(u) * total)
    return int(np.searchsorted(run, np.uint64(until), side="right"))


def verify_ref(p, q, tokens, u, V):
    """One request: p float32 [K + 1, V] (of any probability type, widened), q float32 [K, V] or None, tokens [K], u
    float32 [K + 1] -> (accepted, out tokens [K + 1], error bits 32 / 64)."""
    K, err = len(tokens), 0
    for x in tokens:
        err |= 32 if x >= V else 0
    a, refused = 0, False
    while a < K and 0 <= tokens[a] < V:
        x = tokens[a]
        px = float(p[a][x])
        qx = 1.0 if q is None else float(q[a][x])
        uu = float(u[a])
        if any(math.isnan(z) for z in (px, qx, uu)):
            refused = True
        elif math.isinf(px) or math.isinf(qx) or math.isinf(uu):
            refused = not uu * qx < px
        else:
            refused = not Fraction(uu) * Fraction(qx) < Fraction(px)
        if refused:
            break
        a += 1
    row = np.asarray(p[a], dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        if refused and q is not None:
            w = row - np.asarray(q[a], dtype=np.float32)
        elif refused:
            w = row.copy()
            w[tokens[a]] = 0
        else:
            w = row
    token = draw_ref(w, u[K])
    if token < 0 and refused:
        token = draw_ref(row, u[K])
    if token < 0:
        err |= 64
    return a, list(tokens[:a]) + [token] + [-1] * (K - a), err
