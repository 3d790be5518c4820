"""Pins for the oracle of the operators around decode attention
(oracle/ops_ref.py): closed forms, invariants and second formulations. CPU
only."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle.ops_ref import accum_ref, axis_of_pairs, draw_ref, evict_ref, evict_select, rope_ref, verify_ref


def test_axes_of_pairs_by_hand():
    assert axis_of_pairs([2, 1, 1], False) == [0, 0, 1, 2]
    assert axis_of_pairs([4], True) == [0, 0, 0, 0]
    # alternating: 0 1 2 0 1 2 ... until an axis has its pairs, then axis 0
    assert axis_of_pairs([4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    for sections in ([12, 10, 10], [22, 5, 5], [16, 8, 8]):
        axes = axis_of_pairs(sections, True)
        assert [axes.count(a) for a in range(len(sections))] == sections


@pytest.mark.parametrize("adjacent", [0, 1])
def test_rope_keeps_norms_composes_and_is_relative(adjacent):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 24))
    f = (100.0 ** -(np.arange(8) / 8)).astype(np.float32)
    pos = np.array([[0, 5, -7]])
    y, mag = rope_ref(x, pos, f, [8], 0, adjacent)
    assert np.array_equal(y[0], x[0])                                  # position 0 turns nothing
    assert np.array_equal(y[..., 16:], x[..., 16:]) and (mag[..., 16:] == 0).all()
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), atol=1e-12)
    z, _ = rope_ref(y, -pos, f, [8], 0, adjacent)
    assert np.allclose(z, x, atol=1e-12)                               # turned back
    # the product of two turned vectors depends on the difference of their positions alone
    a, b = rng.standard_normal((2, 1, 1, 24))
    dots = []
    for shift in (0, 11, 1000):
        u, _ = rope_ref(a, np.array([[3 + shift]]), f, [8], 0, adjacent)
        v, _ = rope_ref(b, np.array([[9 + shift]]), f, [8], 0, adjacent)
        dots.append((u * v).sum())
    assert np.allclose(dots, dots[0], atol=1e-10)


def test_rope_axes_follow_their_positions():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 1, 16))
    f = np.ones(8, dtype=np.float32)
    for mix in (0, 1):
        axes = axis_of_pairs([4, 2, 2], mix)
        for a in range(3):
            pos = np.zeros((3, 1), dtype=np.int64)
            pos[a] = 1
            y, _ = rope_ref(x, pos, f, [4, 2, 2], mix, 0)
            moved = [i for i in range(8) if y[0, 0, i] != x[0, 0, i]]
            assert moved == [i for i in range(8) if axes[i] == a]


def test_accum_adds_one_for_every_row():
    """A row's softmax weights sum to one, so the step adds G * rows that see something."""
    rng = np.random.default_rng(3)
    B, s_q, H, G, D, lens = 3, 3, 2, 8, 16, [9, 2, 0]
    q, ks = rng.standard_normal((B, s_q, H, G, D)), [rng.standard_normal((L, H, D)) for L in lens]
    lse = np.full((B, s_q, H, G), -math.inf)
    for b, L in enumerate(lens):
        for j in range(s_q):
            n = L - s_q + 1 + j
            if n > 0:
                s = np.einsum("hgd,thd->hgt", q[b, j], ks[b][:n]) * 0.25
                lse[b, j] = torch.logsumexp(torch.from_numpy(s), -1).numpy()
    add, err = accum_ref(q, lambda b: ks[b], lens, lse, 0.25, s_q)
    assert np.allclose(add[0].sum(0), G * 3) and np.allclose(add[1].sum(0), G * 2) and add[2].shape == (0, H)
    assert all((e >= 0).all() for e in err)
    one, _ = accum_ref(q, lambda b: ks[b], lens, lse, 0.25, s_q, accepted=[0, -1, 2])
    assert np.allclose(one[0].sum(0), G) and (one[1] == 0).all()
    assert (one[0][7:] == 0).all()            # the first query token sees 7 of the 9 tokens


def test_evict_select_by_hand_and_by_sort():
    w = np.array([0.5, 3.0, 1.0, 1.0, 2.0, 1.0, 0.25, 9.0], dtype=np.float32)
    assert evict_select(w, 8, 0, 0) == list(range(8))
    assert evict_select(w, 3, 0, 0) == [1, 4, 7]
    assert evict_select(w, 4, 0, 0) == [1, 2, 4, 7]                    # of the three at 1.0 the lowest
    assert evict_select(w, 4, 1, 1) == [0, 1, 4, 7]
    assert evict_select(w, 2, 1, 1) == [0, 7]
    w[3] = math.nan
    w[5] = -0.0
    assert evict_select(w, 1, 0, 0) == [3]
    rng = np.random.default_rng(4)
    for _ in range(50):
        L = int(rng.integers(1, 60))
        w = rng.integers(0, 6, L).astype(np.float32)
        F, R = int(rng.integers(0, 4)), int(rng.integers(0, 4))
        N = F + R + int(rng.integers(0, 20)) or 1
        got = evict_select(w, N, F, R)
        assert got == sorted(set(got)) and len(got) == min(L, N)
        if L > N:
            mid = torch.from_numpy(w[F:L - R])
            order = torch.sort(mid, descending=True, stable=True).indices[:N - F - R]
            assert [t for t in got if F <= t < L - R] == sorted((order + F).tolist())


def test_evict_ref_moves_rows():
    P, H, row = 4, 2, 3
    pool = np.arange(8 * P * H * row, dtype=np.int64).astype(np.uint8).reshape(8, P, H, row)
    w = np.random.default_rng(5).random((8, H, P)).astype(np.float32)
    table, into = np.array([[2, 5]]), np.array([[7, -1]])
    kept, new, (got,), gw, err = evict_ref([7], table, into, [pool], w, 3, 1, 1)
    assert new.tolist() == [3] and err == 0
    for h in range(H):
        assert kept[0, h, 0] == 0 and kept[0, h, 2] == 6
        for i, t in enumerate(kept[0, h]):
            assert np.array_equal(got[7, i, h], pool[table[0, t // P], t % P, h])
            assert gw[7, h, i] == w[table[0, t // P], h, t % P]
    mask = np.ones_like(pool, dtype=bool)
    mask[7, :3] = False
    assert np.array_equal(got[mask], pool[mask])
    _, new, _, _, err = evict_ref([-3], table, into, [pool], w, 3, 1, 1)
    assert new.tolist() == [0] and err == 4


def test_draw_follows_the_running_sums():
    w = [0.0, 0.25, 0.5, 0.0, 0.25, 0.0]
    assert [draw_ref(w, u) for u in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999)] == [1, 1, 2, 2, 4, 4]
    assert draw_ref(w, 1.0) == 4 and draw_ref(w, 7.0) == 4 and draw_ref(w, math.nan) == 1 and draw_ref(w, -2.0) == 1
    assert draw_ref([0.0, math.nan, -1.0], 0.5) == -1
    # a step is 2^-44: half of one is a tie that goes to 0, a little more is a step
    assert draw_ref([2.0 ** -45, 2.0 ** -44], 0.0) == 1 and draw_ref([1.01 * 2.0 ** -45, 1.0], 0.0) == 0
    rng = np.random.default_rng(6)
    for _ in range(100):
        p = rng.random(37).astype(np.float32) ** 4
        p /= p.sum()
        u = np.float32(rng.random())
        c = np.cumsum(p.astype(np.float64))
        if np.abs(c / c[-1] - float(u)).min() > 1e-9:
            assert draw_ref(p, u) == int((c <= float(u) * c[-1]).sum())


def test_verify_gives_the_targets_distribution():
    """With u on a fine grid, first token accepted or redrawn is distributed as the target's first row."""
    V, n = 5, 40
    rng = np.random.default_rng(7)
    p, q = (rng.random((2, V)).astype(np.float32), rng.random((1, V)).astype(np.float32))
    p /= p.sum(1, keepdims=True)
    q /= q.sum(1, keepdims=True)
    count = np.zeros(V)
    for x in range(V):
        for i in range(n):
            for k in range(n):
                u = np.array([(i + 0.5) / n, (k + 0.5) / n], dtype=np.float32)
                a, out, err = verify_ref(p, q, [x], u, V)
                assert err == 0 and out[a] >= 0 and out[:a] == [x][:a] and len(out) == 2
                count[out[0]] += float(q[0, x]) / (n * n)
    assert np.abs(count - p[0]).max() < 2.0 / n


def test_verify_edges():
    p = np.array([[0.0, 1.0, 0.0], [0.5, 0.5, 0.0]], dtype=np.float32)
    u = np.array([0.5, 0.6], dtype=np.float32)
    assert verify_ref(p, None, [1], u, 3) == (1, [1, 1], 0)
    assert verify_ref(p, None, [0], u, 3) == (0, [1, -1], 0)
    assert verify_ref(p, None, [-1], u, 3) == (0, [1, -1], 0)           # the chain ends: row 0 is drawn from whole
    assert verify_ref(p, None, [3], u, 3) == (0, [1, -1], 32)
    assert verify_ref(p, np.array([[0.0, 1.0, 0.0]], dtype=np.float32), [0], u, 3) == (0, [1, -1], 0)  # nothing left: p
    assert verify_ref(p * 0, None, [0], u, 3) == (0, [-1, -1], 64)
    # next to the border: u q and p one part in 2^40 apart decide
    q = np.array([[np.float32(1 / 3), 0, 0]], dtype=np.float32)
    uq = Fraction(float(np.float32(0.7))) * Fraction(float(q[0, 0]))
    near = np.float32(float(uq))
    p2 = np.array([[near, 1 - near, 0], [1, 0, 0]], dtype=np.float32)
    assert (verify_ref(p2, q, [0], np.array([0.7, 0.1], dtype=np.float32), 3)[0] == 1) == (uq < Fraction(float(near)))
