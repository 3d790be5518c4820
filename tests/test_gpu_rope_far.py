"""Rotary angles at the ends of the int32 positions, against exact arithmetic:
position times frequency is a rational number, reduced modulo 2 pi with pi to
300 bits.

Tolerance: cos and sin are off by at most 2 pi (2^-26 + 2^-32 + |pos| (|f| + 1)
2^-64) for the angle and 2^-23 for sincospif (2 ulp); two products, a sum and its
parts' roundings add 3 * 2^-24 of the pair's magnitudes |a| + |b|; the result is
rounded once to bf16, 2^-8 of it."""
import math
from fractions import Fraction

import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu

POSITIONS = [-(1 << 31), -(1 << 31) + 1, -(1 << 30), -1234567891, -1, 0, 1, (1 << 28) + 1, (1 << 29) - 3, (1 << 30) + 7, 1999999999,
             (1 << 31) - 65, (1 << 31) - 2, (1 << 31) - 1]
FREQUENCIES = [1.0, 0.5, 100.5, 1e-4, 0.1234567, 2.0 ** -20, 3.14159274, 6.2831855, 1e-9, -0.75, 1e-30, 17.0, 0.0, 1.17549435e-38,
               0.33333334, 999.999]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _two_pi():
    def atan_inv(n, one):                        # arctan(1 / n) in units of 1 / one, by its series
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total
    one = 1 << 300
    return 2 * Fraction(4 * (4 * atan_inv(5, one) - atan_inv(239, one)), one)


def _angle(pos, f, two_pi):
    """pos * f modulo 2 pi, in (-pi, pi]."""
    x = Fraction(pos) * Fraction(f)
    return float(x - round(x / two_pi) * two_pi)


def test_pi_and_the_reduction():
    two_pi = _two_pi()
    assert float(two_pi) == 2 * math.pi
    for f in (1.0, 0.25):
        for pos in (1, 2, 1000, -777):
            assert math.isclose(math.sin(_angle(pos, f, two_pi)), math.sin(pos * f), abs_tol=1e-12)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("latent", [False, True])
def test_positions_at_the_ends(latent, adjacent):
    freq = torch.tensor(FREQUENCIES, dtype=torch.float32)
    pairs, N = len(FREQUENCIES), len(POSITIONS)
    H, G, D = (1, 128, 576) if latent else (1, 8, 64)
    off, rot = 512 if latent else 0, 2 * pairs
    g = torch.Generator().manual_seed(9)
    x = torch.randn(N, (G * H + (1 if latent else 2)) * D, generator=g).to(torch.bfloat16)
    desc = da.Desc.make(B=N, H_kv=H, G=G, D_qk=D, D_v=512 if latent else D, page_size=8, max_pages_per_seq=1, num_pages=N,
                        kv_dtype=da.KV_MLA656 if latent else da.KV_BF16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(N, 8, 1, 656 if latent else 2 * D, dtype=torch.uint8, device="cuda")
    vpool, err = None if latent else torch.zeros_like(pool), i32([0])
    q_out, xd = torch.empty(N, G, D, dtype=torch.bfloat16, device="cuda"), x.cuda()
    da.rope_append(desc, da.Rope.make(rot, adjacent=adjacent), xd[:, :G * D], xd[:, G * D:(G + 1) * D], None if latent else xd[:, (G + 1) * D:],
                   freq.cuda(), i32([POSITIONS]), i32([0] * N), i32([[n] for n in range(N)]), q_out, pool, vpool, device_error=err)
    assert int(err.item()) == 0
    row = pool[:, 0, 0].cpu()
    k = (row[:, 528:] if latent else row).contiguous().view(torch.bfloat16).double()[:, :rot]
    got = torch.cat([q_out.cpu().double()[:, :, off:off + rot], k[:, None]], 1)        # [N, G + 1, rot]
    xin = x[:, :(G + 1) * D].double().view(N, G + 1, D)[:, :, off:off + rot]
    two_pi = _two_pi()
    for i, f in enumerate(freq.tolist()):
        u, v = (2 * i, 2 * i + 1) if adjacent else (i, i + pairs)
        for n, pos in enumerate(POSITIONS):
            t = _angle(pos, f, two_pi)
            c, s = math.cos(t), math.sin(t)
            a, b = xin[n, :, u], xin[n, :, v]
            tol = (a.abs() + b.abs()) * (2 * math.pi * (2.0 ** -26 + 2.0 ** -32 + abs(pos) * (abs(f) + 1) * 2.0 ** -64) + 2.0 ** -23 + 3 * 2.0 ** -24)
            for at, want in ((u, a * c - b * s), (v, a * s + b * c)):
                diff = (got[n, :, at] - want).abs()
                assert (diff <= tol + want.abs() * 2.0 ** -8).all(), (pos, f, float((diff - tol).max()))


def test_frequencies_that_are_no_numbers():
    """An infinite or NaN frequency gives NaN in its own pairs and nowhere else."""
    D, i32 = 64, lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    desc = da.Desc.make(B=1, H_kv=1, G=8, D_qk=D, D_v=D, page_size=8, max_pages_per_seq=1, num_pages=1)
    freq = torch.full((32,), 0.5, device="cuda")
    freq[3], freq[7], freq[9] = math.inf, math.nan, -math.inf
    x = torch.randn(1, 10 * D, device="cuda").to(torch.bfloat16)
    q_out, pool, vpool = torch.empty(1, 8, D, dtype=torch.bfloat16, device="cuda"), *(torch.zeros(1, 8, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    da.rope_append(desc, da.Rope.make(D), x[:, :8 * D], x[:, 8 * D:9 * D], x[:, 9 * D:], freq, i32([[5]]), i32([0]), i32([[0]]), q_out, pool, vpool)
    bad = torch.zeros(D, dtype=torch.bool)
    for i in (3, 7, 9):
        bad[i] = bad[i + 32] = True
    assert torch.equal(torch.isnan(q_out[0].cpu()), bad.expand(8, D)) and torch.equal(torch.isnan(pool[0, 0, 0].cpu()), bad)
    assert torch.equal(vpool[0, 0, 0], x[0, 9 * D:])
