"""The oracle of the cache in 8 bits with scales per block: its codes are those of
the formats, its scales the smallest that fit, and its rule for a growing block
keeps the errors that the header names."""
import numpy as np
import torch

from oracle.serving_ref import E4M3, QMAX, append_block_ref, cached, codes_of, scale_for, values_of


def test_e4m3_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, want, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 100001), np.random.RandomState(1).randn(20000) * 2.0 ** -7])
    got = codes_of(x, "fp8")
    # through float32: these points are far from the rounding of a double to it
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    near = np.abs(np.abs(values_of(got, "fp8") - x) - np.abs(values_of(want, "fp8") - x)) < 1e-6
    assert near.all() and (got == want).mean() > 0.9999
    assert codes_of(np.array([np.nan, np.inf, -np.inf, 1000.0]), "fp8").tolist() == [0x7F, 0x7E, 0xFE, 0x7E]
    assert values_of(codes_of(np.array([np.nan, np.inf, -np.inf, 1.5, 2.5, -0.5]), "int8"), "int8").tolist() == [0, 127, -127, 2, 2, 0]


def test_scales_are_the_smallest_powers():
    for kind, q in QMAX.items():
        for e in (-100, -3, 0, 9, 100):
            assert scale_for(q * 2.0 ** e, kind) == 2.0 ** e
            assert scale_for(np.nextafter(q * 2.0 ** e, np.inf), kind) == 2.0 ** (e + 1)
        assert scale_for(0.0, kind) == 2.0 ** -126


def test_tokens_one_by_one_stay_within_the_errors_of_the_header():
    g = np.random.RandomState(3)
    for kind in ("fp8", "int8"):
        x = torch.from_numpy(g.randn(40, 2, 128) * np.exp(g.randn(40, 2, 1))).to(torch.bfloat16).double().numpy()
        pools = [np.zeros((2, 32, 2, 128), np.uint8) for _ in range(2)]
        scales = [np.zeros((2, 2, 2), np.float32) for _ in range(2)]
        table = np.array([[1, 0]])
        for t in range(40):
            pools, scales, err = append_block_ref(kind, pools, scales, [x[t:t + 1], x[t:t + 1]], [0, 1], [t], table)
            assert err == 0
        got = cached(kind, pools[0], scales[0], table[0], 40)
        step = np.stack([scales[0][[1, 0][t // 32], :, t % 32 // 16] for t in range(40)])[..., None].astype(np.float64)
        if kind == "int8":
            assert (np.abs(got - x) < step).all()
        else:
            normal = np.abs(got) >= step / 64
            assert (np.abs(got - x) <= np.where(normal, np.abs(x) * 2.0 ** -4, step * 2.0 ** -9)).all()
