"""The 8-bit cache's CPU definitions checked by themselves: codes against torch's own e4m3
type, rounding against an exhaustive search, exponents against the inequality that defines them."""
import numpy as np

from oracle import chunk8


def test_values_are_e4m3():
    import torch
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(chunk8.VALUES, t.double().numpy())


def test_encode_is_nearest_even():
    import torch
    rng = np.random.default_rng(0)
    ties = (chunk8._UP[1:] + chunk8._UP[:-1]) / 2
    x = np.concatenate([ties, -ties, rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 0.01,
                        chunk8._UP, [0.0, -0.0, 448.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(chunk8.encode(x), want)
    err = np.abs(chunk8.VALUES[chunk8.encode(x)] - x)
    best = np.abs(chunk8._UP[None, :] - np.abs(x.astype(np.float64))[:, None]).min(1)
    np.testing.assert_array_equal(err, best)
    np.testing.assert_array_equal(chunk8.encode([np.nan, np.inf, -np.inf]), [0x7f] * 3)


def test_exponent():
    for a, e in ((448.0, 0), (448.5, 1), (447.0, 0), (224.0, -1), (1.75, -8), (1.7500001, -7),
                 (1.0, -8), (0.0, -124), (1e-40, -124), (3.3895313892515355e38, 120)):
        assert chunk8.exponent(a) == e, a


def test_quantise_and_values():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 64, 8)) * 2.0 ** rng.integers(-20, 20, (3, 2, 1, 1))
    for block in (16, 32, 64):
        codes, scales = chunk8.quantise(x, block)
        y = chunk8.values(codes, scales, block)
        step = np.repeat(chunk8.factor(scales), block, -1)[..., None]
        assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step))
        again = chunk8.quantise(y, block)
        np.testing.assert_array_equal(chunk8.values(*again, block), y)


def test_runs():
    pos = np.array([4, 5, 0, 1, 2, 3, -1, 7, 8])
    page = np.array([1, 1, 2, 2, 2, -1, 3, 9, 3])
    slot = np.array([30, 31, 14, 15, 16, 17, 0, 0, 40])
    got, flags = chunk8.runs(pos, page, slot, 16, 32, 4)
    assert got == [(0, 2, 1, 1), (2, 4, 2, 0), (4, 5, 2, 1)] and flags == 8
    got, flags = chunk8.runs(np.zeros(20), np.zeros(20, int), np.zeros(20, int), 16, 16, 1)
    assert got == [(0, 16, 0, 0)] and flags == 128
