"""CPU tests of the 4-bit format's reference: every byte of a group is one slot's
code or scale, and quantising is idempotent and as exact as documented."""
from __future__ import annotations

import numpy as np

import kv4_ref as kv4


def test_places_fill_a_group():
    for byte, shift, scale in kv4.places():
        codes = set(zip(byte.ravel().tolist(), shift.ravel().tolist()))
        assert codes == {(b, s) for b in range(2048) for s in (0, 4)}
        assert sorted(scale.ravel().tolist()) == list(range(2048, 2304))


def test_scales_are_the_upper_bits_of_a_half():
    half = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(half, kv4.SCALES)
    assert float(np.float16(6 * kv4.SCALES[-1])) == 61440.0


def test_quantised_values_stay():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 256)) * np.exp(rng.standard_normal((50, 1)) * 3)
    y = kv4.number(*kv4.quantise(x))
    assert np.array_equal(kv4.number(*kv4.quantise(y)), y)
    # half a step between levels (1 of 6 at most), and what the scale's rounding
    # (2^-4 of it) cuts off the largest value
    big = np.abs(x.reshape(-1, 16)).max(1)
    assert (np.abs(x - y).reshape(-1, 16).max(1) <= big * (1 + 2.0 ** -4) / 6 + 1e-12).all()


def test_written_tokens_read_back():
    rng = np.random.default_rng(2)
    k4, v4 = (rng.integers(0, 256, (3, 2, 32, 144), dtype=np.uint8) for _ in range(2))
    row, k, v = [2, 0], rng.standard_normal((40, 2, 256)), rng.standard_normal((40, 2, 256))
    for j in range(5, 40):
        kv4.write(k4, v4, row, j, k[j], v[j])
    assert np.array_equal(kv4.read(k4, row, 5, 40, True), kv4.number(*kv4.quantise(k[5:])))
    assert np.array_equal(kv4.read(v4, row, 5, 40, False), kv4.number(*kv4.quantise(v[5:])))
