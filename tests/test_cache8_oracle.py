"""Pins of the oracle of rotary positions and the 8-bit cache: complex
rotations, exact rationals, worked rows, and equality with the paged oracle
where one token is new."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from block_wise_int4_amd import mnb


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 12))
    pos, freqs = np.array([0, 1, -7, 1000, 2 ** 30]), rng.random(4)
    y = oracle.rope(x, pos, freqs, interleaved, 1.5)
    pairs = x[..., :8].reshape(5, 3, 4, 2) if interleaved else np.moveaxis(x[..., :8].reshape(5, 3, 2, 4), 2, 3)
    z = (pairs[..., 0] + 1j * pairs[..., 1]) * 1.5 * np.exp(1j * pos[:, None, None] * freqs)
    got = y[..., :8].reshape(5, 3, 4, 2) if interleaved else np.moveaxis(y[..., :8].reshape(5, 3, 2, 4), 2, 3)
    assert np.allclose(got[..., 0] + 1j * got[..., 1], z, rtol=0, atol=1e-6)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(y[0], np.concatenate([1.5 * x[0, :, :8], x[0, :, 8:]], axis=-1), rtol=1e-15)


def test_codes_are_the_nearest_of_the_exact_quotient():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * np.exp(rng.standard_normal((40, 1)) * 9)).astype(np.float32)
    x[0] = np.arange(64) - 63.5            # amax 63.5: s = 0.5, and codes twice the numbers
    x[1] = 0.0
    x[2] = 127 * np.float32(2.0 ** -140)   # a scale below the normal range
    x[3, :4] = [np.finfo(np.float32).max, -1e38, 1e30, 0]
    codes, scale = oracle.quantize_rows(x)
    assert scale[1] == 0 and not codes[1].any() and float(scale[3]) * 127 <= np.finfo(np.float32).max
    assert scale[0] == 0.5 and codes[0].tolist() == [2 * i - 127 for i in range(64)]
    assert scale[2] == np.float32(2.0 ** -140) and (codes[2] == 127).all()
    for r in range(40):
        if not scale[r]:
            continue
        s = Fraction(float(scale[r]))
        for c, v in zip(codes[r].tolist(), x[r].tolist()):
            exact = Fraction(v) / s
            assert abs(exact - c) <= Fraction(1, 2) or abs(c) == 127
            if abs(exact - c) == Fraction(1, 2):
                assert c % 2 == 0
    assert np.abs(codes.astype(int)).max(axis=1).tolist() == [0 if not s else 127 for s in scale]


def test_rows_that_are_not_finite():
    x = np.ones((3, 8), dtype=np.float32)
    x[0, 3], x[1, 0] = np.inf, np.nan
    codes, scale = oracle.quantize_rows(x)
    assert np.isnan(scale).tolist() == [True, True, False] and not codes[:2].any() and (codes[2] == 127).all()


def test_visible_rows():
    # single tokens; several, cut by max_new and max_len; starts out of range
    assert oracle.visible(3, [5, 0, -2], None, 4, 1) == [(0, 0, 4), (1, 1, 0), (2, 2, 0)]
    assert oracle.visible(9, [5, 3, 9], [0, 2, 2, 6], 8, 3) == [(0, 0, 4), (0, 1, 5), (2, 2, 6), (2, 3, 7), (2, 4, 8)]
    assert oracle.visible(4, [2, 2], [-3, 1, 9], 8, 9) == [(0, 0, 2), (1, 1, 0), (1, 2, 1), (1, 3, 2)]


def test_attention_is_the_paged_one_for_single_tokens_and_causal_for_several():
    rng = np.random.default_rng(2)
    q = rng.standard_normal((3, 4, 8))
    kc, vc = rng.integers(-127, 128, (2, 6, 2, 16, 8)).astype(np.int8)
    ks, vs = rng.random((2, 6, 2, 16)).astype(np.float32)
    table, lens = np.array([[0, 1], [2, -1], [3, 4]]), [20, 16, 32]
    k, v = kc * ks.astype(float)[..., None], vc * vs.astype(float)[..., None]
    one = oracle.attention_i8(q, kc, vc, ks, vs, table, lens, None, 32, 1, 0.01)
    assert np.allclose(one, oracle.paged_attention(q, k, v, table, lens, 32, 0.01), rtol=1e-13)
    # the rows of one request, as its steps one after another
    rows = oracle.attention_i8(q, kc, vc, ks, vs, table[2:], [32], [0, 3], 32, 3, 0.01)
    for i in range(3):
        step = oracle.paged_attention(q[i:i + 1], k, v, table[2:], [30 + i], 32, 0.01)
        assert np.allclose(rows[i], step[0], rtol=1e-13)


def test_frequencies():
    f, gain = mnb.rope_frequencies(64, 1e6, device="cpu")
    assert gain == 1.0 and np.allclose(f.numpy(), [1e6 ** (-2 * i / 64) for i in range(32)], rtol=1e-15)
    assert np.allclose(mnb.rope_frequencies(64, 1e6, linear=4.0, device="cpu")[0].numpy() * 4, f.numpy(), rtol=1e-15)
    s = mnb.rope_frequencies(64, 1e6, stretch=8.0, device="cpu")[0].numpy()
    assert s[0] == f[0] == 1.0 and np.isclose(s[-1] * 8, f[-1].item(), rtol=1e-12)
    p, gain = mnb.rope_frequencies(64, 1e4, by_parts=(4.0, 2048, 1.0, 32.0), device="cpu")
    base = mnb.rope_frequencies(64, 1e4, device="cpu")[0].numpy()
    turns = 2048 * base / (2 * np.pi)
    assert np.isclose(gain, 0.1 * np.log(4.0) + 1.0)
    assert np.allclose(p.numpy()[turns >= 32], base[turns >= 32]) and (turns >= 32).any()
    assert np.allclose(p.numpy()[turns <= 1] * 4, base[turns <= 1]) and (turns <= 1).any()
    mixed = (turns > 1) & (turns < 32)
    assert ((p.numpy() < base) & (p.numpy() > base / 4))[mixed].all() and (np.diff(p.numpy()) < 0).all()
    for bad in (dict(rot_dim=7), dict(rot_dim=8, linear=2.0, stretch=2.0), dict(rot_dim=8, base=-1.0),
                dict(rot_dim=2, stretch=2.0), dict(rot_dim=8, by_parts=(0.5, 10, 1, 2)),
                dict(rot_dim=8, by_parts=(2.0, 10, 3, 2))):
        with pytest.raises(ValueError):
            mnb.rope_frequencies(device="cpu", **bad)
