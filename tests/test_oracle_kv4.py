"""The oracle of the 4-bit cache entries against hand-made values, and of rotary positions with several axes
against complex rotation (CPU only)."""
import numpy as np
import pytest

from oracle import kvcache, layer


def test_e2m1_values_are_the_ocp_format():
    # 1 sign, 2 exponent bits (bias 1), 1 fraction bit
    for c in range(8):
        e, f = c >> 1, c & 1
        assert kvcache.E2M1[c] == (f * 0.5 if e == 0 else (1 + f / 2) * 2.0 ** (e - 1))


def test_e2m1_nearest_with_ties_to_the_even_code():
    for s in (1.0, 0.75, 2.0 ** -24, 65504.0):
        x = np.array([0, .24, .25, .26, .74, .75, .76, 1.24, 1.25, 1.26, 1.74, 1.75, 2.49, 2.5, 2.51, 3.49, 3.5, 4.99, 5,
                      5.01, 6, 7, 1e9]) * s
        want = [0, 0, 0, 1, 1, 2, 2, 2, 2, 3, 3, 4, 4, 4, 5, 5, 6, 6, 6, 7, 7, 7, 7]
        assert list(kvcache.e2m1_encode(x, s)) == want
        assert list(kvcache.e2m1_encode(-x[1:], s)) == [c + 8 for c in want[1:]]
    rng = np.random.default_rng(0)
    x = rng.standard_normal(100000) * 3
    got = kvcache.E2M1[kvcache.e2m1_encode(x, 1.0) & 7]
    best = np.abs(np.abs(x)[:, None] - kvcache.E2M1[None, :]).min(1)
    assert np.array_equal(np.abs(np.abs(x) - got), best)


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256, 512])
def test_order_holds_every_channel_once(D):
    o = kvcache.kv4_order(D)
    assert sorted(o) == list(range(D))
    assert np.array_equal(o[1::2], o[0::2] + 1) and not (o[0::2] % 2).any()


def test_order_by_hand():
    assert list(kvcache.kv4_order(32)) == list(range(32))
    assert list(kvcache.kv4_order(64)[:8]) == [0, 1, 32, 33, 2, 3, 34, 35]
    assert list(kvcache.kv4_order(96)[:4]) == [0, 1, 32, 33] and list(kvcache.kv4_order(96)[64:68]) == [64, 65, 66, 67]
    assert list(kvcache.kv4_order(128)[:10]) == [0, 1, 32, 33, 64, 65, 96, 97, 2, 3]
    assert list(kvcache.kv4_order(192)[128:134]) == [128, 129, 160, 161, 130, 131]


def test_entries_by_hand_and_there_and_back():
    x = np.zeros(64)
    x[:6] = [6.0, -3.0, 0.5, 2.5, -0.25, 1.0]
    x[33] = -12.0
    b, s = kvcache.kv4_quantize_values(x)
    assert list(kvcache.fp16_decode(s)) == [1.0, 2.0]
    assert b[0] == 7 | (8 + 5) << 4 and b[1] == 0 | (8 + 7) << 4 and b[2] == 1 | 4 << 4 and b[4] == 8 | 2 << 4
    assert list(kvcache.kv4_values(b, s)[[0, 1, 2, 3, 4, 5, 33]]) == [6, -3, .5, 2, 0, 1, -12]
    rng = np.random.default_rng(1)
    for D in (32, 96, 128, 192):
        v = rng.standard_normal((50, 3, D)) * 2.0 ** rng.integers(-20, 15, size=(50, 3, 1))
        b, s = kvcache.kv4_quantize_values(v)
        sv = np.repeat(kvcache.fp16_decode(s), 32, axis=-1)
        # half of the widest step (2 between 4 and 6) at the most, and what the scale's rounding cuts off at 6
        assert np.max(np.abs(kvcache.kv4_values(b, s) - v) - sv * (1 + 6 * 2.0 ** -11)) <= 0
        again, s2 = kvcache.kv4_quantize_values(kvcache.kv4_values(b, s))
        full = (np.abs(kvcache.kv4_values(b, s)).reshape(50, 3, -1, 32).max(-1) == 6 * kvcache.fp16_decode(s))
        assert full.all() and np.array_equal(s, s2) and np.array_equal(again & 0x77, b & 0x77)


def test_scale_range():
    x = np.zeros((6, 32))
    x[1, 3], x[2, 3], x[3, 3], x[4, 3], x[5, 3] = 1e-9, 1e6, np.nan, -np.inf, 6 * 65504.0
    b, s = kvcache.kv4_quantize_values(x)
    assert list(s[:, 0]) == [0x3C00, 1, 0x7BFF, 0x7E00, 0x7E00, 0x7BFF]
    assert kvcache.kv4_values(b, s)[2, 3] == 6 * 65504.0
    assert kvcache.kv4_bytes_per_token_head(128) == 144


def test_several_axes_against_complex_rotation():
    rng = np.random.default_rng(3)
    x, f = rng.standard_normal((7, 2, 16)), 10.0 ** -np.arange(6)
    pos, axes = rng.integers(0, 50, size=(3, 7)), np.array([0, 1, 2, 0, 2, 1])
    for inter in (False, True):
        y = layer.rope(x, pos, f, 1.5, inter, axes)
        for i in range(6):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 6)
            z = 1.5 * (x[..., a] + 1j * x[..., b]) * np.exp(1j * f[i] * pos[axes[i]])[:, None]
            assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., b], z.imag, atol=1e-12)
        assert np.array_equal(y[..., 12:], x[..., 12:])
        same = np.broadcast_to(pos[0], (3, 7))
        assert np.array_equal(layer.rope(x, same, f, 1.0, inter, axes), layer.rope(x, pos[0], f, 1.0, inter))
