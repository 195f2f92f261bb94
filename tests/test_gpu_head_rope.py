"""GPU norms of query and key heads with rotary positions (one axis or several), alone and into the cache of 8 or 4
bits, against the float64 oracle.

Tolerances, with u = 2^-24 and r the row's largest |x w| rho (its value before the rotation):
  bf16 rows   2^-8 of the value (one rounding) + 24 u r: the sum of squares (8 + 6 additions, half of that in rho), the
              reciprocal root and its factors 6 u, the products with w 2 u, the rotation's cosines and three roundings
              4 u of each of two terms
  8-bit K     half a step of the stored scale, 2^-11 of 127 steps that the scale's rounding to fp16 takes off the
              largest codes, and that of the fp32 value (24 u r), as in test_gpu_rope_kv.py
  4-bit K, V  the oracle's codes and scales themselves (K is computed in 64 bits: a code on the other side of a border
              takes a value within 2^-50 of it; V is compared as it came)."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import kvcache, layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, codes, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


def _rows(rng, T, H, D, gain=1.0):
    b = oracle.f32_to_bf16_bits((gain * rng.standard_normal((T, H, D))).astype(np.float32))
    return bf16_to_gpu(b), bits_to_f64(b)


def _weight(rng, D):
    b = oracle.f32_to_bf16_bits((1 + 0.3 * rng.standard_normal(D)).astype(np.float32))
    return bf16_to_gpu(b), bits_to_f64(b)


def _spin(rng, T, R, n, far=1000, dtype=torch.int64):
    """Frequencies, positions and axes (n > 1), on the GPU and as arrays."""
    f = 10000.0 ** (-2.0 * np.arange(R // 2) / R)
    pos = rng.integers(0, far, size=(n, T) if n > 1 else T)
    axes = rng.integers(0, n, size=R // 2) if n > 1 else None
    gpu = (torch.from_numpy(f).to(dev()), torch.from_numpy(pos).to(dtype).to(dev()),
           None if axes is None else torch.from_numpy(axes.astype(np.int32)).to(dev()))
    return gpu, (f, pos, axes)


def _turned(x, w, spin, inter, factor=1.0, eps=EPS):
    f, pos, axes = spin
    y = layer.norm_heads(x, w, eps)
    return layer.rope(y, pos, f, factor, inter, axes), np.abs(y).max(-1, keepdims=True) * max(1.0, abs(factor))


def _check_rows(got, want, top, what=""):
    g = bits_to_f64(bf16_bits(got))
    over = np.abs(g - want) - 2.0 ** -8 * np.abs(want) - 24 * U * top
    assert np.max(over) <= 0, f"{what}: {np.max(over):.3e} beyond the bound"


def _values(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _check_entries4(cache, at, k64, v64, what=""):
    """Entries `at` of a 4-bit cache are those of k64 and v64 (a zero's sign aside)."""
    for cc, ss, x in ((cache.k_codes, cache.k_scales, k64), (cache.v_codes, cache.v_scales, v64)):
        b, s = kvcache.kv4_quantize_values(x)
        gc, gs = codes(cc)[at], _values(ss)[at]
        assert np.array_equal(gs, s), f"{what}: scales"
        finite = np.repeat(oracle.fp16_decode(s) < np.inf, 32, axis=-1)
        got, want = kvcache.kv4_values(gc, gs), kvcache.kv4_values(b, s)
        assert np.array_equal(got[finite], want[finite]), f"{what}: codes"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads", [(28, 4, 128, 128), (16, 16, 64, 64), (9, 3, 64, 32), (12, 4, 96, 96), (8, 1, 192, 96),
                                   (16, 2, 256, 64), (3, 1, 72, 20), (2, 5, 80, 48), (1, 1, 8, 2), (4, 2, 512, 512),
                                   (5, 3, 32, 10), (7, 2, 160, 160), (2, 2, 208, 16)])
def test_norm_rope(heads, inter):
    Hq, Hk, D, R = heads
    rng = np.random.default_rng(D + R + inter)
    for T, n in ((1, 1), (5, 3), (67, 2), (1024, 1), (2051, 3)):
        if T * D > 2051 * 128:
            continue
        print(f"norm_rope heads={heads} inter={inter} T={T} axes={n}", flush=True)
        (q, q64), (k, k64) = _rows(rng, T, Hq, D, 3.0), _rows(rng, T, Hk, D, 0.1)
        (wq, wq64), (wk, wk64) = _weight(rng, D), _weight(rng, D)
        (f, pos, ax), spin = _spin(rng, T, R, n)
        gq, gk = qlq.norm_rope(q, k, wq, wk, pos, f, EPS, 1.25, inter, ax)
        for got, x, w in ((gq, q64, wq64), (gk, k64, wk64)):
            _check_rows(got, *_turned(x, w, spin, inter, 1.25), what=f"T={T}")


@pytest.mark.parametrize("which", ["q", "k", "neither"])
def test_norm_of_one_or_neither(which):
    rng = np.random.default_rng(4)
    (q, q64), (k, k64), (w, w64) = _rows(rng, 33, 6, 128), _rows(rng, 33, 2, 128), _weight(rng, 128)
    (f, pos, _), spin = _spin(rng, 33, 128, 1)
    a, b = (w if which == n else None for n in "qk")
    gq, gk = qlq.norm_rope(q, k, a, b, pos, f)
    _check_rows(gq, *_turned(q64, w64 if which == "q" else None, spin, False))
    _check_rows(gk, *_turned(k64, w64 if which == "k" else None, spin, False))


@pytest.mark.parametrize("R", [64, 128, 20])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_with_axes(R, inter):
    rng = np.random.default_rng(R)
    x, x64 = _rows(rng, 131, 3, 128)
    (f, pos, ax), spin = _spin(rng, 131, R, 3, dtype=torch.int32)
    got = qlq.rope(x, pos, f, 0.5, inter, axes=ax)
    _check_rows(got, *_turned(x64, None, spin, inter, 0.5))
    # one axis for all frequencies is plain rotation, to the roundings of fp32
    one = qlq.rope(x, pos[:1].contiguous(), f, 1.0, inter, axes=torch.zeros_like(ax))
    _check_rows(one, *_turned(x64, None, (spin[0], spin[1][0], None), inter))
    # entries of axes outside 0 .. 2 count as the nearest
    wild = torch.where(ax == 2, torch.full_like(ax, 1 << 30), torch.where(ax == 0, torch.full_like(ax, -5), ax))
    assert torch.equal(qlq.rope(x, pos, f, 0.5, inter, axes=wild), got)


def test_far_and_negative_positions():
    rng = np.random.default_rng(8)
    x, x64 = _rows(rng, 6, 2, 64)
    f = np.concatenate([[1.0, 0.999], 10.0 ** -np.arange(30)])
    pos = np.array([[-3, 1 << 24, (1 << 31) + 5, -(1 << 20), 7, 0], [1, -1, 1 << 20, 123456789, 1 << 33, -(1 << 24)]])
    ax = np.arange(32) % 2
    ang = pos[ax].T * f                                  # exact angles' roundings to 64 bits stay: 2^-53 of 2^33
    got = qlq.rope(x, torch.from_numpy(pos).to(dev()), torch.from_numpy(f).to(dev()),
                   axes=torch.from_numpy(ax.astype(np.int32)).to(dev()))
    a, b = x64[..., :32], x64[..., 32:]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    want = np.concatenate([a * c - b * s, a * s + b * c], -1)
    _check_rows(got, want, np.abs(x64).max(-1, keepdims=True))


def test_every_quarter_turn():
    # angles around all multiples of pi / 4 over two turns either way, positions 1 (the frequency is the angle)
    f = np.concatenate([m * np.pi / 4 + np.array([-1e-3, -1e-9, 0, 1e-9, 1e-3]) for m in range(-8, 9)])[:84]
    x = torch.zeros(1, 1, 168, dtype=torch.bfloat16, device=dev())
    x[..., :84] = 1.0
    got = bits_to_f64(bf16_bits(qlq.rope(x, torch.ones(1, 1, dtype=torch.int64, device=dev()), torch.from_numpy(f).to(dev()),
                                         axes=torch.zeros(84, dtype=torch.int32, device=dev()))))[0, 0]
    want = np.concatenate([np.cos(f), np.sin(f)])
    assert np.max(np.abs(got - want) - 2.0 ** -8 * np.abs(want) - 4 * U) <= 0


def test_strides_in_place_and_unaligned_rows():
    rng = np.random.default_rng(5)
    T, Hq, Hk, D = 19, 4, 2, 64
    wide = bf16_to_gpu(oracle.f32_to_bf16_bits(rng.standard_normal((T, (Hq + 2 * Hk) * D + 3)).astype(np.float32)))
    (wq, wq64), (wk, wk64) = _weight(rng, D + 1), _weight(rng, D + 1)
    wq, wk, wq64, wk64 = wq[1:], wk[1:], wq64[1:], wk64[1:]           # (2 bytes off a vector's alignment)
    (f, pos, _), spin = _spin(rng, T, D, 1)
    for off in (0, 1):                                                # odd rows: nothing is 16-byte aligned
        q = wide[:, off:off + Hq * D].unflatten(-1, (Hq, D))
        k = wide[:, off + Hq * D:off + (Hq + Hk) * D].unflatten(-1, (Hk, D))
        q64, k64 = bits_to_f64(bf16_bits(q.contiguous())), bits_to_f64(bf16_bits(k.contiguous()))
        want = _turned(q64, wq64, spin, False), _turned(k64, wk64, spin, False)
        gq, gk = qlq.norm_rope(q, k, wq, wk, pos, f, EPS)
        _check_rows(gq, *want[0])
        _check_rows(gk, *want[1])
        guard = wide.clone()
        oq = guard[:, off:off + Hq * D].unflatten(-1, (Hq, D))
        ok = guard[:, off + Hq * D:off + (Hq + Hk) * D].unflatten(-1, (Hk, D))
        rest = guard.clone()
        qlq.norm_rope(oq, ok, wq, wk, pos, f, EPS, q_out=oq, k_out=ok)        # in place
        assert torch.equal(oq, gq) and torch.equal(ok, gk)
        keep = torch.ones_like(guard, dtype=torch.bool)
        keep[:, off:off + (Hq + Hk) * D] = False
        assert torch.equal(guard[keep], rest[keep])


def test_rows_of_zeros_and_of_extremes():
    rng = np.random.default_rng(6)
    q, q64 = _rows(rng, 4, 2, 64)
    q[0] = 0.0
    q[1] *= 2.0 ** -60
    q[2] *= 2.0 ** 50                                                  # squares 2^100
    q64 = bits_to_f64(bf16_bits(q))
    w, w64 = _weight(rng, 64)
    (f, pos, _), spin = _spin(rng, 4, 64, 1)
    gq, gk = qlq.norm_rope(q, q, w, w, pos, f, 1e-5)
    _check_rows(gq, *_turned(q64, w64, spin, False, eps=1e-5))
    assert torch.equal(gq, gk) and not gq[0].any()
    q[3, 1, 7] = float("nan")
    gq, _ = qlq.norm_rope(q, q, w, w, pos, f, 1e-5)
    assert bool(torch.isnan(gq[3, 1]).all()) and bool(torch.isfinite(gq[3, 0].float()).all())


HEADS = [(28, 4, 128, 128), (16, 16, 64, 64), (3, 1, 96, 96), (2, 2, 192, 64), (4, 3, 32, 20), (2, 1, 256, 256), (3, 5, 160, 48),
         (1, 2, 224, 224), (2, 1, 512, 512)]


def test_norms_whose_products_or_squares_leave_fp32():
    # Rows and weights whose products x w are beyond fp32 though the results are not, beside rows of ordinary size;
    # squares that fp32 loses beside an eps as small (powers of two move nothing in the derivation of the bounds).
    rng = np.random.default_rng(77)
    T, H, D = 9, 6, 128
    spin_gpu, spin = _spin(rng, T, D, 1)
    f, pos, _ = spin_gpu
    for gain, wgain, eps in ((2.0 ** 123, 2.0 ** 20, 1e-6), (2.0 ** 66, 2.0 ** 63, 1e-6), (2.0 ** -72, 1.0, 2.0 ** -140),
                             (2.0 ** -60, 8.0, 2.0 ** -126), (2.0 ** -40, 1.0, 2.0 ** -70)):
        b = rng.standard_normal((T, H, D))
        b[1::2] *= gain
        b[::2] *= max(gain, 1e-3) if gain < 1 else 1.0
        xb = oracle.f32_to_bf16_bits(b.astype(np.float32))
        x, x64 = bf16_to_gpu(xb), bits_to_f64(xb)
        wb = oracle.f32_to_bf16_bits((wgain * (1 + 0.3 * rng.standard_normal(D))).astype(np.float32))
        w, w64 = bf16_to_gpu(wb), bits_to_f64(wb)
        for inter in (False, True):
            q, k = qlq.norm_rope(x, x, w, w, pos, f, eps=eps, interleaved=inter)
            want, top = _turned(x64, w64, spin, inter, eps=float(np.float32(eps)))
            _check_rows(q, want, top, f"q, gain {gain:.0e}")
            assert torch.equal(q, k)
        cache = qlq.kv_cache(64, H, D, device=dev(), bits=4)
        at = torch.arange(T, device=dev())
        qlq.norm_rope_kv_append(x, x, x, w, w, pos, f, cache, at, eps=eps)
        want, _ = _turned(x64, w64, spin, False, eps=float(np.float32(eps)))
        _check_entries4(cache, np.arange(T), want, x64, f"gain {gain:.0e}")


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads", HEADS)
def test_append_four_bits(heads, inter, normed):
    Hq, Hk, D, R = heads
    rng = np.random.default_rng(D + R)
    for T, n in ((1, 1), (7, 3), (130, 1), (1030, 2), (2049, 1)):
        if T * D > 2049 * 128:
            continue
        print(f"append4 heads={heads} inter={inter} norm={normed} T={T} axes={n}", flush=True)
        (q, q64), (k, k64), (v, v64) = _rows(rng, T, Hq, D), _rows(rng, T, Hk, D, 2.0), _rows(rng, T, Hk, D, 0.3)
        (wq, wq64), (wk, wk64) = (_weight(rng, D), _weight(rng, D)) if normed else ((None, None),) * 2
        (f, pos, ax), spin = _spin(rng, T, R, n, dtype=torch.int32 if T == 7 else torch.int64)
        cache = qlq.kv_cache(T + 40, Hk, D, dev(), bits=4)
        before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        slots = rng.permutation(T + 40)[:T]
        slots[T // 3] = [-1, T + 40, 1 << 40, -(1 << 40), T + 41][n + inter]
        s = torch.from_numpy(slots).to(dev())
        if normed:
            got = qlq.norm_rope_kv_append(q, k, v, wq, wk, pos, f, cache, s, EPS, 0.75, inter, ax)
        else:
            got = qlq.rope_kv_append(q, k, v, pos, f, cache, s, 0.75, inter, axes=ax)
        _check_rows(got, *_turned(q64, wq64, spin, inter, 0.75))
        here = (slots >= 0) & (slots < T + 40)
        turned, _ = _turned(k64, wk64, spin, inter, float(np.float32(0.75)))
        _check_entries4(cache, slots[here], turned[here], v64[here], f"T={T}")
        rest = np.setdiff1d(np.arange(T + 40), slots[here])
        for a, b in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), before):
            assert torch.equal(a[rest], b[rest])
        # reading back: bf16 of the entries, zeros for a slot outside
        gk, gv = qlq.kv_gather(cache, s)
        for g, cc, ss in ((gk, cache.k_codes, cache.k_scales), (gv, cache.v_codes, cache.v_scales)):
            want = kvcache.kv4_values(codes(cc)[slots[here]], _values(ss)[slots[here]])
            assert np.array_equal(bf16_bits(g)[here] & 0x7FFF, oracle.f32_to_bf16_bits(want.astype(np.float32)) & 0x7FFF)
            assert np.array_equal(bits_to_f64(bf16_bits(g)[here]) > 0, want > 0)
            assert not g[T // 3].any()


@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256, 480])
def test_kv_append_four_bits_without_rotation(D):
    rng = np.random.default_rng(D)
    for T, H in ((1, 1), (50, 3), (1500, 2)):
        (k, k64), (v, v64) = _rows(rng, T, H, D), _rows(rng, T, H, D)
        # ties: values on the borders between codes of scales that are powers of two, and of 1.5 of them
        for a, g64 in ((k, k64), (v, v64)):
            a[0, 0, :12] = torch.tensor([6, 5, -5, 3.5, 2.5, 1.75, 1.25, -.75, .25, -.25, .125, 4.5]) * (1.5 if D == 64 else 1.0)
            g64[0] = bits_to_f64(bf16_bits(a[0]))
            a[0, 0, 12:32] = 0
            g64[0, 0, 12:32] = 0
        cache = qlq.kv_cache(T, H, D, dev(), bits=4)
        assert qlq.kv_append(k, v, cache, torch.arange(T, device=dev(), dtype=torch.int32)) is cache
        _check_entries4(cache, np.arange(T), k64, v64, f"{T},{H}")


@pytest.mark.parametrize("H,D", [(3, 128), (1, 256), (5, 384), (2, 512), (3, 96), (1, 32), (7, 224)])
@pytest.mark.parametrize("n", [1, 67])
def test_gather_four_bits_of_any_codes_and_scales(H, D, n):
    print(f"gather4 H={H} D={D} n={n}", flush=True)
    rng = np.random.default_rng(D + n)
    P = 40
    kc, vc = (rng.integers(0, 256, size=(P, H, D // 2)).astype(np.uint8) for _ in range(2))
    ks, vs = (oracle.fp16_encode(rng.uniform(1e-3, 900, size=(P, H, D // 32)).astype(np.float32)) for _ in range(2))
    up = lambda a, t: torch.from_numpy(a).view(t).to(dev())
    cache = qlq.QuantizedKV4(up(kc, torch.uint8), up(ks, torch.float16), up(vc, torch.uint8), up(vs, torch.float16))
    at = rng.integers(0, P, size=n)
    at[n // 2], at[-1] = (-1, P) if n > 2 else (3, 3)
    gk, gv = qlq.kv_gather(cache, torch.from_numpy(at).to(dev()))
    inside = (at >= 0) & (at < P)
    for got, c, sc in ((gk, kc, ks), (gv, vc, vs)):
        want = np.zeros((n, H, D))
        want[inside] = kvcache.kv4_values(c, sc)[at[inside]]
        assert np.array_equal(bf16_bits(got), oracle.f32_to_bf16_bits(want.astype(np.float32)))


@pytest.mark.parametrize("rotated", [False, True])
def test_four_bit_groups_of_zeros_extremes_and_nans(rotated):
    T, D = 8, 96
    x = np.random.default_rng(2).standard_normal((T, 1, D)).astype(np.float32)
    x[0], x[1, 0, :32], x[2, 0, 32:64] = 0, 0, 1e-30
    x[3, 0, :32] *= 1e6
    x[4], x[5, 0, 40], x[6, 0, 70] = 3e38, np.nan, np.inf
    x[7, 0, 64:] = -2.0 ** -27
    b = oracle.f32_to_bf16_bits(x)
    g, x64 = bf16_to_gpu(b), bits_to_f64(b)
    cache = qlq.kv_cache(T, 1, D, dev(), bits=4)
    s = torch.arange(T, device=dev())
    if rotated:
        # half a turn: the same values negated, their groups as they are
        f = torch.full((D // 2,), np.pi, dtype=torch.float64, device=dev())
        qlq.rope_kv_append(g, g, g, torch.zeros(T, dtype=torch.int64, device=dev()), f, cache, s)
    else:
        qlq.kv_append(g, g, cache, s)
    if rotated:                                             # (0 turns: x cos 0; a NaN or infinity reaches its partner)
        with np.errstate(invalid="ignore"):
            k64 = layer.rope(x64, np.zeros(T), np.ones(D // 2))
    else:
        k64 = x64
    _check_entries4(cache, np.arange(T), k64, x64)
    assert np.isnan(oracle.fp16_decode(_values(cache.v_scales)[5, 0, 1])) and _values(cache.v_scales)[6, 0, 2] == 0x7E00


@pytest.mark.parametrize("heads", HEADS[:7])
def test_append_eight_bits(heads):
    Hq, Hk, D, R = heads
    rng = np.random.default_rng(D)
    for T, n, inter in ((1, 1, False), (61, 3, True), (1100, 2, False)):
        (q, q64), (k, k64), (v, v64) = _rows(rng, T, Hq, D), _rows(rng, T, Hk, D, 2.0), _rows(rng, T, Hk, D, 0.3)
        (wq, wq64), (wk, wk64) = _weight(rng, D), _weight(rng, D)
        (f, pos, ax), spin = _spin(rng, T, R, n)
        cache = qlq.kv_cache(T, Hk, D, dev())
        s = torch.from_numpy(rng.permutation(T)).to(dev())
        got = qlq.norm_rope_kv_append(q, k, v, wq, wk, pos, f, cache, s, EPS, interleaved=inter, axes=ax)
        _check_rows(got, *_turned(q64, wq64, spin, inter))
        at = s.cpu().numpy()
        turned, top = _turned(k64, wk64, spin, inter)
        ks = oracle.fp16_decode(_values(cache.k_scales)[at])
        step = np.repeat(ks, 32, -1)
        kv = codes(cache.k_codes).view(np.int8)[at] * step
        assert np.max(np.abs(kv - turned) - step * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -6) - 24 * U * top) <= 0
        am = np.abs(turned).reshape(T, Hk, -1, 32).max(-1)
        assert np.max(np.abs(ks - am / 127) - 2.0 ** -11 * am / 127 - 2.0 ** -25 - 24 * U * top / 127) <= 0
        _, _, vq, vs = oracle.kv_quantize(bf16_bits(v), bf16_bits(v))
        assert np.array_equal(codes(cache.v_codes)[at] & 0x7F, vq & 0x7F) and np.array_equal(_values(cache.v_scales)[at], vs)


def test_eight_bits_with_axes_is_the_plain_append_on_one_axis():
    rng = np.random.default_rng(9)
    (q, _), (k, _), (v, _) = _rows(rng, 40, 4, 128), _rows(rng, 40, 2, 128), _rows(rng, 40, 2, 128)
    (f, pos, _), _ = _spin(rng, 40, 128, 1)
    a, b, s = qlq.kv_cache(40, 2, 128), qlq.kv_cache(40, 2, 128), torch.arange(40, device=dev())
    qa = qlq.rope_kv_append(q, k, v, pos, f, a, s)
    qb = qlq.rope_kv_append(q, k, v, pos[None].contiguous(), f, b, s, axes=torch.zeros(64, dtype=torch.int32, device=dev()))
    # angles of other roundings: neighbours at most
    assert (qa.view(torch.int16).int() - qb.view(torch.int16).int()).abs().max() <= 1
    assert (a.k_codes.int() - b.k_codes.int()).abs().max() <= 1
    assert torch.equal(a.v_codes, b.v_codes) and torch.equal(a.v_scales, b.v_scales)


def test_offsets_beyond_four_gigabytes():
    H, D = 16, 512
    pool = ((1 << 32) // (H * D // 2)) + 9
    cache = qlq.QuantizedKV4(*(torch.empty((pool, H, D // n), dtype=t, device=dev())
                               for n, t in ((2, torch.uint8), (32, torch.float16)) * 2))
    rng = np.random.default_rng(3)
    (k, k64), (v, v64) = _rows(rng, 3, H, D), _rows(rng, 3, H, D)
    s = torch.tensor([pool - 1, 0, pool - 7], device=dev())
    qlq.kv_append(k, v, cache, s)
    small = qlq.QuantizedKV4(*(t[s].contiguous() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)))
    _check_entries4(small, np.arange(3), k64, v64)
    for a, b in zip(qlq.kv_gather(cache, s), qlq.kv_gather(small, torch.arange(3, device=dev()))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [4, 8])
def test_captured_and_on_another_stream(bits):
    rng = np.random.default_rng(11)
    T, Hq, Hk, D = 24, 8, 2, 128
    q, k, v = (_rows(rng, T, h, D)[0] for h in (Hq, Hk, Hk))
    (wq, _), (wk, _) = _weight(rng, D), _weight(rng, D)
    (f, pos, ax), _ = _spin(rng, T, D, 3)
    s = torch.from_numpy(rng.permutation(64)[:T]).to(dev())
    cache, twin = (qlq.kv_cache(64, Hk, D, dev(), bits=bits) for _ in range(2))
    step = lambda c: qlq.norm_rope_kv_append(q, k, v, wq, wk, pos, f, c, s, axes=ax)
    side = torch.cuda.Stream()
    want = step(twin)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = step(cache)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(cache.k_codes, twin.k_codes)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(cache)
        gk, gv = qlq.kv_gather(cache, s)
        rq, rk = qlq.norm_rope(q, k, wq, wk, pos, f, axes=ax)
    for i in range(5):
        q.copy_(_rows(rng, T, Hq, D)[0])
        k.copy_(_rows(rng, T, Hk, D)[0])
        pos.add_(17)
        s.copy_(torch.from_numpy(rng.permutation(64)[:T]))
        want = step(twin)
        wk_, wv_ = qlq.kv_gather(twin, s)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(gk, wk_) and torch.equal(gv, wv_), i
        assert torch.equal(cache.k_codes, twin.k_codes) and torch.equal(cache.v_scales, twin.v_scales)
        for a, b in zip((rq, rk), qlq.norm_rope(q, k, wq, wk, pos, f, axes=ax)):
            assert torch.equal(a, b)


def test_binding_refusals_on_the_gpu():
    rng = np.random.default_rng(0)
    (q, _), (k, _), (w, _) = _rows(rng, 4, 2, 64), _rows(rng, 4, 2, 64), _weight(rng, 64)
    (f, pos, ax), _ = _spin(rng, 4, 64, 3)
    c4, c8, s = qlq.kv_cache(8, 2, 64, bits=4), qlq.kv_cache(8, 2, 64), torch.arange(4, device=dev())
    bad = [lambda: qlq.norm_rope(q.float(), k, w, w, pos, f, axes=ax),
           lambda: qlq.norm_rope(q, k[:3], w, w, pos, f, axes=ax),
           lambda: qlq.norm_rope(q, k, w.float(), w, pos, f, axes=ax),
           lambda: qlq.norm_rope(q, k, w[:32], w, pos, f, axes=ax),
           lambda: qlq.norm_rope(q, k, w.cpu(), w, pos, f, axes=ax),
           lambda: qlq.norm_rope(q, k, w, w, pos, f),                               # several axes without axes=
           lambda: qlq.norm_rope(q, k, w, w, pos[0], f, axes=ax),
           lambda: qlq.norm_rope(q, k, w, w, pos, f, axes=ax.long()),
           lambda: qlq.norm_rope(q, k, w, w, pos, f, axes=ax[:31]),
           lambda: qlq.norm_rope(q, k, w, w, pos.t().contiguous(), f, axes=ax),
           lambda: qlq.norm_rope(q, k, w, w, pos.float(), f, axes=ax),
           lambda: qlq.norm_rope(q, k, w, w, pos, f.float(), axes=ax),
           lambda: qlq.norm_rope(q, k, w, w, pos, f, axes=ax, k_out=k.float()),
           lambda: qlq.rope(q, pos, f),
           lambda: qlq.kv_append(k, k, qlq.kv_cache(8, 2, 96, bits=4), s),
           lambda: qlq.kv_append(k, k, qlq.QuantizedKV4(c8.k_codes, c8.k_scales, c8.v_codes, c8.v_scales), s),
           lambda: qlq.kv_append(k, k, qlq.QuantizedKV(c4.k_codes, c4.k_scales, c4.v_codes, c4.v_scales), s),
           lambda: qlq.kv_quantize(k, k, out=c4), lambda: qlq.kv_dequantize(c4),
           lambda: qlq.kv_gather(c4, s.float())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: qlq.norm_rope(q, k, w, w, pos, f, eps=0.0, axes=ax),
                 lambda: qlq.norm_rope(q, k, w, w, pos, f, attention_factor=float("nan"), axes=ax)):
        with pytest.raises(qlq.QlqError):
            call()


def _odd_values(rng, T, H, D, R):
    """Rows whose channels from R on hold infinities, NaNs and negative zeros beside ordinary values."""
    b = oracle.f32_to_bf16_bits(rng.standard_normal((T, H, D)).astype(np.float32))
    odd = np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x8000, 0x0000, 0x7F81, 0x0001], np.uint16)
    at = rng.random((T, H, D)) < 0.3
    at[..., :R] = False
    b[at] = rng.choice(odd, size=int(at.sum()))
    return b


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sizes", [(96, 32), (128, 64), (64, 10), (72, 20), (512, 34), (192, 96), (80, 2)])
def test_channels_that_do_not_rotate_are_copied(sizes, inter):
    D, R = sizes
    rng = np.random.default_rng(D + R)
    print(f"unrotated D={D} R={R} inter={inter}", flush=True)
    for T, H in ((5, 3), (900, 2)):
        b = _odd_values(rng, T, H, D, R)
        x, zero = bf16_to_gpu(b), torch.zeros(R // 2, dtype=torch.int32, device=dev())
        (f, pos, _), spin = _spin(rng, T, R, 1)
        got = [qlq.rope(x, pos[None].contiguous(), f, 0.75, inter, axes=zero), *qlq.norm_rope(x, x, None, None, pos, f, EPS, 0.75, inter)]
        in_place = x.clone()
        got.append(qlq.rope(in_place, pos[None].contiguous(), f, 0.75, inter, axes=zero, out=in_place))
        for g in got:
            assert np.array_equal(bf16_bits(g)[..., R:], b[..., R:]), "channels from R on"
            _check_rows(g[..., :R].contiguous(), *_turned(bits_to_f64(b[..., :R]), None, spin, inter, 0.75))


@pytest.mark.parametrize("inter", [False, True])
def test_infinities_that_do_not_rotate_on_their_way_into_the_cache(inter):
    # the entries of the plain append (8 bits), and the oracle's (4), in the groups of channels that do not rotate
    T, H, D, R = 40, 2, 128, 32
    rng = np.random.default_rng(3)
    b = oracle.f32_to_bf16_bits(rng.standard_normal((T, H, D)).astype(np.float32))
    at = rng.random((T, H, D - R)) < 0.05
    b[..., R:][at] = rng.choice(np.array([0x7F80, 0xFF80], np.uint16), size=int(at.sum()))
    x, s = bf16_to_gpu(b), torch.arange(T, device=dev())
    (f, pos, _), spin = _spin(rng, T, R, 1)
    plain, axes, four = qlq.kv_cache(T, H, D), qlq.kv_cache(T, H, D), qlq.kv_cache(T, H, D, bits=4)
    qlq.rope_kv_append(x, x, x, pos, f, plain, s, interleaved=inter)
    for c in (axes, four):
        q = qlq.rope_kv_append(x, x, x, pos[None].contiguous(), f, c, s, interleaved=inter, axes=torch.zeros(R // 2, dtype=torch.int32, device=dev()))
        assert np.array_equal(bf16_bits(q)[..., R:], b[..., R:])
    assert torch.equal(plain.k_codes[..., R:], axes.k_codes[..., R:])
    assert torch.equal(plain.k_scales[..., R // 32:], axes.k_scales[..., R // 32:])
    want, _ = _turned(bits_to_f64(b), None, spin, inter)
    _check_entries4(four, np.arange(T), want, bits_to_f64(b))


@pytest.mark.parametrize("inter", [False, True])
def test_a_norm_with_an_infinity_that_does_not_rotate(inter):
    # x / infinity: NaN where the infinity stands, zeros beside it
    rng = np.random.default_rng(4)
    x, _ = _rows(rng, 6, 2, 96)
    x[2, 1, 71] = float("inf")
    w, _ = _weight(rng, 96)
    (f, pos, _), _ = _spin(rng, 6, 32, 1)
    for g in qlq.norm_rope(x, x, w, w, pos, f, interleaved=inter):
        want = torch.zeros(96, dtype=torch.bool, device=dev())
        want[71] = True
        assert torch.equal(torch.isnan(g[2, 1]), want) and not g[2, 1][~want].any()
        assert bool(torch.isfinite(g[2, 0].float()).all()) and bool(torch.isfinite(g[3].float()).all())


@pytest.mark.parametrize("gains", [(2.0 ** 59, 2.0 ** 70, 1e-6), (2.0 ** -75, 2.0 ** -72, 2.0 ** -60), (2.0 ** -80, 2.0 ** -66, 2.0 ** -140),
                                   (2.0 ** 62, 2.0 ** 100, 1.0), (2.0 ** 120, 2.0 ** -90, 1e-6)])
def test_norms_whose_products_leave_fp32_beside_squares_that_do_not(gains):
    gain, wgain, eps = gains
    rng = np.random.default_rng(78)
    print(f"norm_rope range gain={gain:.0e} weight={wgain:.0e} eps={eps:.0e}", flush=True)
    for H, D in ((6, 128), (3, 72)):
        (x, x64), (f, spin) = _rows(rng, 9, H, D, gain), _spin(rng, 9, D, 1)
        wb = oracle.f32_to_bf16_bits((wgain * (1 + 0.3 * rng.standard_normal(D))).astype(np.float32))
        w, w64 = bf16_to_gpu(wb), bits_to_f64(wb)
        for inter in (False, True):
            want, top = _turned(x64, w64, spin, inter, eps=float(np.float32(eps)))
            for g in qlq.norm_rope(x, x, w, w, f[1], f[0], eps=eps, interleaved=inter):
                # (results below 2^-126: bf16's steps there are 2^-133, half of one is the rounding)
                over = np.abs(bits_to_f64(bf16_bits(g)) - want) - 2.0 ** -8 * np.abs(want) - 24 * U * top - 2.0 ** -134
                assert np.max(over) <= 0, f"D={D} inter={inter}: {np.max(over):.3e} beyond the bound"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads", [(2, 1, 256, 256), (3, 2, 512, 512), (1, 1, 512, 34), (2, 3, 480, 96)])
def test_wide_heads_of_many_tokens(heads, inter):
    # a wave per token, its largest rows: alone, into 4 bits and into 8
    Hq, Hk, D, R = heads
    rng = np.random.default_rng(D + R + 7)
    for T, n in ((801, 1), (1030, 2)):
        print(f"wide heads={heads} inter={inter} T={T}", flush=True)
        (q, q64), (k, k64), (v, v64) = _rows(rng, T, Hq, D), _rows(rng, T, Hk, D, 2.0), _rows(rng, T, Hk, D, 0.3)
        (wq, wq64), (wk, wk64) = _weight(rng, D), _weight(rng, D)
        (f, pos, ax), spin = _spin(rng, T, R, n)
        want, wantk = _turned(q64, wq64, spin, inter, 0.75), _turned(k64, wk64, spin, inter, 0.75)
        gq, gk = qlq.norm_rope(q, k, wq, wk, pos, f, EPS, 0.75, inter, ax)
        _check_rows(gq, *want)
        _check_rows(gk, *wantk)
        s = torch.from_numpy(rng.permutation(T)).to(dev())
        c4, c8, w8 = qlq.kv_cache(T, Hk, D, bits=4), qlq.kv_cache(T, Hk, D), qlq.kv_cache(T, Hk, D)
        for c in (c4, c8):
            assert torch.equal(qlq.norm_rope_kv_append(q, k, v, wq, wk, pos, f, c, s, EPS, 0.75, inter, ax), gq)
        _check_entries4(c4, s.cpu().numpy(), wantk[0], v64, f"T={T}")
        # 8 bits: V as the plain append has it, K within half a step and what the scale's rounding takes
        qlq.kv_append(k, v, w8, s)
        assert torch.equal(c8.v_codes, w8.v_codes) and torch.equal(c8.v_scales, w8.v_scales)
        at = s.cpu().numpy()
        step = np.repeat(oracle.fp16_decode(_values(c8.k_scales)[at]), 32, -1)
        kv = codes(c8.k_codes).view(np.int8)[at] * step
        assert np.max(np.abs(kv - wantk[0]) - step * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -6) - 24 * U * wantk[1]) <= 0
