"""GPU rotary positions, cache append and gather against the float64 oracle.

Tolerances (u = 2^-24): the reduced angle in [-pi, pi] is rounded once to fp32 (2^-23 absolute at most),
sine and cosine add 2 u: c and s are within 2^-22 of the exact ones (times the factor m, which adds a rounding:
below ROT = 2^-21 m).  a c - b s adds three roundings of at most (|a| + |b|) m: within (|a| + |b|) (ROT + 4 u m).
q is then rounded to bf16 (2^-8 relative).  K codes come from the fp32 value: a stored scale must lie between the
fp16 scales of the smallest and largest absmax within that bound, a code between the codes of the smallest and
largest value.  Without rotation everything is bit-exact (the codec's rules on the same bf16 values)."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _bits(rng, *shape, spread=True):
    a = rng.standard_normal(shape)
    if spread:
        a = a * 2.0 ** rng.integers(-5, 6, size=shape[:-1] + (1,))
    return oracle.f32_to_bf16_bits(a.astype(np.float32))


def _u16(t):
    return t.detach().cpu().view(torch.int16).numpy().view(np.uint16)


def _rot_error(x64, n, m, interleaved):
    """Bound on the fp32 rotation's error, per channel of x64 [T, H, D]."""
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    e = np.zeros_like(x64)
    both = np.abs(x64[..., ia]) + np.abs(x64[..., ib])
    e[..., ia] = e[..., ib] = both * abs(m) * (2.0 ** -21 + 4 * U)
    return e


def _rope_ref(bits, pos, f, m, interleaved):
    x = bits_to_f64(bits)
    return layer.rope(x, pos, f.cpu().numpy(), m, interleaved), _rot_error(x, len(f), m, interleaved)


def _check_q(got, ref, err, what):
    g = bits_to_f64(bf16_bits(got))
    over = np.abs(g - ref) - (2.0 ** -8 * np.abs(ref) + 1.01 * err + 1e-38)
    assert np.max(over) <= 0, f"{what}: {np.max(over):.3e} beyond the bound"


ROPE = [  # T, H, D, rotary_dim
    (1, 1, 8, 8), (5, 3, 64, 64), (3, 2, 64, 24), (7, 5, 128, 128), (2, 9, 96, 96), (4, 3, 128, 2), (2, 3, 72, 36),
    (3, 4, 256, 64), (2, 2, 512, 512), (1030, 3, 64, 32), (9, 40, 128, 100)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROPE)
def test_rope_matches_the_oracle(case, interleaved):
    T, H, D, R = case
    print(f"rope T={T} H={H} D={D} R={R} interleaved={interleaved}", flush=True)
    rng = np.random.default_rng(T + H + D + R)
    xb = _bits(rng, T, H, D)
    pos = rng.integers(0, 200000, size=T)
    pos[0] = 0
    f, m = qlq.rope_inv_freq(R, scaling={"type": "yarn", "factor": 4.0, "original_max_positions": 32768})
    ref, err = _rope_ref(xb, pos, f, m, interleaved)
    x = bf16_to_gpu(xb)
    p = torch.from_numpy(pos).to(dev())
    y = qlq.rope(x, p, f, m, interleaved)
    _check_q(y, ref, err, "rope")
    assert np.array_equal(bf16_bits(y)[..., R:], xb[..., R:]), "channels beyond rotary_dim"
    assert torch.equal(qlq.rope(x, p.int(), f, m, interleaved), y)
    # strided tokens in and out, not 16-byte aligned; the gaps stay as they were
    wide = torch.full((T, H * D + 3), 5.0, dtype=torch.bfloat16, device=dev())
    src = wide.as_strided((T, H, D), (H * D + 3, D, 1), 3)
    src.copy_(x)
    dst_buf = torch.full((T, H * D + 8), 9.0, dtype=torch.bfloat16, device=dev())
    dst = dst_buf.as_strided((T, H, D), (H * D + 8, D, 1), 0)
    assert torch.equal(qlq.rope(src, p, f, m, interleaved, out=dst), y)
    assert bool((dst_buf[:, H * D:] == 9.0).all())
    # in place, dense and strided
    assert torch.equal(qlq.rope(src, p, f, m, interleaved, out=src), y) and bool((wide[:, :3] == 5.0).all())
    assert torch.equal(qlq.rope(x, p, f, m, interleaved, out=x), y)


def test_rope_far_and_negative_positions():
    # angles are reduced in 64 bits: the same bound holds at positions of millions
    rng = np.random.default_rng(3)
    pos = np.array([0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, 1 << 36, -(1 << 36)])
    xb = _bits(rng, len(pos), 2, 128)
    f, _ = qlq.rope_inv_freq(128, 500000.0)
    # frequencies that are multiples of 2^-20, so that every product position * frequency is exact in float64
    f = torch.round(f * 2 ** 20).clamp(min=1) / 2 ** 20
    ref, err = _rope_ref(xb, pos, f, 1.0, False)
    y = qlq.rope(bf16_to_gpu(xb), torch.from_numpy(pos).to(dev()), f)
    _check_q(y, ref, err, "far positions")


APPEND = [(1, 4, 128), (5, 1, 32), (7, 3, 96), (16, 4, 128), (3, 2, 256), (2, 2, 512), (9, 12, 64), (4, 2, 192),
          (1100, 2, 64), (3, 1, 480)]


@pytest.mark.parametrize("THD", APPEND)
def test_append_is_the_codec_bit_for_bit(THD):
    T, H, D = THD
    print(f"append T={T} H={H} D={D}", flush=True)
    rng = np.random.default_rng(T * 31 + H + D)
    kb, vb = _bits(rng, T, H, D), _bits(rng, T, H, D)
    kb[0, 0, :32] = 0
    vb[-1, -1] = 0
    pool = T + 9
    slots = rng.permutation(pool)[:T]
    if T > 2:
        slots[1], slots[2] = -1, pool                  # padding and a slot outside: not written
    c = qlq.kv_cache(pool, H, D)
    before = [t.clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]
    wide = torch.zeros((T, 2 * H * D), dtype=torch.bfloat16, device=dev())     # one projection's k | v
    kg, vg = (wide.as_strided((T, H, D), (2 * H * D, D, 1), o) for o in (0, H * D))
    kg.copy_(bf16_to_gpu(kb))
    vg.copy_(bf16_to_gpu(vb))
    qlq.kv_append(kg, vg, c, torch.from_numpy(slots).to(dev()))
    kq, ks, vq, vs = oracle.kv_quantize(kb, vb)
    put = [i for i in range(T) if 0 <= slots[i] < pool]
    at = slots[put]
    assert np.array_equal(c.k_codes.cpu().numpy()[at], kq[put])
    assert np.array_equal(_u16(c.k_scales)[at], ks[put])
    assert np.array_equal(c.v_codes.cpu().numpy()[at], vq[put])
    assert np.array_equal(_u16(c.v_scales)[at], vs[put])
    rest = np.setdiff1d(np.arange(pool), at)
    for t, b in zip((c.k_codes, c.k_scales, c.v_codes, c.v_scales), before):
        assert torch.equal(t[rest], b[rest]), "entries of no token"
    # the same through int32 slots and unaligned rows
    c2 = qlq.kv_cache(pool, H, D)
    odd = torch.zeros((T * H * D + 1,), dtype=torch.bfloat16, device=dev())[1:].view(T, H, D)
    odd.copy_(kg)
    qlq.kv_append(odd, vg.contiguous(), c2, torch.from_numpy(slots.astype(np.int32)).to(dev()))
    assert torch.equal(c2.k_codes, c.k_codes) and torch.equal(c2.v_codes, c.v_codes)
    assert torch.equal(c2.k_scales, c.k_scales) and torch.equal(c2.v_scales, c.v_scales)


FUSED = [  # T, Hq, Hk, D, R
    (1, 1, 1, 32, 32), (5, 7, 1, 64, 64), (3, 28, 4, 128, 128), (4, 6, 2, 96, 48), (2, 16, 2, 256, 256),
    (6, 9, 3, 64, 20), (1030, 4, 2, 64, 64), (2, 3, 1, 192, 192)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", FUSED)
def test_rope_kv_append_matches_the_oracle(case, interleaved):
    T, Hq, Hk, D, R = case
    print(f"rope+append T={T} Hq={Hq} Hk={Hk} D={D} R={R} interleaved={interleaved}", flush=True)
    rng = np.random.default_rng(T + 3 * Hq + 5 * Hk + D + R)
    qb, kb, vb = _bits(rng, T, Hq, D), _bits(rng, T, Hk, D), _bits(rng, T, Hk, D)
    pos = rng.integers(0, 131072, size=T)
    f, m = qlq.rope_inv_freq(R, 500000.0, {"type": "llama3", "factor": 8.0, "original_max_positions": 8192})
    m = 1.25
    pool = T + 5
    slots = rng.permutation(pool)[:T]
    if T > 2:
        slots[2] = -1
    qkv = torch.zeros((T, (Hq + 2 * Hk) * D), dtype=torch.bfloat16, device=dev())
    stride = (Hq + 2 * Hk) * D
    q, k, v = (qkv.as_strided((T, h, D), (stride, D, 1), o * D) for h, o in ((Hq, 0), (Hk, Hq), (Hk, Hq + Hk)))
    for t, b in ((q, qb), (k, kb), (v, vb)):
        t.copy_(bf16_to_gpu(b))
    c = qlq.kv_cache(pool, Hk, D)
    p, s = torch.from_numpy(pos).to(dev()), torch.from_numpy(slots).to(dev())
    qo = qlq.rope_kv_append(q, k, v, p, f, c, s, attention_factor=m, interleaved=interleaved)
    _check_q(qo, *_rope_ref(qb, pos, f, m, interleaved), "q")
    assert np.array_equal(bf16_bits(q), qb) and np.array_equal(bf16_bits(k), kb), "inputs untouched"
    put = [i for i in range(T) if slots[i] >= 0]
    at = slots[put]
    # V: the codec, bit for bit
    _, _, vq, vs = oracle.kv_quantize(kb, vb)
    assert np.array_equal(c.v_codes.cpu().numpy()[at], vq[put]) and np.array_equal(_u16(c.v_scales)[at], vs[put])
    # K: between the codes of the bound's ends
    k64, err = _rope_ref(kb, pos, f, m, interleaved)
    k64, err = k64[put], err[put] * 1.01
    g = (len(put), Hk, D // 32, 32)
    mag = np.abs(k64).reshape(g)
    e = err.reshape(g)
    lo, hi = np.maximum(mag - e, 0).max(-1), (mag + e).max(-1)
    ks = oracle.fp16_decode(_u16(c.k_scales)[at])
    enc = lambda a: oracle.fp16_decode(oracle.fp16_encode((a / 127.0).astype(np.float32)))
    assert np.all(ks >= enc(lo * (1 - 2 * U))) and np.all(ks <= enc(hi * (1 + 2 * U))), "K scales"
    val, s2 = k64.reshape(g), ks[..., None]
    a, b = np.rint((val - e) / s2 * (1 - 2 * U * np.sign(val - e))), np.rint((val + e) / s2 * (1 + 2 * U * np.sign(val + e)))
    got = c.k_codes.cpu().numpy()[at].reshape(g).astype(np.float64)
    assert np.all(got >= np.clip(a, -127, 127)) and np.all(got <= np.clip(b, -127, 127)), "K codes"
    # rotating q in place gives the same bits
    c2 = qlq.kv_cache(pool, Hk, D)
    q_in = qlq.rope_kv_append(q, k, v, p.int(), f, c2, s.int(), attention_factor=m, interleaved=interleaved, q_out=q)
    assert torch.equal(q_in, qo) and torch.equal(c2.k_codes, c.k_codes) and torch.equal(c2.k_scales, c.k_scales)
    assert np.array_equal(bf16_bits(v), vb)


@pytest.mark.parametrize("THD", [(1, 1, 32), (300, 4, 128), (40, 3, 96), (5, 2, 1024)])
def test_gather_is_dequantize_of_chosen_slots(THD):
    T, H, D = THD
    rng = np.random.default_rng(T + D)
    c = qlq.kv_quantize(bf16_to_gpu(_bits(rng, T, H, D)), bf16_to_gpu(_bits(rng, T, H, D)))
    k_all, v_all = qlq.kv_dequantize(c)
    slots = torch.from_numpy(np.concatenate([rng.integers(0, T, size=2 * T), [-1, T, 0, 0]])).to(dev())
    for s in (slots, slots.int()):
        k, v = qlq.kv_gather(c, s)
        ok = (s >= 0) & (s < T)
        at = s.long().clamp(0, T - 1)
        assert torch.equal(k, torch.where(ok[:, None, None], k_all[at], torch.zeros_like(k)))
        assert torch.equal(v, torch.where(ok[:, None, None], v_all[at], torch.zeros_like(v)))


def test_append_and_gather_beyond_four_gigabytes():
    # slots whose code offset passes 2^32 bytes
    H, D = 8, 512
    pool = (1 << 32) // (H * D) + 64
    c = qlq.QuantizedKV(torch.empty((pool, H, D), dtype=torch.int8, device=dev()),
                        torch.empty((pool, H, D // 32), dtype=torch.float16, device=dev()),
                        torch.empty((pool, H, D), dtype=torch.uint8, device=dev()),
                        torch.empty((pool, H), dtype=torch.float16, device=dev()))
    rng = np.random.default_rng(1)
    kb, vb = _bits(rng, 4, H, D), _bits(rng, 4, H, D)
    slots = torch.tensor([pool - 1, 3, pool - 40, (1 << 31) // (H * D) + 1], device=dev())
    qlq.kv_append(bf16_to_gpu(kb), bf16_to_gpu(vb), c, slots)
    k, v = qlq.kv_gather(c, slots)
    kd, vd = oracle.kv_dequantize(*oracle.kv_quantize(kb, vb))
    assert np.array_equal(bf16_bits(k), kd) and np.array_equal(bf16_bits(v), vd)


def test_rope_binding_refusals_on_the_gpu():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=dev())
    f, _ = qlq.rope_inv_freq(64)
    pos = torch.arange(4, device=dev())
    c = qlq.kv_cache(8, 2, 64)
    bad = [lambda: qlq.rope(x.transpose(0, 1), pos, f), lambda: qlq.rope(x, pos[:3], f),
           lambda: qlq.rope(x, pos.float(), f), lambda: qlq.rope(x, pos, f.float()), lambda: qlq.rope(x, pos, f.cpu()),
           lambda: qlq.rope(x, pos.cpu(), f), lambda: qlq.rope(x, pos, f, out=x[:2]),
           lambda: qlq.kv_append(x, x[:, :1], c, pos), lambda: qlq.kv_append(x, x, qlq.kv_cache(8, 3, 64), pos),
           lambda: qlq.kv_append(x, x, qlq.kv_cache(8, 2, 64, device="cpu"), pos),
           lambda: qlq.rope_kv_append(x, x, x[:2], pos, f, c, pos), lambda: qlq.kv_gather(c, pos.float()),
           lambda: qlq.kv_gather(c, pos, k_out=x[:2])]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    f2, _ = qlq.rope_inv_freq(128)
    with pytest.raises(qlq.QlqError):
        qlq.rope(x, pos, f2)                           # rotary_dim above head_dim
