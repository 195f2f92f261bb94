"""Host-side checks of the operators between the linears (CPU only): refusals of the C ABI and of
the binding, the rotary frequencies, and the oracle against closed forms and brute force."""
import ctypes
import math

import numpy as np
import pytest
import torch

import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10008)


def _refused(name, *args, status=1, say=""):
    L = qlq.lib()
    st = getattr(L, name)(*args)
    msg = L.qlq_last_error().decode()
    assert st == status and say in msg, (name, st, msg)


# ------------------------------------------------------------------------------------- refusals
def test_norm_refusals():
    ok = dict(x=FAKE, r=None, w=FAKE, M=4, K=64, eps=1e-6, y=FAKE, ro=None)

    def norm(say="", status=1, **kw):
        a = {**ok, **kw}
        _refused("qlq_rms_norm", a["x"], a["r"], a["w"], a["M"], a["K"], a["eps"], a["y"], a["ro"], None, say=say,
                 status=status)
        a["y"] = a["y"] if a["y"] is None else ctypes.c_void_p(0x20000) if a["ro"] is None else a["y"]
        _refused("qlq_rms_norm_quant_static", a["x"], a["r"], a["w"], a["M"], a["K"], a["eps"], 1.0, 0, a["y"],
                 a["ro"], None, say=say, status=status)
        _refused("qlq_rms_norm_quant_dynamic", a["x"], a["r"], a["w"], a["M"], a["K"], a["eps"], 0, a["y"], FAKE,
                 a["ro"], None, say=say, status=status)

    for f in ("x", "w", "y"):
        norm(**{f: None}, say="null")
    for f in ("M", "K"):
        norm(**{f: 0}, say=">= 1")
        norm(**{f: (1 << 24) + 1}, say="2^24")
    for bad in (0.0, -1e-6, math.inf, math.nan):
        norm(eps=bad, say="eps")
    norm(ro=FAKE, say="residual")
    norm(r=FAKE, ro=FAKE, say="two buffers")
    norm(x=ODD, say="misaligned")
    norm(r=ODD, say="misaligned")
    _refused("qlq_rms_norm", FAKE, None, FAKE, 4, 64, 1e-6, ODD, None, None, say="misaligned")
    for bad in (0.0, -1.0, math.inf, math.nan):
        _refused("qlq_rms_norm_quant_static", FAKE, None, FAKE, 4, 64, 1e-6, bad, 0, FAKE, None, None,
                 say="input_scale")
    _refused("qlq_rms_norm_quant_static", FAKE, None, FAKE, 4, 64, 1e-6, 1.0, 7, FAKE, None, None, status=2)
    _refused("qlq_rms_norm_quant_dynamic", FAKE, None, FAKE, 4, 64, 1e-6, 7, FAKE, FAKE, None, None, status=2)
    _refused("qlq_rms_norm_quant_dynamic", FAKE, None, FAKE, 4, 64, 1e-6, 0, FAKE, None, None, None, say="null")
    _refused("qlq_rms_norm_quant_dynamic", FAKE, None, FAKE, 4, 64, 1e-6, 0, FAKE, ctypes.c_void_p(0x10002), None,
             None, say="misaligned")


def test_rope_refusals():
    ok = dict(x=FAKE, xs=256, T=4, H=2, D=128, pos=FAKE, p64=1, f=FAKE, R=128, m=1.0, out=FAKE, os=256)

    def rope(say, **kw):
        a = {**ok, **kw}
        _refused("qlq_rope", a["x"], a["xs"], a["T"], a["H"], a["D"], a["pos"], a["p64"], a["f"], a["R"], a["m"], 0,
                 a["out"], a["os"], None, say=say)

    for f in ("x", "pos", "f", "out"):
        rope("null", **{f: None})
    for f in ("T", "H", "D"):
        rope(">= 1", **{f: 0})
    rope("multiple of 8", D=100)
    rope("at most 512", D=520)
    for R in (0, 1, 63, 130):
        rope("rotary_dim", R=R)
    rope("factor", m=math.nan)
    rope("stride", xs=255)
    rope("stride", os=255)
    rope("stride", xs=-256, T=1)
    rope("equal strides", xs=512)
    rope("misaligned", x=ODD)
    rope("misaligned", pos=ctypes.c_void_p(0x10004))
    rope("misaligned", f=ctypes.c_void_p(0x10004))


def test_append_and_gather_refusals():
    ok = dict(k=FAKE, ks=256, v=FAKE, vs=256, T=4, H=2, D=128, s=FAKE, s64=1, pool=64, kc=FAKE, ksc=FAKE, vc=FAKE,
              vsc=FAKE)

    def append(say, **kw):
        a = {**ok, **kw}
        _refused("qlq_kv_append", a["k"], a["ks"], a["v"], a["vs"], a["T"], a["H"], a["D"], a["s"], a["s64"],
                 a["pool"], a["kc"], a["ksc"], a["vc"], a["vsc"], None, say=say)
        _refused("qlq_rope_kv_append", FAKE, 256, a["k"], a["ks"], a["v"], a["vs"], a["T"], 2, a["H"], a["D"], FAKE,
                 1, FAKE, 32, 1.0, 0, a["s"], a["s64"], a["pool"], a["kc"], a["ksc"], a["vc"], a["vsc"],
                 ctypes.c_void_p(0x40000), 256, None, say=say)

    for f in ("k", "v", "s", "kc", "ksc", "vc", "vsc"):
        append("null", **{f: None})
    for f in ("T", "H"):
        append(">= 1", **{f: 0})
    append("multiple of 32", D=80)
    append("at most 512", D=544)
    append("slots", pool=0)
    append("slots", pool=1 << 31)
    append("stride", ks=255)
    append("stride", vs=255)
    append("16-byte", kc=OFF8)
    append("16-byte", vc=OFF8)
    append("misaligned", s=ctypes.c_void_p(0x10004))
    for D, say in ((100, "multiple of 32"), (1056, "1024")):
        _refused("qlq_kv_gather", FAKE, FAKE, FAKE, FAKE, 64, 2, D, FAKE, 1, 4, FAKE, FAKE, None, say=say)
    _refused("qlq_kv_gather", FAKE, FAKE, FAKE, FAKE, 64, 2, 128, FAKE, 1, 0, FAKE, FAKE, None)
    _refused("qlq_kv_gather", FAKE, FAKE, FAKE, FAKE, 64, 2, 128, FAKE, 1, 4, OFF8, FAKE, None, say="16-byte")
    _refused("qlq_kv_gather", FAKE, FAKE, FAKE, FAKE, 64, 2, 128, None, 1, 4, FAKE, FAKE, None, say="null")


def test_attention_refusals():
    ok = dict(q=FAKE, qs=4096, T=4, B=4, Hq=32, Hk=8, D=128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pool=1024, bt=FAKE,
              mp=8, page=16, sl=FAKE, q0=None, scale=1.0, causal=1, window=0, out=FAKE, lse=None, ws=FAKE,
              wb=1 << 40)

    def attn(say, status=1, **kw):
        a = {**ok, **kw}
        _refused("qlq_kv_attention", *[a[f] for f in ("q", "qs", "T", "B", "Hq", "Hk", "D", "kc", "ks", "vc", "vs",
                                                     "pool", "bt", "mp", "page", "sl", "q0", "scale", "causal",
                                                     "window", "out", "lse", "ws", "wb")], None, say=say,
                 status=status)

    for f in ("q", "kc", "ks", "vc", "vs", "bt", "sl", "out"):
        attn("null", **{f: None})
    for f in ("T", "B", "Hq", "Hk", "mp"):
        attn(">= 1", **{f: 0})
    attn("multiple of KV heads", Hq=30)
    for D in (16, 48, 160, 512):
        attn("head_dim", status=2, D=D, qs=1 << 20)
    attn("one row per sequence", T=5)
    attn("stride", qs=4095)
    attn("16-byte", qs=4100)
    for f, say in (("q", "16-byte"), ("kc", "16-byte"), ("vc", "16-byte"), ("ks", "16-byte"), ("out", "misaligned")):
        attn(say, **{f: OFF8})
    attn("misaligned", vs=ODD)
    attn("misaligned", sl=ctypes.c_void_p(0x10002))
    attn("misaligned", lse=ctypes.c_void_p(0x10002))
    for page in (0, 3, 8, 24, 1 << 21):
        attn("power of two", page=page)
    attn("multiple of page_size", pool=1000)
    attn("2^31", mp=1 << 27, page=16)
    for bad in (math.inf, math.nan):
        attn("scale", scale=bad)
    attn("window", window=-1)
    attn("causal", window=5, causal=0)
    need = qlq.kv_attention_workspace_bytes(4, 4, 32, 8, 128)
    assert need > 262144
    attn("workspace", wb=need - 256)
    attn("workspace", ws=None)
    attn("256-byte", ws=ctypes.c_void_p(0x10010))
    attn("not supported", B=65537, T=65537)
    attn("not supported", Hq=1032, Hk=8, qs=1032 * 128)
    attn("too large", status=2, B=60000, T=60000, mp=1 << 17, page=16)


def test_workspace_sizes():
    w = qlq.kv_attention_workspace_bytes
    assert w(0, 0, 32, 8, 128) == 0 and w(4, 4, 32, 5, 128) == 0 and w(4, 4, 32, 8, 100) == 0
    assert w(5, 4, 32, 8, 128) == 0 and w(5, 4, 32, 8, 128, one_each=False) > 0
    for B in (1, 7, 64, 300, 1000):
        for Hq, Hk in ((1, 1), (28, 4), (32, 8), (64, 1), (128, 128), (1023, 1023), (1024, 1024)):
            for D in (32, 128, 256):
                for one in (True, False):
                    assert 262144 < w(B, B, Hq, Hk, D, one) < (1 << 31)
                    assert w(B, B, Hq, Hk, D, one) % 256 == 0


def test_binding_refusals():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    t3 = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    f, _ = qlq.rope_inv_freq(64, device="cpu")
    c = qlq.kv_cache(16, 2, 64, device="cpu")
    pos = torch.arange(4)
    with pytest.raises(ValueError):
        qlq.rms_norm(t, w)
    with pytest.raises(ValueError):
        qlq.rms_norm_quant_static(t, w, 1.0, "int8")
    with pytest.raises(ValueError):
        qlq.rms_norm_quant_dynamic(t, w, "int4")
    with pytest.raises(ValueError):
        qlq.rope(t3, pos, f)
    with pytest.raises(ValueError):
        qlq.kv_append(t3, t3, c, pos)
    with pytest.raises(ValueError):
        qlq.rope_kv_append(t3, t3, t3, pos, f, c, pos)
    with pytest.raises(ValueError):
        qlq.kv_gather(c, pos)
    with pytest.raises(ValueError):
        qlq.kv_attention(t3, c, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32), 16)
    for bad in ((0, 2, 64), (4, 0, 64), (4, 2, 48)):
        with pytest.raises(ValueError):
            qlq.kv_cache(*bad, device="cpu")


# ------------------------------------------------------------------------------------- frequencies
def test_inv_freq_rules():
    f0, m0 = qlq.rope_inv_freq(128, device="cpu")
    assert f0.dtype == torch.float64 and m0 == 1.0
    i = np.arange(64)
    assert np.allclose(f0.numpy(), 10000.0 ** (-2.0 * i / 128), rtol=1e-14)
    f, m = qlq.rope_inv_freq(128, scaling={"type": "linear", "factor": 4.0}, device="cpu")
    assert torch.equal(f, f0 / 4.0) and m == 1.0
    # ntk: the slowest pair is slowed by exactly the factor, the fastest is left alone
    f, _ = qlq.rope_inv_freq(128, scaling={"type": "ntk", "factor": 4.0}, device="cpu")
    assert f[0] == 1.0 and abs(float(f[-1] / f0[-1]) - 0.25) < 1e-12
    # yarn: unchanged above beta_fast turns over the original positions, / factor below beta_slow
    n = 32768
    f, m = qlq.rope_inv_freq(128, scaling={"type": "yarn", "factor": 4.0, "original_max_positions": n}, device="cpu")
    assert abs(m - (0.1 * math.log(4.0) + 1.0)) < 1e-15
    turns = n * f0.numpy() / (2 * math.pi)
    r = (f / f0).numpy()
    lo = math.floor(128 * math.log(n / (32 * 2 * math.pi)) / (2 * math.log(10000.0)))
    hi = math.ceil(128 * math.log(n / (2 * math.pi)) / (2 * math.log(10000.0)))
    assert np.allclose(r[:lo + 1], 1.0) and np.allclose(r[hi:], 0.25) and np.all(np.diff(r) <= 1e-15)
    assert np.all(turns[:lo] > 32.0) and np.all(turns[hi:] < 1.0)
    # llama3: by wavelength
    f, m = qlq.rope_inv_freq(128, 500000.0, {"type": "llama3", "factor": 8.0, "original_max_positions": 8192},
                             device="cpu")
    g, _ = qlq.rope_inv_freq(128, 500000.0, device="cpu")
    wave = 2 * math.pi / g.numpy()
    r = (f / g).numpy()
    assert np.allclose(r[wave < 8192 / 4.0], 1.0) and np.allclose(r[wave > 8192 / 1.0], 1 / 8.0)
    mid = (wave > 8192 / 4.0) & (wave < 8192)
    s = (8192 / wave[mid] - 1.0) / 3.0
    assert mid.any() and np.allclose(r[mid], (1 - s) / 8.0 + s)


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=64, base=1.0),
                                dict(rotary_dim=64, base=math.inf),
                                dict(rotary_dim=64, scaling={"type": "other", "factor": 2.0}),
                                dict(rotary_dim=64, scaling={"type": "linear", "factor": 0.0}),
                                dict(rotary_dim=64, scaling={"type": "linear", "beta_fast": 3}),
                                dict(rotary_dim=64, scaling={"type": "yarn", "factor": 2.0}),
                                dict(rotary_dim=2, scaling={"type": "ntk", "factor": 2.0}),
                                dict(rotary_dim=64, scaling={"type": "llama3", "factor": 2.0, "low_freq_factor": 4.0,
                                                             "original_max_positions": 8})])
def test_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        qlq.rope_inv_freq(device="cpu", **kw)


# ------------------------------------------------------------------------------------- the oracle
def test_oracle_norm_closed_form():
    x = np.array([[3.0, -4.0, 0.0, 0.0]])
    y, h = layer.rms_norm(x, np.array([1.0, 2.0, 3.0, 4.0]), 1e-30)
    assert np.allclose(y, [[3.0 / 2.5, -8.0 / 2.5, 0.0, 0.0]]) and np.array_equal(h, x)
    y2, h2 = layer.rms_norm(x, np.ones(4), 1e-30, residual=-x)
    assert not y2.any() and not h2.any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_is_a_rotation_by_position(interleaved):
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(8) / 8.0)
    q, k = rng.standard_normal((2, 5, 1, 24))
    # scores depend on the distance of positions only; the tail (channels 16..23) is untouched
    for shift in (0, 17, 100000):
        a = layer.rope(q, np.arange(5) + shift, f, interleaved=interleaved)
        b = layer.rope(k, np.arange(5) + shift, f, interleaved=interleaved)
        s = np.einsum("ihd,jhd->ij", a, b)
        if shift == 0:
            s0 = s
        assert np.allclose(s, s0, atol=1e-9) and np.array_equal(a[..., 16:], q[..., 16:])
    assert np.allclose(layer.rope(q, np.zeros(5), f, factor=2.0, interleaved=interleaved)[..., :16], 2 * q[..., :16])


def test_oracle_attention_masks_pages_and_empty_rows():
    rng = np.random.default_rng(1)
    Hq, Hk, D, page, pool = 4, 2, 32, 4, 32
    k, v = rng.standard_normal((2, pool, Hk, D))
    q = rng.standard_normal((6, Hq, D))
    table = np.array([[5, 2, 7], [1, 99, 3], [-1, 0, 0], [0, 0, 0]])
    lens, starts = [9, 10, 3, 0], [0, 3, 4, 5, 6]
    out, lse, written, _ = layer.kv_attention(q, k, v, table, lens, page, starts)
    assert written.all()
    # brute force, sequence 0 (three queries) and 1 (its page 99 does not exist: tokens 4..7 are left out)
    for row, toks in ((0, range(7)), (1, range(8)), (2, range(9)), (3, [0, 1, 2, 3, 8, 9])):
        b = 0 if row < 3 else 1
        for h in range(Hq):
            at = [table[b][t // page] * page + t % page for t in toks]
            s = np.array([q[row, h] @ k[a, h // 2] for a in at]) / math.sqrt(D)
            p = np.exp(s) / np.exp(s).sum()
            assert np.allclose(out[row, h], sum(pi * v[a, h // 2] for pi, a in zip(p, at)))
            assert np.allclose(lse[row, h], np.log(np.exp(s).sum()))
    # a sequence whose only page does not exist, and an empty one: nothing to see
    assert not out[4:].any() and np.all(np.isneginf(lse[4:]))
    # window 1 sees the token itself
    out1, _, _, _ = layer.kv_attention(q[:1], k, v, table[:1], [9], page, window=1)
    assert np.allclose(out1[0], np.repeat(v[table[0][2] * page + 0], 2, axis=0))
    # more queries than cached tokens: the first ones stand before the cache's first token
    out2, lse2, _, _ = layer.kv_attention(q[:3], k, v, table[:1], [1], page, [0, 3])
    assert not out2[:2].any() and np.isneginf(lse2[:2]).all() and np.allclose(out2[2], np.repeat(v[20], 2, axis=0))
