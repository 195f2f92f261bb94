"""Host-side checks (CPU only) of the norms of query and key heads with the rotation, rotary axes, and the 4-bit cache:
refusals of the C ABI and of the binding."""
import ctypes
import math

import pytest
import torch

import weight_quantized_linear_qlinear_amd as qlq
from tests.test_layer_host import FAKE, ODD, OFF8, _refused

OUT, OUT2 = ctypes.c_void_p(0x40000), ctypes.c_void_p(0x80000)
OK = dict(q=FAKE, qs=512, k=FAKE, ks=256, T=4, Hq=4, Hk=2, D=128, wq=FAKE, wk=FAKE, eps=1e-6, pos=FAKE, p64=1, ax=None,
          n=1, f=FAKE, R=128, m=1.0, qo=OUT, qos=512)


def _norm_rope(say, status=1, **kw):
    a = {**OK, "ko": OUT2, "kos": 256, **kw}
    _refused("qlq_norm_rope", a["q"], a["qs"], a["k"], a["ks"], a["T"], a["Hq"], a["Hk"], a["D"], a["wq"], a["wk"], a["eps"],
             a["pos"], a["p64"], a["ax"], a["n"], a["f"], a["R"], a["m"], 0, a["qo"], a["qos"], a["ko"], a["kos"], None,
             say=say, status=status)


def _append(say, status=1, **kw):
    a = {**OK, **dict(v=FAKE, vs=256, s=FAKE, s64=1, pool=64, bits=4, kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE), **kw}
    _refused("qlq_norm_rope_kv_append", a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["Hq"], a["Hk"], a["D"],
             a["wq"], a["wk"], a["eps"], a["pos"], a["p64"], a["ax"], a["n"], a["f"], a["R"], a["m"], 0, a["s"], a["s64"],
             a["pool"], a["bits"], a["kc"], a["ksc"], a["vc"], a["vsc"], a["qo"], a["qos"], None, say=say, status=status)


@pytest.mark.parametrize("call", [_norm_rope, _append])
def test_shared_refusals(call):
    for f in ("q", "k", "pos", "f", "qo"):
        call("null", **{f: None})
    for f in ("T", "Hq", "D"):
        call(">= 1", **{f: 0})
    call("at most 512", D=544)
    for R in (0, 1, 63, 130):
        call("rotary_dim", R=R)
    call("factor", m=math.nan)
    for n in (0, -1, 17):
        call("n_axes", n=n, ax=FAKE)
    call("axis of each frequency", n=2, ax=None)
    for bad in (0.0, -1e-6, math.inf, math.nan):
        call("eps", eps=bad)
        call("eps", eps=bad, wk=None)
    for f in ("qs", "ks", "qos"):
        call("stride", **{f: 200})
    call("equal strides", qo=FAKE, qos=1024)
    for f in ("q", "k", "wq", "wk", "qo"):
        call("misaligned", **{f: ODD})
    call("misaligned", pos=ctypes.c_void_p(0x10004))
    call("misaligned", f=ctypes.c_void_p(0x10004))
    call("misaligned", ax=ctypes.c_void_p(0x10002), n=2)
    call("65536 heads", Hk=65537, ks=65537 * 128)


def test_norm_rope_refusals():
    _norm_rope("null", ko=None)
    _norm_rope("multiple of 8", D=100)
    _norm_rope(">= 1", Hk=-1)
    _norm_rope("stride", kos=200)
    _norm_rope("equal strides", ko=FAKE, kos=512)
    _norm_rope("misaligned", ko=ODD)


def test_append_refusals():
    for f in ("v", "s", "kc", "ksc", "vc", "vsc"):
        _append("null", **{f: None})
    _append(">= 1", Hk=0)
    _append("multiple of 32", D=80)
    for bits in (0, 2, 16):
        _append("4 or 8 bits", status=2, bits=bits)
    for pool in (0, 1 << 31):
        _append("slots", pool=pool)
    _append("stride", vs=200)
    _append("16-byte", kc=OFF8)
    _append("16-byte", vc=OFF8, bits=8)
    _append("misaligned", v=ODD)
    _append("misaligned", s=ctypes.c_void_p(0x10004))


def test_kv4_append_and_gather_refusals():
    ok = dict(k=FAKE, ks=256, v=FAKE, vs=256, T=4, H=2, D=128, s=FAKE, s64=1, pool=64, kc=FAKE, ksc=FAKE, vc=FAKE, vsc=FAKE)

    def append(say, **kw):
        a = {**ok, **kw}
        _refused("qlq_kv4_append", a["k"], a["ks"], a["v"], a["vs"], a["T"], a["H"], a["D"], a["s"], a["s64"], a["pool"],
                 a["kc"], a["ksc"], a["vc"], a["vsc"], None, say=say)
        if not {"k", "v", "ks", "vs"} & set(kw):
            _refused("qlq_kv4_gather", a["kc"], a["ksc"], a["vc"], a["vsc"], a["pool"], a["H"], a["D"], a["s"], a["s64"],
                     a["T"], FAKE, FAKE, None, say=say)

    for f in ("k", "v", "s", "kc", "ksc", "vc", "vsc"):
        append("null", **{f: None})
    for f in ("T", "H"):
        append(">= 1", **{f: 0})
    append("multiple of 32", D=80)
    append("at most 512", D=544)
    append("slots", pool=0)
    append("slots", pool=1 << 31)
    append("stride", ks=255)
    append("16-byte", vc=OFF8)
    append("misaligned", s=ctypes.c_void_p(0x10004))
    for out in ((None, FAKE), (FAKE, OFF8)):
        _refused("qlq_kv4_gather", FAKE, FAKE, FAKE, FAKE, 64, 2, 128, FAKE, 1, 4, *out, None)


def test_kv4_attention_refusals_and_workspace():
    ok = dict(q=FAKE, qs=4096, T=4, B=4, Hq=32, Hk=8, D=128, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pool=1024, bt=FAKE, mp=4,
              page=64, sl=FAKE, q0=None, scale=0.1, causal=1, window=0, out=OUT, lse=None, ws=FAKE, wb=1 << 30)

    def attention(say, status=1, **kw):
        a = {**ok, **kw}
        _refused("qlq_kv4_attention", *(a[f] for f in ok), None, say=say, status=status)

    for f in ("q", "kc", "ks", "vc", "vs", "bt", "sl", "out"):
        attention("null", **{f: None})
    attention("workspace", ws=None)
    attention("workspace", wb=qlq.kv_attention_workspace_bytes(4, 4, 32, 8, 128, True, 4) - 256)
    attention("16-byte", vs=OFF8)
    attention("16-byte", ks=OFF8)
    attention("16-byte", kc=OFF8)
    attention("head_dim", status=2, D=160, qs=5120)
    attention("multiple of KV heads", Hk=7)
    attention("power of two", page=48)
    attention("multiple of page_size", pool=1000)
    attention("one row per sequence", T=5)
    attention("window", window=-1)
    attention("causal", causal=0, window=5)
    attention("too large", status=2, B=65536, T=65536, mp=1 << 20, page=1024, pool=1 << 20)
    for n in (4, 8):
        b = qlq.kv_attention_workspace_bytes(4, 4, 32, 8, 128, True, n)
        assert b > 262144 and b % 256 == 0
    assert qlq.kv_attention_workspace_bytes(5, 4, 32, 8, 128, True, 4) == 0
    with pytest.raises(ValueError):
        qlq.kv_attention_workspace_bytes(4, 4, 32, 8, 128, True, 2)


def test_rope_axes():
    cpu = dict(device="cpu")
    assert qlq.rope_axes([3, 2, 2], **cpu).tolist() == [0, 0, 0, 1, 1, 2, 2]
    assert qlq.rope_axes([4, 2, 2], "cyclic", **cpu).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert qlq.rope_axes([2, 4], "cyclic", **cpu).tolist() == [0, 1, 0, 1, 1, 1]
    assert qlq.rope_axes([5], **cpu).tolist() == [0] * 5 and qlq.rope_axes([0, 3], **cpu).tolist() == [1] * 3
    assert qlq.rope_axes([5], **cpu).dtype == torch.int32
    for bad in ([], [0, 0], [-1, 3], [1] * 17):
        with pytest.raises(ValueError):
            qlq.rope_axes(bad, **cpu)
    with pytest.raises(ValueError):
        qlq.rope_axes([3, 3], "rows", **cpu)


def test_cache_of_four_bits_and_what_refuses_it():
    c = qlq.kv_cache(32, 2, 96, "cpu", bits=4)
    assert isinstance(c, qlq.QuantizedKV4) and c.k_codes.shape == (32, 2, 48) and c.v_scales.shape == (32, 2, 3)
    assert isinstance(qlq.kv_cache(32, 2, 96, "cpu"), qlq.QuantizedKV)
    with pytest.raises(ValueError):
        qlq.kv_cache(32, 2, 96, "cpu", bits=2)
    with pytest.raises(ValueError):
        qlq.kv_dequantize(c)
    x = torch.zeros(3, 2, 96, dtype=torch.bfloat16)
    f, pos = torch.ones(48, dtype=torch.float64), torch.arange(3)
    for call in (lambda: qlq.kv_quantize(x, x, out=c), lambda: qlq.norm_rope(x, x, None, None, pos, f),
                 lambda: qlq.norm_rope_kv_append(x, x, x, None, None, pos, f, c, pos),
                 lambda: qlq.kv_append(x, x, c, pos), lambda: qlq.kv_gather(c, pos)):
        with pytest.raises(ValueError):
            call()
