"""The operators between the linears run together as a decoder layer uses them: norm to codes, the qkv linear,
rotary positions and the cache append, attention, the o linear, the next norm with the residual.

Every stage is checked against float64 from what the GPU gave the stage, so that no tolerance has to carry the
stages before it: the norm's codes and the rotated q and k by a half step of what they are rounded to (with 2^-18
relative for the fp32 steps before the rounding), the linears by this suite's tolerance for them, attention by the
half step of bf16 plus the 11 bits that weights (and, with many rows, K and V) have: a score A moves by 2^-11 A."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, check_close, codes, dev

pytestmark = pytest.mark.gpu

HID, HQ, HK, D, PAGE, PAGES = 256, 8, 2, 64, 16, 24
QKV = (HQ + 2 * HK) * D
EPS = 1e-5


class Layer:
    def __init__(self, qtype):
        rng = np.random.default_rng(11)
        w = lambda n, k: bf16_to_gpu(oracle.f32_to_bf16_bits((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32)))
        self.qtype = qtype
        self.wqkv, self.wo = qlq.quantize_weight(w(QKV, HID), qtype), qlq.quantize_weight(w(HID, HQ * D), qtype)
        self.g1, self.g2 = (bf16_to_gpu(oracle.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(HID)).astype(np.float32)))
                            for _ in range(2))
        self.freq, self.factor = qlq.rope_inv_freq(D, device=dev())

    def step(self, x, cache, positions, slots, table, lens, q_start=None, out=None, seen=None):
        """One layer on x [T, HID]; seen, if given, collects every stage's tensors."""
        T = x.shape[0]
        xq, xs = qlq.rms_norm_quant_dynamic(x, self.g1, self.qtype, EPS)
        qkv = qlq.qlinear_w8a8_dynamic(xq, xs, self.wqkv)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([HQ * D, HK * D, HK * D], dim=-1))
        rot = qlq.rope_kv_append(q, k, v, positions, self.freq, cache, slots, self.factor)
        att = qlq.kv_attention(rot, cache, table, lens, PAGE, q_start=q_start, out=out)
        aq, as_ = qlq.quantize_act_dynamic(att.reshape(T, HQ * D), self.qtype)
        o = qlq.qlinear_w8a8_dynamic(aq, as_, self.wo)
        yq, ys, h = qlq.rms_norm_quant_dynamic(o, self.g2, self.qtype, EPS, residual=x)
        if seen is not None:
            seen.update(x=x, xq=xq, xs=xs, qkv=qkv, rot=rot, att=att, aq=aq, as_=as_, o=o, yq=yq, ys=ys, h=h)
        return yq, ys, h


def _values(c, s, qtype):
    v = codes(c)
    v = v.view(np.int8).astype(np.float64) if qtype == "int8" else oracle.e4m3fn_decode(v).astype(np.float64)
    return v * s.cpu().numpy().astype(np.float64).reshape(-1, 1)


def _check_norm(x, w, c, s, qtype, residual=None):
    y, h = layer.rms_norm(bits_to_f64(bf16_bits(x)), bits_to_f64(bf16_bits(w)), EPS,
                          None if residual is None else bits_to_f64(bf16_bits(residual)))
    step = s.cpu().numpy().astype(np.float64).reshape(-1, 1)
    half = 0.5 * step if qtype == "int8" else np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * step)
    assert np.max(np.abs(_values(c, s, qtype) - y) - half * (1 + 2.0 ** -10) - 2.0 ** -18 * np.abs(y).max()) <= 0
    return h


def _check_linear(c, s, qw, got, qtype):
    w = codes(qlq.unpack_weight(qw))
    w = w.view(np.int8).astype(np.float64) if qtype == "int8" else oracle.e4m3fn_decode(w).astype(np.float64)
    ref = _values(c, s, qtype) @ (w * qw.scale.cpu().numpy().astype(np.float64)[:, None]).T
    check_close(bits_to_f64(bf16_bits(got)), ref)


def _cache_values(cache):
    kc, vc = codes(cache.k_codes).view(np.int8), codes(cache.v_codes)
    ks, vs = (t.cpu().numpy().astype(np.float64) for t in (cache.k_scales, cache.v_scales))
    P = kc.shape[0]
    k = (kc.reshape(P, HK, D // 32, 32) * ks[..., None]).reshape(P, HK, D)
    return k, oracle.e4m3fn_decode(vc).astype(np.float64) * vs[..., None], ks, vs


def _check_stages(lay, seen, cache, positions, slots, table, lens, starts, wide):
    qt, live = lay.qtype, slots.cpu().numpy() >= 0
    _check_norm(seen["x"], lay.g1, seen["xq"], seen["xs"], qt)
    _check_linear(seen["xq"], seen["xs"], lay.wqkv, seen["qkv"], qt)
    qkv = bits_to_f64(bf16_bits(seen["qkv"])).reshape(-1, HQ + 2 * HK, D)
    f = lay.freq.cpu().numpy()
    turned = layer.rope(qkv[:, :HQ + HK], positions.cpu().numpy(), f, lay.factor)
    big = np.abs(qkv).max()
    rot = bits_to_f64(bf16_bits(seen["rot"]))
    assert np.max(np.abs(rot - turned[:, :HQ]) - 2.0 ** -8 * np.abs(turned[:, :HQ]) - 2.0 ** -18 * big) <= 0
    k, v, ks, vs = _cache_values(cache)
    at = slots.cpu().numpy()[live]
    kstep = np.repeat(ks[at], 32, axis=-1)
    # K: half a step, and what the scale's rounding to fp16 (2^-11) takes off the largest codes
    assert np.max(np.abs(k[at] - turned[live, HQ:]) - kstep * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -6)) <= 0
    v64 = qkv[live, HQ + HK:]
    assert np.max(np.abs(v[at] - v64) - (2.0 ** -4 + 2.0 ** -10) * np.abs(v64) - 2.0 ** -9 * vs[at][..., None]) <= 0
    o64, _, written, S = layer.kv_attention(rot, k, v, table.cpu().numpy(), lens.cpu().numpy(), PAGE, starts)
    got = bits_to_f64(bf16_bits(seen["att"]))
    A = D ** -0.5 * np.abs(rot).sum(-1).max() * np.abs(k).max()
    W = 2.0 ** -11 + 2.0 ** -18 * (A + 16) + (2.0 ** -11 * (1 + 2 * A) if wide else 0.0)
    over = np.abs(got - o64) - 2.0 ** -8 * np.abs(o64) - S * W - 2.0 ** -19 * np.abs(v).max()
    assert np.max(over[written]) <= 0
    _check_linear(seen["aq"], seen["as_"], lay.wo, seen["o"], qt)
    h = _check_norm(seen["o"], lay.g2, seen["yq"], seen["ys"], qt, residual=seen["x"])
    hb = bits_to_f64(bf16_bits(seen["h"]))
    assert np.max(np.abs(hb - h) - 2.0 ** -8 * np.abs(h)) <= 0
    return written


def _rows(seed, T):
    rng = np.random.default_rng(seed)
    return bf16_to_gpu(oracle.f32_to_bf16_bits(rng.standard_normal((T, HID)).astype(np.float32)))


def _start(qtype):
    """A layer, an empty cache, and pages for three sequences (the third stays empty: a batch's padding)."""
    table = torch.from_numpy(np.random.default_rng(2).permutation(PAGES)[:21].reshape(3, 7).astype(np.int32)).to(dev())
    return Layer(qtype), qlq.kv_cache(PAGES * PAGE, HK, D, dev()), table


def _slots(table, b, t):
    return int(table[b, t // PAGE]) * PAGE + t % PAGE


def _prefill(lay, cache, table, lengths, seen=None):
    """Two prompts and padding rows behind them; (sequence lengths, slots, positions, out)."""
    T = sum(lengths) + 6
    pos = torch.tensor([t for n in lengths for t in range(n)] + [0] * 6, device=dev())
    slots = torch.tensor([_slots(table, b, t) for b, n in enumerate(lengths) for t in range(n)] + [-1] * 6, device=dev())
    lens = torch.tensor(lengths + [0], dtype=torch.int32, device=dev())
    starts = torch.tensor([0, lengths[0], sum(lengths), sum(lengths)], dtype=torch.int32, device=dev())
    out = torch.full((T, HQ, D), 7.0, dtype=torch.bfloat16, device=dev())
    lay.step(_rows(1, T), cache, pos, slots, table, lens, starts, out, seen)
    return pos, slots, lens, starts, out


@pytest.mark.parametrize("qtype", ["int8", "fp8_e4m3fn"])
def test_prompts_then_tokens(qtype):
    lay, cache, table = _start(qtype)
    before = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
    lengths, seen = [61, 5], {}
    pos, slots, lens, starts, out = _prefill(lay, cache, table, lengths, seen)
    written = _check_stages(lay, seen, cache, pos, slots, table, lens, starts.cpu().numpy(), wide=True)
    assert written.sum() == 66 and torch.all(out[66:] == 7.0)      # rows of no sequence: as they were
    used = torch.zeros(PAGES * PAGE, dtype=torch.bool, device=dev())
    used[slots[slots >= 0]] = True
    for a, b in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), before):
        assert torch.equal(a[~used], b[~used])                     # and so are entries of no slot
    for n in range(12):                                            # the first sequence crosses two page ends
        lengths = [lengths[0] + 1, lengths[1] + 1]
        pos = torch.tensor([lengths[0] - 1, lengths[1] - 1, 0], device=dev())
        slots = torch.tensor([_slots(table, 0, lengths[0] - 1), _slots(table, 1, lengths[1] - 1), -1], device=dev())
        lens = torch.tensor(lengths + [0], dtype=torch.int32, device=dev())
        seen = {}
        lay.step(_rows(100 + n, 3), cache, pos, slots, table, lens, seen=seen)
        _check_stages(lay, seen, cache, pos, slots, table, lens, np.arange(4), wide=False)
        assert torch.all(seen["att"][2] == 0)                      # a sequence without tokens


def test_captured_layer_replays_as_the_eager_one_runs():
    """Decode steps through one captured layer, its inputs changed in place; an eager twin on a second cache runs
    between the replays."""
    lay, cache, table = _start("fp8_e4m3fn")
    lengths = [61, 5]
    _prefill(lay, cache, table, lengths)
    twin = qlq.QuantizedKV(*(t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)))
    x, pos = _rows(5, 3), torch.zeros(3, dtype=torch.int64, device=dev())
    slots, lens = torch.full((3,), -1, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lay.step(x, cache, pos, slots, table, lens)                # (slots -1, lengths 0: changes nothing)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lay.step(x, cache, pos, slots, table, lens)
    for n in range(8):
        lengths = [lengths[0] + 1, lengths[1] + 1]
        x.copy_(_rows(200 + n, 3))
        pos.copy_(torch.tensor([lengths[0] - 1, lengths[1] - 1, 0]))
        slots.copy_(torch.tensor([_slots(table, 0, lengths[0] - 1), _slots(table, 1, lengths[1] - 1), -1]))
        lens.copy_(torch.tensor(lengths + [0], dtype=torch.int32))
        want = lay.step(x, twin, pos, slots, table, lens)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
        for a, b in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales),
                        (twin.k_codes, twin.k_scales, twin.v_codes, twin.v_scales)):
            assert torch.equal(a, b), n
