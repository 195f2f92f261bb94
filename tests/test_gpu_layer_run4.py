"""A decoder layer over the 4-bit cache as it runs: norm to codes, the qkv linear, norms of query and key heads with the
rotation of three axes and the append in one pass, attention, the o linear; prompts (one with an image), then single
tokens, padding rows among them; eager, and captured and replayed.

Every stage is checked against float64 from what the GPU gave the stage before it (test_gpu_layer_run.py); K and V against
the oracle's own codes."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_linear_qlinear_amd as qlq
from oracle import kvcache, layer
from tests.gpu_util import bf16_bits, bf16_to_gpu, bits_to_f64, codes, dev
from tests.test_gpu_head_rope import _check_entries4, _check_rows, _values
from tests.test_gpu_layer_run import _check_linear, _check_norm

pytestmark = pytest.mark.gpu

HID, HQ, HK, D, PAGE, PAGES = 256, 8, 2, 128, 16, 24
EPS = 1e-5


class Layer:
    def __init__(self, qtype):
        rng = np.random.default_rng(21)
        w = lambda n, k: bf16_to_gpu(oracle.f32_to_bf16_bits((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32)))
        g = lambda n: bf16_to_gpu(oracle.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(n)).astype(np.float32)))
        self.qtype = qtype
        self.wqkv = qlq.quantize_weight(w((HQ + 2 * HK) * D, HID), qtype)
        self.wo = qlq.quantize_weight(w(HID, HQ * D), qtype)
        self.g1, self.gq, self.gk = g(HID), g(D), g(D)
        self.freq, _ = qlq.rope_inv_freq(D, device=dev())
        self.axes = qlq.rope_axes([16, 24, 24], "cyclic", dev())

    def step(self, x, cache, positions, slots, table, lens, q_start=None, out=None, seen=None):
        T = x.shape[0]
        xq, xs = qlq.rms_norm_quant_dynamic(x, self.g1, self.qtype, EPS)
        qkv = qlq.qlinear_w8a8_dynamic(xq, xs, self.wqkv)
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([HQ * D, HK * D, HK * D], dim=-1))
        rot = qlq.norm_rope_kv_append(q, k, v, self.gq, self.gk, positions, self.freq, cache, slots, EPS, axes=self.axes)
        att = qlq.kv_attention(rot, cache, table, lens, PAGE, q_start=q_start, out=out)
        aq, as_ = qlq.quantize_act_dynamic(att.reshape(T, HQ * D), self.qtype)
        o = qlq.qlinear_w8a8_dynamic(aq, as_, self.wo)
        if seen is not None:
            seen.update(x=x, xq=xq, xs=xs, qkv=qkv, rot=rot, att=att, aq=aq, as_=as_, o=o)
        return o


def _check(lay, s, cache, positions, slots, table, lens, starts, wide):
    live = slots.cpu().numpy() >= 0
    _check_norm(s["x"], lay.g1, s["xq"], s["xs"], lay.qtype)
    _check_linear(s["xq"], s["xs"], lay.wqkv, s["qkv"], lay.qtype)
    qkv = bits_to_f64(bf16_bits(s["qkv"])).reshape(-1, HQ + 2 * HK, D)
    gq, gk = (bits_to_f64(bf16_bits(g)) for g in (lay.gq, lay.gk))
    pos, ax, f = positions.cpu().numpy(), lay.axes.cpu().numpy(), lay.freq.cpu().numpy()
    q, k = layer.norm_heads(qkv[:, :HQ], gq, EPS), layer.norm_heads(qkv[:, HQ:HQ + HK], gk, EPS)
    _check_rows(s["rot"], layer.rope(q, pos, f, axes=ax), np.abs(q).max(-1, keepdims=True))
    _check_entries4(cache, slots.cpu().numpy()[live], layer.rope(k, pos, f, axes=ax)[live], qkv[live, HQ + HK:])
    kv, vv = (kvcache.kv4_values(codes(c), _values(sc)) for c, sc in
              ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)))
    rot = bits_to_f64(bf16_bits(s["rot"]))
    o64, _, written, S = layer.kv_attention(rot, kv, vv, table.cpu().numpy(), lens.cpu().numpy(), PAGE, starts)
    A = D ** -0.5 * np.abs(rot).sum(-1).max() * np.abs(kv).max()
    W = 2.0 ** -11 + 2.0 ** -18 * (A + 16) + (2.0 ** -11 * (1 + 2 * A) if wide else 0.0)
    over = np.abs(bits_to_f64(bf16_bits(s["att"])) - o64) - 2.0 ** -8 * np.abs(o64) - S * W - 2.0 ** -19 * np.abs(vv).max()
    assert np.max(over[written]) <= 0
    _check_linear(s["aq"], s["as_"], lay.wo, s["o"], lay.qtype)
    return written


def _rows(seed, T):
    return bf16_to_gpu(oracle.f32_to_bf16_bits(np.random.default_rng(seed).standard_normal((T, HID)).astype(np.float32)))


def _slot(table, b, t):
    return int(table[b, t // PAGE]) * PAGE + t % PAGE


def _prefill(lay, cache, table, seen=None):
    """A prompt of 12 tokens, an image of 5 x 7 patches and 14 tokens, one of 5 tokens, and 6 padding rows."""
    first = [(t, t, t) for t in range(12)] + [(12, 12 + i // 7, 12 + i % 7) for i in range(35)]
    first += [(t, t, t) for t in range(19, 33)]
    lengths = [len(first), 5]
    pos = torch.tensor(first + [(t, t, t) for t in range(5)] + [(0, 0, 0)] * 6, device=dev()).t().contiguous()
    slots = torch.tensor([_slot(table, b, t) for b, n in enumerate(lengths) for t in range(n)] + [-1] * 6, device=dev())
    lens = torch.tensor(lengths + [0], dtype=torch.int32, device=dev())
    starts = torch.tensor([0, lengths[0], sum(lengths), sum(lengths)], dtype=torch.int32, device=dev())
    T = sum(lengths) + 6
    out = torch.full((T, HQ, D), 7.0, dtype=torch.bfloat16, device=dev())
    lay.step(_rows(1, T), cache, pos, slots, table, lens, starts, out, seen)
    return lengths, pos, slots, lens, starts, out


def _start(qtype):
    table = torch.from_numpy(np.random.default_rng(2).permutation(PAGES)[:21].reshape(3, 7).astype(np.int32)).to(dev())
    return Layer(qtype), qlq.kv_cache(PAGES * PAGE, HK, D, dev(), bits=4), table


@pytest.mark.parametrize("qtype", ["int8", "fp8_e4m3fn"])
def test_prompts_then_tokens(qtype):
    lay, cache, table = _start(qtype)
    before, seen = [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)], {}
    lengths, pos, slots, lens, starts, out = _prefill(lay, cache, table, seen)
    written = _check(lay, seen, cache, pos, slots, table, lens, starts.cpu().numpy(), wide=True)
    assert written.sum() == 66 and torch.all(out[66:] == 7.0)      # rows of no sequence: as they were
    used = torch.zeros(PAGES * PAGE, dtype=torch.bool, device=dev())
    used[slots[slots >= 0]] = True
    for a, b in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), before):
        assert torch.equal(a[~used], b[~used])                     # and so are entries of no slot
    for n in range(12):                                            # the first sequence crosses a page end
        lengths = [lengths[0] + 1, lengths[1] + 1]
        pos = torch.tensor([[32 + n, 4 + n, 0]] * 3, device=dev()) + 1
        slots = torch.tensor([_slot(table, 0, lengths[0] - 1), _slot(table, 1, lengths[1] - 1), -1], device=dev())
        lens, seen = torch.tensor(lengths + [0], dtype=torch.int32, device=dev()), {}
        lay.step(_rows(100 + n, 3), cache, pos, slots, table, lens, seen=seen)
        _check(lay, seen, cache, pos, slots, table, lens, np.arange(4), wide=False)
        assert torch.all(seen["att"][2] == 0)                      # a sequence without tokens


def test_captured_layer_replays_as_the_eager_one_runs():
    lay, cache, table = _start("fp8_e4m3fn")
    lengths = _prefill(lay, cache, table)[0]
    names = ("k_codes", "k_scales", "v_codes", "v_scales")
    twin = qlq.QuantizedKV4(*(getattr(cache, n).clone() for n in names))
    x, pos = _rows(5, 3), torch.zeros((3, 3), dtype=torch.int64, device=dev())
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
        pos.copy_(torch.tensor([[33 + n, 5 + n, 0]] * 3))
        slots.copy_(torch.tensor([_slot(table, 0, lengths[0] - 1), _slot(table, 1, lengths[1] - 1), -1]))
        lens.copy_(torch.tensor(lengths + [0], dtype=torch.int32))
        want = lay.step(x, twin, pos, slots, table, lens)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), n
        for a in names:
            assert torch.equal(getattr(cache, a), getattr(twin, a)), n
