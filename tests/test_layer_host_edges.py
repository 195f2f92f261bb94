"""Host-side checks (CPU only) of the operators between the linears at the ends of their sizes."""
import ctypes

import numpy as np
import pytest
import torch

import weight_quantized_linear_qlinear_amd as qlq
from oracle import layer
from weight_quantized_linear_qlinear_amd import binding

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced: refused before any launch


def _attention(T, B, Hq, Hk, D, max_pages, page, q_start):
    L = qlq.lib()
    st = L.qlq_kv_attention(FAKE, Hq * D, T, B, Hq, Hk, D, FAKE, FAKE, FAKE, FAKE, 1 << 20, FAKE, max_pages, page, FAKE,
                            q_start, 1.0, 1, 0, FAKE, None, FAKE, 1 << 40, None)
    return st, L.qlq_last_error().decode()


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: for machines without a GPU")
def test_attention_refuses_sizes_that_32_bits_cannot_count():
    # units of 32 tokens: 2^31 of them less than one per wave (the kernels round up to that)
    B = next(b for b in range(60000, 65536) if (1 << 31) % b < 1024 and (1 << 31) % b > 0)
    units = (1 << 31) // B
    assert (1 << 31) - 1024 < B * units < 1 << 31
    assert _attention(B, B, 1, 1, 128, units - 1, 32, None)[0] == 2
    # a sequence's query rows (tokens x heads of the group)
    assert _attention(1 << 21, 1, 1024, 1, 32, 1, 32, FAKE)[0] == 2


def test_attention_workspaces_of_many_streams_are_not_kept_for_ever(monkeypatch):
    # a program that makes a stream per request: the workspaces kept are those of the latest streams
    stream = [0]
    monkeypatch.setattr(binding, "_raw_stream", lambda index: stream[0])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(binding, "_attention_workspaces", {})
    cpu = torch.device("cpu")
    for stream[0] in range(1000):
        ws = binding._attention_workspace(cpu, 300000)
        assert ws.numel() == 300000 and not ws[:262144].any()
        assert binding._attention_workspace(cpu, 290000) is ws
        big = binding._attention_workspace(cpu, 310000)                # grown: in place of the smaller one
        assert big.numel() == 310000 and binding._attention_workspace(cpu, 300000) is big
    kept = binding._attention_workspaces
    assert len(kept) <= 64 and list(kept)[-1] == (None, 999)


# Channels of each pair (a, b) of 8 rotated ones, written out.
PAIRS = {False: [(0, 4), (1, 5), (2, 6), (3, 7)], True: [(0, 1), (2, 3), (4, 5), (6, 7)]}


def _rope_faults(rope):
    """What a rotation gets wrong: pair i turns by position * f[i] as a + i b times factor e^(i theta)."""
    rng = np.random.default_rng(3)
    f = np.array([1.0, 0.37, 0.083, 0.0021])
    x = rng.standard_normal((6, 2, 11))
    pos = np.array([0, 1, 2, 7, 1000, -3])
    faults = []
    for interleaved, pairs in PAIRS.items():
        y = rope(x, pos, f, 1.25, interleaved)
        for i, (a, b) in enumerate(pairs):
            want = 1.25 * (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos * f[i])[:, None]
            if not np.allclose(y[..., a] + 1j * y[..., b], want, rtol=0, atol=1e-12):
                faults.append((interleaved, i))
        if not np.array_equal(y[..., 8:], x[..., 8:]):
            faults.append((interleaved, "tail"))
    # by hand: a unit channel at position 1, frequencies pi / 2 and pi / 6
    s, h = np.sqrt(3) / 2, 0.5
    for interleaved, channel, want in ((False, 0, [0, 0, 1, 0]), (False, 1, [0, s, 0, h]), (False, 2, [-1, 0, 0, 0]),
                                       (False, 3, [0, -h, 0, s]), (True, 0, [0, 1, 0, 0]), (True, 1, [-1, 0, 0, 0]),
                                       (True, 2, [0, 0, s, h]), (True, 3, [0, 0, -h, s])):
        y = rope(np.eye(4)[channel].reshape(1, 1, 4), [1], [np.pi / 2, np.pi / 6], 1.0, interleaved)
        if not np.allclose(y[0, 0], want, rtol=0, atol=1e-15):
            faults.append((interleaved, f"unit {channel}"))
    return faults


def test_oracle_rope_turns_each_pair_by_its_own_angle():
    assert _rope_faults(layer.rope) == []
    # and the check finds a rotation that is none, one the wrong way, one with the other pairing or other frequencies
    for wrong in (lambda x, p, f, m, i: m * x, lambda x, p, f, m, i: layer.rope(x, -np.asarray(p), f, m, i),
                  lambda x, p, f, m, i: layer.rope(x, p, f, m, not i),
                  lambda x, p, f, m, i: layer.rope(x, p, f[::-1], m, i),
                  lambda x, p, f, m, i: layer.rope(x, p, f[::-1], m, not i),
                  lambda x, p, f, m, i: layer.rope(x, p, f, 1.0, i)):
        assert _rope_faults(wrong)
