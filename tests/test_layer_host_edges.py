"""Host-side checks (CPU only) of the operators between the linears at the ends of their sizes."""
import ctypes

import pytest
import torch

import weight_quantized_linear_qlinear_amd as qlq
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
