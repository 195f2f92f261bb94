"""Host-side checks (CPU only) of the operators between the linears at the ends of their sizes."""
import ctypes

import pytest
import torch

import weight_quantized_linear_qlinear_amd as qlq

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
