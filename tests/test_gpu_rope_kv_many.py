"""Rotary positions and cache append for as many tokens as a prompt has: two tokens per workgroup, the last one alone,
and head counts from one row to several batches of rows.  The checks are those of test_gpu_rope_kv.py."""
import pytest

import tests.test_gpu_rope_kv as few

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", [(2048, 2, 64, 64), (2049, 9, 128, 128), (2049, 1, 96, 24), (2501, 5, 512, 100)])
def test_rope(case, interleaved):
    few.test_rope_matches_the_oracle(case, interleaved)


@pytest.mark.parametrize("THD", [(2048, 2, 64), (2049, 8, 128), (2051, 1, 32), (2049, 3, 96)])
def test_append(THD):
    few.test_append_is_the_codec_bit_for_bit(THD)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", [(2048, 1, 1, 64, 64), (2049, 28, 4, 128, 128), (2049, 3, 1, 192, 48), (2501, 7, 2, 32, 20)])
def test_rope_kv_append(case, interleaved):
    few.test_rope_kv_append_matches_the_oracle(case, interleaved)
