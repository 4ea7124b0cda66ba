"""Host tests of include/pa_q8.h beside test_q8_cpu.py's."""
import pytest

from paged_kv_gqa_pa_gb300 import binding
from paged_kv_gqa_pa_gb300 import build as pa_build
from paged_kv_gqa_pa_gb300 import q8


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return q8._lib()


@pytest.mark.parametrize("fn", ["pa_append", "pa_q8_append"])
def test_append_without_q_does_not_look_at_its_norm(lib, fn):
    tail = [None, None] if fn == "pa_q8_append" else []

    def call(q_heads, q_norm, k_norm, eps):
        return getattr(lib, fn)(0, q_heads, 2, 128, 128, 16, 8, 0, 0.0, eps, None, 512, None, 256, None,
                                256, q_norm, k_norm, None, None, None, 512, None, None, *tail, None, None)

    assert call(0, 0x10002, None, -1.0) == binding.PA_OK
    assert call(0, 0x10002, None, float("nan")) == binding.PA_OK
    assert call(0, None, 0x10000, -1.0) == binding.PA_ERR_INVALID_ARG
    assert call(4, 0x10000, None, -1.0) == binding.PA_ERR_INVALID_ARG
