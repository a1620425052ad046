"""Calls of the attention half that its front end refuses, beyond those of test_attn_cpu.py."""
import pytest

from memory_bound_decode_gb300 import binding, build_lib
from tests.test_attn_cpu import A16, ALIGN, attn, cache


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def test_status_array_alignment():
    assert binding.gemv_attn_decode(attn(status=A16 + 2), cache(), 0, check=False) == ALIGN
