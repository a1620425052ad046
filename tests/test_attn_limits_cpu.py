"""Calls of the attention half that its front end refuses, beyond those of test_attn_cpu.py."""
import os
import subprocess

import pytest
import torch

from memory_bound_decode_gb300 import binding, build_lib
from tests.test_attn_cpu import A16, ALIGN, INVALID, attn, cache, rope, tables


ROOM = 1 << 40   # a workspace's size that does for any shape


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


def test_status_array_alignment():
    assert binding.gemv_attn_decode(attn(status=A16 + 2), cache(), 0, check=False) == ALIGN


def evaluate(tmp_path, expressions):
    """C++ expressions over the internal header, as whole numbers."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include <cstdio>\n#include "gemv_attn_internal.h"\nint main() {\n'
                   + "".join(f'std::printf("%lld\\n", static_cast<long long>({e}));\n' for e in expressions) + "}\n")
    subprocess.run(["g++", "-std=c++17", "-I", build_lib.CSRC, "-I", os.path.join(build_lib.cuda_home(), "include"),
                    str(src), "-o", str(exe)], check=True)
    return [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]


def test_table_extent(tmp_path):
    """What is asked into the L2 before the lengths are known ends with the last request's row, also where the rows
    are a slice of wider ones; products in 64 bits."""
    cases = [(1, 4, 4), (1, 100, 4), (3, 9, 2), (0, 5, 5), (1 << 30, 1 << 31, 7)]
    got = evaluate(tmp_path, [f"gemv::attn_table_entries({r}LL, {s}LL, {w}LL)" for r, s, w in cases])
    assert got == [max(0, r - 1) * s + w if r else 0 for r, s, w in cases]


@pytest.mark.parametrize("kind", [binding.GEMV_CACHE_BF16, binding.GEMV_CACHE_FP8])
@pytest.mark.parametrize("name", ["page_stride", "head_stride", "slot_stride"])
@pytest.mark.parametrize("stride", [1 << 60, 1 << 61, 1 << 62, (1 << 63) - 16])
@pytest.mark.parametrize("one", [False, True])
def test_strides_whose_products_wrap(kind, name, stride, one):
    """Twice 2^62 wraps to a negative number, which is below any bound. One page, head or slot makes no difference."""
    f = {name: stride, "kind": kind}
    if one:
        f.update(num_pages=1, page_size=1)
    c = cache(**f)
    assert binding.gemv_attn_decode(attn(workspace_bytes=ROOM), c, 0, check=False) == INVALID
    r = rope(v=A16, v_stride=128, slots=A16)
    assert binding.gemv_rope_append(r, c, 0, check=False) == INVALID


@pytest.mark.parametrize("kind", [binding.GEMV_CACHE_BF16, binding.GEMV_CACHE_FP8])
def test_workspace_too_small(kind):
    """Refused on the host: an address without a size, a negative one, one below what a single CTA needs."""
    need = binding.gemv_attn_query(8, 2, 64, kind, 1)["workspace_bytes"]
    for over in (dict(), dict(workspace_bytes=0), dict(workspace_bytes=-1), dict(workspace_bytes=need - 1)):
        assert binding.gemv_attn_decode(attn(**over), cache(kind=kind), 0, check=False) == INVALID


def test_workspace_size_of_a_tensor():
    for n in (4096, 100):
        assert attn(workspace=torch.zeros(n, dtype=torch.uint8)).workspace_bytes == n
    assert attn(workspace=torch.zeros(64, dtype=torch.float32)).workspace_bytes == 256
    assert attn(workspace_bytes=7).workspace_bytes == 7


@pytest.mark.parametrize("requests", [(1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1])
def test_more_requests_than_are_counted(requests):
    assert binding.gemv_block_tables(tables(requests=requests), 0, check=False) == INVALID


@pytest.mark.parametrize("over", [dict(scale=0.125, softcap=1e-40), dict(scale=-1.0, softcap=1e-45),
                                  dict(scale=3e38), dict(scale=-3e38), dict(scale=1.0, softcap=3e38)])
def test_factors_past_fp32(over):
    """scale / softcap, or either in powers of two, is infinite in FP32: times a score of 0 it would be NaN."""
    assert binding.gemv_attn_decode(attn(**over, workspace_bytes=ROOM), cache(), 0, check=False) == INVALID
