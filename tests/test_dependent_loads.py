"""Kernels launched as programmatic dependents read global memory through coherent loads only (no GPU needed).

Such a kernel may be resident while the kernel before it still writes.  griddepcontrol.wait orders its ordinary
loads behind those writes; the non-coherent path (__ldg, ld.global.nc, or what the compiler makes of a __restrict__
pointer to const) asks that the data be read-only for as long as the kernel is resident, which that data is not.
"""
import glob
import os
import re

import pytest

import bench

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "future_attention_targets_b200", "csrc")
WAITS = re.compile(r"griddepcontrol\.wait|\bgrid_wait\(\)")
NON_COHERENT = re.compile(r"\b__ldg\(|\bld\.global(\.\w+)*\.nc\b|\bld\.global\.nc\b|\bconst\b[^;(){}]*\b__restrict__")


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return bench.strip_comments(f.read())


@pytest.mark.parametrize("name", ["kvpop_paged.cuh", "paged_append.cu", "paged_compact.cu", "paged_decode.cu"])
def test_paged_kernels_load_coherently(name):
    code = code_of(name)
    assert WAITS.search(code) or name.endswith(".cuh")
    assert NON_COHERENT.search(code) is None, NON_COHERENT.search(code).group(0)


def test_every_paged_source_is_looked_at():
    assert sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "paged_*.cu"))) == [
        "paged_append.cu", "paged_compact.cu", "paged_decode.cu"]


SOURCES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


@pytest.mark.parametrize("name", [n for n in SOURCES if WAITS.search(code_of(n))])
def test_kernels_that_wait_load_coherently(name):
    """No source with such a kernel has a non-coherent load; a kernel beside it that is launched without the attribute
    may say __restrict__."""
    code = code_of(name)
    assert not re.search(r"\b__ldg\(|\bld\.global(\.\w+)*\.nc\b", code)
    for kernel in re.split(r"\b__global__\b", code)[1:]:
        if WAITS.search(kernel):
            assert "__restrict__" not in kernel[:kernel.index("{")]


def test_launches_with_the_attribute_are_all_looked_at():
    launching = [n for n in SOURCES if "cudaLaunchAttributeProgrammaticStreamSerialization" in code_of(n)]
    assert launching == ["attn_kernels.cu", "keep_mask.cu", "kvpop_paged.cuh", "static_cache.cu"]
    assert all(WAITS.search(code_of(n)) for n in launching)
