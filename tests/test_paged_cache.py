"""The paged cache's C ABI on the CPU: the header and the binding agree, it compiles as C99, and every bad
argument is refused before any device call (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import future_attention_targets_b200 as kv
from future_attention_targets_b200 import _binding as B
from future_attention_targets_b200 import paged as P
from future_attention_targets_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000      # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    build()
    return P.paged_lib()


def struct(**kw):
    c = P.CacheStruct(k_pages=FAKE, v_pages=FAKE, pos_pages=FAKE, weight_pages=FAKE, page_table=FAKE, count=FAKE, seen=FAKE,
                      n_pages=40, page_size=16, max_pages=10, batch=2, n_kv_heads=2, head_dim=128, capacity=150, dtype=P.BF16)
    c.k_stride[:] = c.v_stride[:] = [2 * 16 * 128, 16 * 128, 128]
    for name, x in kw.items():
        if name in ("k_stride", "v_stride"):
            getattr(c, name)[:] = x
        else:
            setattr(c, name, x)
    return c


def test_header_and_binding_agree(lib):
    with open(P.PAGED_HEADER_PATH) as f:
        text = f.read()
    names = re.findall(r"KVPOP_API\s+[\w\s\*]+?\b(kvpop_\w+)\s*\(", text)
    assert set(names) == set(P.SIGS) and len(names) == 4
    for name in names:
        assert hasattr(lib, name)
    for name in ("PagedCache", "paged_append_kv", "paged_compact_kv", "paged_decode_attention", "paged_decode_workspace_bytes"):
        assert name in kv.__all__ and hasattr(kv, name)


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_is_c99_and_the_struct_matches(lib, tmp_path):
    fields = [n for n, _ in P.CacheStruct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvpop_paged.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", offsetof(kvpop_paged_cache, {n}));\n' for n in fields)
                   + '  printf("%zu\\n", sizeof(kvpop_paged_cache));\n'
                   + "  kvpop_paged_cache c = {0};\n"
                   + "  return kvpop_paged_decode_workspace_bytes(&c, 1, 0) == 0 ? 0 : 1;\n}\n")
    exe = tmp_path / "layout"
    libdir = os.path.dirname(B.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-L", libdir, "-lkvpop", f"-Wl,-rpath,{libdir}", "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0
    got = [int(x) for x in out.stdout.split()]
    assert got == [getattr(P.CacheStruct, n).offset for n in fields] + [ctypes.sizeof(P.CacheStruct)]


BAD_CACHES = [
    (dict(dtype=2), B.INVALID_ARG), (dict(head_dim=96), B.UNSUPPORTED), (dict(head_dim=256), B.UNSUPPORTED),
    (dict(page_size=4), B.UNSUPPORTED), (dict(page_size=24), B.UNSUPPORTED), (dict(page_size=2048), B.UNSUPPORTED),
    (dict(batch=0), B.INVALID_ARG), (dict(n_pages=0), B.INVALID_ARG), (dict(max_pages=-1), B.INVALID_ARG),
    (dict(n_kv_heads=0), B.INVALID_ARG), (dict(batch=65536), B.UNSUPPORTED), (dict(n_kv_heads=1025), B.UNSUPPORTED),
    (dict(capacity=0), B.INVALID_ARG), (dict(capacity=161), B.INVALID_ARG),
    (dict(max_pages=20000, capacity=131073), B.UNSUPPORTED),
    (dict(k_pages=None), B.INVALID_ARG), (dict(v_pages=None), B.INVALID_ARG), (dict(page_table=None), B.INVALID_ARG),
    (dict(count=None), B.INVALID_ARG), (dict(k_pages=FAKE + 8), B.INVALID_ARG), (dict(weight_pages=FAKE + 4), B.INVALID_ARG),
    (dict(k_stride=[-8, 0, 0]), B.INVALID_ARG), (dict(v_stride=[4096, 2048, 4]), B.INVALID_ARG),
    (dict(dtype=P.E4M3, k_stride=[4096, 2048, 8]), B.INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=lambda x: str(x))
def test_bad_caches_are_refused(lib, kw, code):
    c = struct(**kw)
    assert lib.kvpop_paged_decode_attention(FAKE, 512, 4, c, 0.1, 1, FAKE, FAKE, FAKE, 1 << 30, None, None) == code
    assert lib.kvpop_paged_append_kv(FAKE, FAKE, 256, None, c, 16, 4, FAKE, None, None) == code
    cu = B._i32_host([0] + [50] * max(2, min(c.batch, 3)))
    assert lib.kvpop_paged_compact_kv(FAKE, FAKE, FAKE, None, cu, 50, c, None, None) == code
    assert lib.kvpop_paged_decode_workspace_bytes(c, 4, 1) == 0
    assert lib.kvpop_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.INVALID_ARG), (dict(out=None), B.INVALID_ARG), (dict(q=FAKE + 2), B.INVALID_ARG),
    (dict(out=FAKE + 4), B.INVALID_ARG), (dict(scale=0.0), B.INVALID_ARG), (dict(scale=float("nan")), B.INVALID_ARG),
    (dict(heads=3), B.INVALID_ARG), (dict(heads=0), B.INVALID_ARG), (dict(heads=1 << 17), B.UNSUPPORTED),
    (dict(stride=-8), B.INVALID_ARG), (dict(stride=4), B.INVALID_ARG), (dict(ws=None), B.INVALID_ARG),
    (dict(nbytes=100), B.INVALID_ARG), (dict(ws=FAKE + 16), B.INVALID_ARG), (dict(cache=None), B.INVALID_ARG),
    (dict(cache=struct(weight_pages=None)), B.INVALID_ARG),
])
def test_decode_refuses(lib, kw, code):
    a = dict(q=FAKE, stride=512, heads=4, cache=struct(), scale=0.1, out=FAKE, ws=FAKE, nbytes=1 << 30) | kw
    assert lib.kvpop_paged_decode_attention(a["q"], a["stride"], a["heads"], a["cache"], a["scale"], 1, a["out"], None,
                                            a["ws"], a["nbytes"], None, None) == code
    assert lib.kvpop_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), B.INVALID_ARG), (dict(v=None), B.INVALID_ARG), (dict(k=FAKE + 2), B.INVALID_ARG),
    (dict(stride=12), B.INVALID_ARG), (dict(stride=-256), B.INVALID_ARG), (dict(window=-1), B.INVALID_ARG),
    (dict(sinks=-1), B.INVALID_ARG), (dict(window=147), B.INVALID_ARG), (dict(window=0, sinks=150), B.INVALID_ARG),
    (dict(cu=[0, 17, 17]), B.INVALID_ARG), (dict(cu=[0, 2, 1]), B.INVALID_ARG), (dict(cu=[1, 2, 3]), B.INVALID_ARG),
    (dict(cu=[0, 2, 4], window=0), B.INVALID_ARG),
    (dict(cache=struct(seen=None)), B.INVALID_ARG), (dict(cache=struct(pos_pages=None)), B.INVALID_ARG),
    (dict(cache=struct(weight_pages=None)), B.INVALID_ARG),
    (dict(cache=struct(batch=513), cu=[0] * 514), B.UNSUPPORTED),
])
def test_append_refuses(lib, kw, code):
    a = dict(k=FAKE, v=FAKE, stride=256, cu=None, cache=struct(), window=16, sinks=4) | kw
    cu = None if a["cu"] is None else B._i32_host(a["cu"])
    assert lib.kvpop_paged_append_kv(a["k"], a["v"], a["stride"], cu, a["cache"], a["window"], a["sinks"], None, None,
                                     None) == code
    assert lib.kvpop_last_error()


def test_append_of_no_tokens_enqueues_nothing(lib):
    assert lib.kvpop_paged_append_kv(FAKE, FAKE, 256, B._i32_host([0, 0, 0]), struct(), 16, 4, None, None, None) == B.OK


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), B.INVALID_ARG), (dict(v=FAKE + 8), B.INVALID_ARG), (dict(cu=None), B.INVALID_ARG),
    (dict(cu=[0, 20, 40]), B.INVALID_ARG), (dict(cu=[0, 60, 50]), B.INVALID_ARG), (dict(cu=[5, 20, 50]), B.INVALID_ARG),
    (dict(cache=struct(weight_pages=None)), B.INVALID_ARG), (dict(cache=struct(batch=513), cu=[0] * 513 + [50]), B.UNSUPPORTED),
    (dict(cu=[0, 131073, 131073], T=131073), B.UNSUPPORTED),
])
def test_compact_refuses(lib, kw, code):
    a = dict(k=FAKE, v=FAKE, cu=[0, 20, 50], T=50, cache=struct()) | kw
    cu = None if a["cu"] is None else B._i32_host(a["cu"])
    assert lib.kvpop_paged_compact_kv(a["k"], a["v"], FAKE, FAKE, cu, a["T"], a["cache"], None, None) == code
    assert lib.kvpop_last_error()


def test_workspace_covers_its_parts(lib):
    """Split maxima and sums, split outputs and scores: at least their bytes, more with weights than without."""
    for batch, heads, cap in ((1, 8, 4032), (64, 8, 4032), (1, 1, 131072), (3, 2, 8)):
        c = struct(batch=batch, n_kv_heads=heads, capacity=cap, max_pages=(cap + 15) // 16, n_pages=100000)
        for group in (1, 4, 20):
            hq = heads * group
            a, b = (lib.kvpop_paged_decode_workspace_bytes(c, hq, x) for x in (0, 1))
            assert a % 256 == 0 and b % 256 == 0 and b > a
            assert b < 4 << 30


def test_python_refuses_what_is_no_cache():
    import torch
    cpu = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        kv.PagedCache(cpu, cpu, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))
    for call in (lambda: kv.paged_decode_attention(cpu, None), lambda: kv.paged_append_kv(cpu, cpu, "cache", 1, 1),
                 lambda: kv.paged_compact_kv(cpu, cpu, None, [0, 1], 3)):
        with pytest.raises(TypeError, match="PagedCache"):
            call()


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 4, -2 ** 31 - 1, 4.0, "4", None])
def test_python_refuses_numbers_that_are_no_int32(value):
    """A number that does not fit is refused, not cut to its low 32 bits."""
    calls = [lambda: kv.paged_append_kv(None, None, None, value, 2), lambda: kv.paged_append_kv(None, None, None, 4, value)]
    if isinstance(value, int):
        calls.append(lambda: kv.paged_decode_workspace_bytes(None, value))
    for call in calls:
        with pytest.raises((TypeError, ValueError), match="window|sinks|n_q_heads"):
            call()


def test_python_takes_whole_numbers_of_any_type():
    np = pytest.importorskip("numpy")
    assert [P._i32(x, "x") for x in (np.int64(7), np.uint8(7), True, -2 ** 31, 2 ** 31 - 1)] == [7, 7, 1, -2 ** 31, 2 ** 31 - 1]
