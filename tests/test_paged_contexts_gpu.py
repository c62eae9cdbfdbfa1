"""The paged cache's calls in more than one context of a device: a second context beside the first one, and one made
after it was destroyed (what a device reset leaves behind).  A new context loads the kernels anew, so what the library
has set for them (limits of shared memory) has to be set again there.

The checks run in a process of their own, through the C ABI, with the driver's own memory calls: torch knows one
context per device only.  All work is on the contexts' default streams, one call at a time."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

cuda = None


def ok(code):
    assert code == 0, f"driver error {code}"


class Memory:
    """Host arrays copied to the current context's device memory."""

    def __init__(self, arrays):
        self.host, self.ptr = arrays, {}
        for name, x in arrays.items():
            p = ctypes.c_uint64()
            ok(cuda.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(max(x.nbytes, 256))))
            ok(cuda.cuMemcpyHtoD_v2(p, x.ctypes.data_as(ctypes.c_void_p), ctypes.c_size_t(x.nbytes)))
            self.ptr[name] = p.value

    def read_and_free(self):
        ok(cuda.cuCtxSynchronize())
        got = {}
        for name, x in self.host.items():
            got[name] = np.empty_like(x)
            ok(cuda.cuMemcpyDtoH_v2(got[name].ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(self.ptr[name]),
                                    ctypes.c_size_t(x.nbytes)))
            ok(cuda.cuMemFree_v2(ctypes.c_uint64(self.ptr[name])))
        return got


def bf16(rng, *shape):
    return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def cache_of(rng, B, H, d, page, cap, count):
    max_pages = -(-cap // page)
    N = B * max_pages
    return dict(k=bf16(rng, N, H, page, d), v=bf16(rng, N, H, page, d),
                table=rng.permutation(N).astype(np.int32).reshape(B, max_pages),
                count=np.full((B, H), count, np.int32), seen=np.full((B, H), 3 * cap, np.int32),
                pos=rng.integers(0, 3 * cap, (N, H, page)).astype(np.int32),
                weight=rng.random((N, H, page)).astype(np.float32))


def calls():
    """Every kernel that needs more shared memory than a kernel has unasked, by a call each; all that they wrote."""
    from future_attention_targets_b200 import _binding as B
    from future_attention_targets_b200 import paged as P
    lib, rng = P.paged_lib(), np.random.default_rng(5)

    def struct(m, a, d, page, cap, Bn, H):
        c = P.CacheStruct(k_pages=m.ptr["k"], v_pages=m.ptr["v"], pos_pages=m.ptr["pos"], weight_pages=m.ptr["weight"],
                          page_table=m.ptr["table"], count=m.ptr["count"], seen=m.ptr["seen"], n_pages=a["k"].shape[0],
                          page_size=page, max_pages=a["table"].shape[1], batch=Bn, n_kv_heads=H, head_dim=d,
                          capacity=cap, dtype=P.BF16)
        c.k_stride[:] = c.v_stride[:] = [H * page * d, page * d, d]
        return c

    got = []
    for d, page, cap, Bn, H, m_new, window in ((64, 64, 48000, 1, 1, 20, 64), (128, 8, 16, 450, 1, None, 4)):
        a = cache_of(rng, Bn, H, d, page, cap, cap)
        T = Bn if m_new is None else m_new
        a |= dict(k_new=bf16(rng, T, H, d), v_new=bf16(rng, T, H, d), evicted=np.zeros((T, H), np.int32))
        m = Memory(a)
        cu = None if m_new is None else B._i32_host([0, m_new])
        st = lib.kvpop_paged_append_kv(m.ptr["k_new"], m.ptr["v_new"], H * d, cu, struct(m, a, d, page, cap, Bn, H), window,
                                       2, m.ptr["evicted"], None, None)
        assert st == B.OK, lib.kvpop_last_error()
        out = m.read_and_free()
        assert (out["evicted"] >= 0).all()
        got.append(out)
    for d in (64, 128):
        Bn, H, G, page, cap = 2, 2, 4, 16, 2000
        a = cache_of(rng, Bn, H, d, page, cap, 1990)
        a |= dict(q=bf16(rng, Bn, H * G, d), out=np.zeros((Bn, H * G, d), np.uint16), lse=np.zeros((Bn, H * G), np.float32))
        m = Memory(a)
        c = struct(m, a, d, page, cap, Bn, H)
        need = lib.kvpop_paged_decode_workspace_bytes(c, H * G, 1)
        ws = ctypes.c_uint64()
        ok(cuda.cuMemAlloc_v2(ctypes.byref(ws), ctypes.c_size_t(need)))
        st = lib.kvpop_paged_decode_attention(m.ptr["q"], H * G * d, H * G, c, 0.1, 1, m.ptr["out"], m.ptr["lse"], ws.value,
                                              need, None, None)
        assert st == B.OK, lib.kvpop_last_error()
        out = m.read_and_free()
        ok(cuda.cuMemFree_v2(ws))
        assert np.isfinite(out["lse"]).all() and (out["lse"] != 0).all()
        got.append(out)
    return got


def run_checks():
    global cuda
    cuda = ctypes.CDLL("libcuda.so.1")
    ok(cuda.cuInit(0))
    first = ctypes.c_void_p()
    ok(cuda.cuDevicePrimaryCtxRetain(ctypes.byref(first), 0))
    ok(cuda.cuCtxSetCurrent(first))
    want = calls()

    def same(where):
        for i, (x, y) in enumerate(zip(want, calls())):
            for name in x:
                assert np.array_equal(x[name].view(np.uint8), y[name].view(np.uint8)), (where, i, name)

    for turn in range(2):
        ctx = ctypes.c_void_p()
        ok(cuda.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))     # current from here on
        same(f"context {turn + 2}")
        ok(cuda.cuCtxSetCurrent(first))
        same("the first context again")
        ok(cuda.cuCtxDestroy_v2(ctx))
    ok(cuda.cuDevicePrimaryCtxRelease_v2(0))


@pytest.mark.gpu
def test_paged_calls_in_several_contexts():
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "CONTEXTS_OK" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])


if __name__ == "__main__":
    run_checks()
    print("CONTEXTS_OK")
