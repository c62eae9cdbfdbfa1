"""Which kernels a call launches: the call is captured, not run, and the captured graph's nodes are read through the
driver.  A test that is about one kernel or one way of dealing work out says so by this, so that it fails, and is not
left empty, when the choice between kernels changes."""
import ctypes

import torch


class KernelNodeParams(ctypes.Structure):        # CUDA_KERNEL_NODE_PARAMS_v2 of the driver API
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("shared_bytes", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kernel", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def launches(call):
    """[(mangled name, CTAs, threads per CTA)] of call(stream), in the graph's order; every buffer that the call needs
    has to be given to it."""
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(code):
        assert code == 0, f"driver error {code}"

    stream = torch.cuda.Stream()
    graph = ctypes.c_void_p()
    torch.cuda.synchronize()
    ok(cu.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), 2))        # relaxed
    try:
        call(stream)
    finally:
        ok(cu.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph)))
    try:
        n = ctypes.c_size_t()
        ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
        nodes = (ctypes.c_void_p * n.value)()
        ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
        got = []
        for node in nodes:
            p, name = KernelNodeParams(), ctypes.c_char_p()
            ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
            if p.func:
                ok(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
            else:
                ok(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kernel)))
            got.append((name.value.decode(), p.grid[0] * p.grid[1] * p.grid[2], p.block[0]))
        return got
    finally:
        ok(cu.cuGraphDestroy(graph))
