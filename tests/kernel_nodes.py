"""Which kernels a call launches: it is captured, on a stream of its own, into
a graph that is read and thrown away, never run."""

import ctypes

import torch

_cu = None


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _call(name, *args):
    global _cu
    _cu = _cu or ctypes.CDLL("libcuda.so.1")
    status = getattr(_cu, name)(*args)
    assert status == 0, f"{name}: {status}"


def kernels_of(call):
    """(name, CTAs of a cluster, CTAs) of each kernel that call(stream) launches, which it must have done once before."""
    s = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
    torch.cuda.synchronize()
    _call("cuStreamBeginCapture_v2", handle, 1)  # of this thread's calls
    try:
        call(s)
    finally:
        _call("cuStreamEndCapture", handle, ctypes.byref(graph))
    n = ctypes.c_size_t()
    _call("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    _call("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    out = []
    for node in nodes:
        node, kind = ctypes.c_void_p(node), ctypes.c_int()
        _call("cuGraphNodeGetType", node, ctypes.byref(kind))
        if kind.value != 0:  # no kernel
            continue
        p, name, cluster = _KernelNode(), ctypes.c_char_p(), (ctypes.c_uint * 16)()
        _call("cuGraphKernelNodeGetParams_v2", node, ctypes.byref(p))
        if p.func:
            _call("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(p.func))
        else:
            _call("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(p.kern))
        _call("cuGraphKernelNodeGetAttribute", node, 4, cluster)  # the cluster's dimensions
        out.append((name.value.decode(), max(1, cluster[0]), p.grid[0]))
    _call("cuGraphDestroy", graph)
    return out
