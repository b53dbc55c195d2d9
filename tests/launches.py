"""What a call of the library launches: its kernels' names, grids, clusters and shared memory, and how many of
their CTAs an SM holds, read off a captured graph that is not run."""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

Launch = namedtuple("Launch", "name grid block smem cluster held")
RELAXED, KERNEL_NODE, CLUSTER_DIMENSION = 2, 0, 4


class _Params(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class _Attribute(ctypes.Union):
    _fields_ = [("pad", ctypes.c_char * 64), ("dim", ctypes.c_uint * 3)]


def launches(call):
    """The kernels that call(), which allocates nothing, launches on the current stream, in order."""
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(rc):
        assert rc == 0, f"CUDA driver error {rc}"

    def name(p):
        s = ctypes.c_char_p()
        if p.func:
            ok(cu.cuFuncGetName(ctypes.byref(s), ctypes.c_void_p(p.func)))
        else:
            ok(cu.cuKernelGetName(ctypes.byref(s), ctypes.c_void_p(p.kern)))
        return s.value.decode()

    def held(p):
        n = ctypes.c_int()
        ok(cu.cuOccupancyMaxActiveBlocksPerMultiprocessor(ctypes.byref(n), ctypes.c_void_p(p.func or p.kern),
                                                          p.block[0] * p.block[1] * p.block[2], ctypes.c_size_t(p.smem)))
        return n.value

    graph, stream = ctypes.c_void_p(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ok(cu.cuStreamBeginCapture_v2(ctypes.c_void_p(stream.cuda_stream), RELAXED))
        try:
            call()
        finally:
            rc = cu.cuStreamEndCapture(ctypes.c_void_p(stream.cuda_stream), ctypes.byref(graph))
    ok(rc)
    try:
        n = ctypes.c_size_t()
        ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
        nodes = (ctypes.c_void_p * n.value)()
        ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
        found = []
        for node in nodes:
            kind, p, a = ctypes.c_int(), _Params(), _Attribute()
            ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
            if kind.value != KERNEL_NODE:
                continue
            ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
            ok(cu.cuGraphKernelNodeGetAttribute(ctypes.c_void_p(node), CLUSTER_DIMENSION, ctypes.byref(a)))
            found.append(Launch(name(p), tuple(p.grid), tuple(p.block), p.smem, tuple(a.dim), held(p)))
        return found
    finally:
        ok(cu.cuGraphDestroy(graph))
