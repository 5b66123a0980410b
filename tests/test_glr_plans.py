"""GPU tests of how the gated recurrence's calls are launched: what a call does is decided by its sizes, not by the
calls before it."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# The grids of a call's kernels, read from a captured graph.
GRIDS = r"""
import ctypes, sys
import torch
import linear_attention_prefill_gb300 as lap

cu = ctypes.CDLL("libcuda.so.1")


class Kernel(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")] \
        + [("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def grids(call):
    stream, graph, n = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_size_t()
    raw = ctypes.c_void_p(stream.cuda_stream)
    assert cu.cuStreamBeginCapture_v2(raw, 2) == 0
    call(stream)
    assert cu.cuStreamEndCapture(raw, ctypes.byref(graph)) == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        k = Kernel()
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        out.append((k.gx, k.bx))
    assert cu.cuGraphDestroy(graph) == 0
    return out


def fwd(N, T, D):
    x = torch.zeros(N, T, D, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    return grids(lambda s: lap.gdn_glr_chunk_fwd(x, x, y=y, output_final_state=False, stream=s))


def bwd(N, T, D):
    x = torch.zeros(N, T, D, dtype=torch.bfloat16, device="cuda")
    dx, dg, st = torch.empty_like(x), torch.empty_like(x), torch.zeros(N, (T + 63) // 64, D, device="cuda")
    return grids(lambda s: lap.gdn_glr_chunk_bwd(x, x, x, st, dx=dx, dg=dg, stream=s))


if sys.argv[1] == "short first":
    fwd(1, 10, 64), bwd(1, 10, 64), fwd(2, 33, 64), bwd(2, 33, 64)
print([f(*size) for size in ((20, 1024, 2560), (16, 2048, 2560), (1, 4096, 2560), (13, 640, 2560)) for f in (fwd, bwd)])
"""


def test_a_short_call_before_does_not_change_a_plan():
    out = [subprocess.run([sys.executable, "-c", GRIDS, how], capture_output=True, text=True, timeout=300)
           for how in ("", "short first")]
    assert all(o.returncode == 0 for o in out), out[0].stderr[-2000:] + out[1].stderr[-2000:]
    assert out[0].stdout == out[1].stdout and "(" in out[0].stdout
