"""Which launches of the calls over rows sorted by group are dependent ones (FP8BLK_PDL)."""
import ctypes

import pytest
import torch

import fp8_blockwise_scaled_b200 as fb
from tests.gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


class _EdgeData(ctypes.Structure):
    """CUgraphEdgeData; type 1: the edge of a programmatic dependent launch."""
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte),
                ("reserved", ctypes.c_ubyte * 5)]


def _dependent_launches(call):
    """Programmatic edges of the graph that a captured call makes."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        out = call()
    most = 16
    count, data = ctypes.c_size_t(most), (_EdgeData * most)()
    ends = (ctypes.c_void_p * most)(), (ctypes.c_void_p * most)()
    status = ctypes.CDLL("libcuda.so.1").cuGraphGetEdges_v2(ctypes.c_void_p(graph.raw_cuda_graph()), *ends, data,
                                                            ctypes.byref(count))
    assert status == 0 and 0 < count.value <= most
    del graph, out
    return sum(e.type == 1 for e in data[:count.value])


@pytest.mark.parametrize("env,rows,dependent", [(None, 100, True), ("0", 100, False), ("1", 100, True),
                                                (None, 1000, False), ("0", 1000, False), ("1", 1000, True)])
def test_variable_decides_where_it_is_set(env, rows, dependent, monkeypatch):
    """Few rows a group launch dependently on their own; FP8BLK_PDL=0 turns that off, FP8BLK_PDL=1 on for all."""
    require_cuda()
    groups, n, k = 4, 128, 256
    x = torch.zeros((rows, k), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 10, 20, 30, rows], dtype=torch.int32, device="cuda")
    q, s = fb.fp8blk_quantize_weight_128x128(torch.zeros((groups * n, k), dtype=torch.bfloat16, device="cuda"))
    if env is None:
        monkeypatch.delenv("FP8BLK_PDL", raising=False)
    else:
        monkeypatch.setenv("FP8BLK_PDL", env)
    assert _dependent_launches(lambda: fb.grouped_linear_forward(x, q, s, off)) == int(dependent)
    assert fb.fp8blk_get_device_error() == 0
