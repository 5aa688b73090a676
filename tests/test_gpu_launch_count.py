"""The kernels that the router's gradient says it launches, against the nodes
of a captured call."""
import ctypes

import pytest
import torch

import fp8_block_scaled_sigmoid_b200 as moe
from fp8_block_scaled_sigmoid_b200 import _abi
from tests.test_gpu_route_grad import _call, _case

pytestmark = pytest.mark.gpu


def _nodes(graph):
    rt = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    n = ctypes.c_size_t(0)
    assert rt.cudaGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("T,E,d,want_dc", [
    (40, 32, 256, True), (200, 256, 7168, True), (200, 256, 7168, False), (4608, 384, 384, True),
    (4608, 384, 384, False), (6000, 128, 2048, True),
])
def test_route_backward_counts_its_kernels(cuda_dev, T, E, d, want_dc):
    c = _case(T, E, d, 4, 0, 3, cuda_dev)
    kw = dict(dlogits=torch.empty(T, E, device=cuda_dev), du=torch.empty(T, d, device=cuda_dev), want_dcentroids=want_dc,
              dcentroids=torch.empty(E, d, device=cuda_dev) if want_dc else None,
              ws=torch.empty(_abi.moe_route_backward_workspace_size(T, d, E), dtype=torch.uint8, device=cuda_dev))
    _call(c, 0, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        n0 = _abi.launch_count
        _call(c, 0, **kw)
        counted = _abi.launch_count - n0
    assert counted == _nodes(graph)
    del graph


def test_an_empty_batch_launches_none(cuda_dev):
    c = _case(0, 32, 256, 4, 0, 11, cuda_dev)
    n0 = _abi.launch_count
    moe.moe_route_backward(c["dgate"], c["z"], c["idx"], c["gate"], c["u"], c["cent"])
    assert _abi.launch_count == n0
