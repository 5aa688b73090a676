"""GPU checks of how the router's gradient may be called: results left out,
captured and replayed, two calls at once."""
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import _abi
from tests.test_gpu_route_grad import _call, _case, _check

pytestmark = pytest.mark.gpu

# both products side by side: dC whole, dC in parts, du from half operands with dC in parts and whole
SIZES = [(1024, 256, 7168, 8), (3000, 16, 128, 2), (4608, 384, 384, 8), (4200, 384, 7168, 4)]


def _raw(c, dlogits, du, dc):
    """The C call, any of whose results may be NULL."""
    T, E = c["z"].shape
    d, K = c["u"].shape[1], c["idx"].shape[1]
    ws = torch.empty(_abi.moe_route_backward_workspace_size(T, d, E), dtype=torch.uint8, device=c["z"].device)
    p = lambda t: None if t is None else t.data_ptr()
    _abi._check(_abi.lib().moe_route_backward(
        p(c["dgate"]), p(c["z"]), p(c["idx"]), p(c["gate"]), p(c["u"]), d, p(c["cent"]), T, d, E, K, None, None, 0, 0.0,
        p(c["base"]), p(dlogits), p(du), p(dc), p(ws), ws.nbytes, None, torch.cuda.current_stream().cuda_stream), "raw")


@pytest.mark.parametrize("T,E,d,K", SIZES)
def test_results_left_out(cuda_dev, T, E, d, K):
    c = _case(T, E, d, K, 0, 41, cuda_dev)
    want = _call(c, 0)
    new = lambda *s: torch.full(s, float("nan"), device=cuda_dev)
    dz, du, dc = new(T, E), new(T, d), new(E, d)
    _raw(c, None, None, None)
    _raw(c, dz, None, None)
    assert torch.equal(dz, want[0])
    _raw(c, None, du, None)
    assert torch.equal(du, want[1])           # a tile of du is one CTA's, wherever it runs
    dz.fill_(float("nan"))
    _raw(c, dz, None, dc)
    assert torch.equal(dz, want[0])
    _check(c, 0, (dz, want[1], dc))           # dC's parts may be others without du beside them
    du.fill_(float("nan"))
    _raw(c, None, du, dc)
    assert torch.equal(du, want[1]) and torch.equal(dc, want[2])


@pytest.mark.parametrize("T,E,d,K", SIZES)
def test_captured_and_replayed(cuda_dev, T, E, d, K):
    """New contents behind the captured addresses, several replays in a row."""
    c = _case(T, E, d, K, 0, 42, cuda_dev)
    other = _case(T, E, d, K, 0, 43, cuda_dev)
    bufs = dict(dlogits=torch.empty(T, E, device=cuda_dev), du=torch.empty(T, d, device=cuda_dev),
                dcentroids=torch.empty(E, d, device=cuda_dev))
    _call(c, 0, **bufs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c, 0, **bufs)
    for _ in range(3):
        for k in ("dgate", "z", "idx", "gate", "u", "cent", "base"):
            c[k].copy_(other[k])
        for v in bufs.values():
            v.fill_(float("nan"))
        graph.replay()
        got = [bufs[k].clone() for k in ("dlogits", "du", "dcentroids")]
        want = _call(other, 0)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        other = _case(T, E, d, K, 0, 44, cuda_dev)
    del graph


def test_two_calls_at_once(cuda_dev):
    """Calls on two streams, each with its own scratch, share the SMs."""
    cases = [_case(T, E, d, K, 0, 45 + i, cuda_dev) for i, (T, E, d, K) in enumerate(SIZES[:1] + SIZES[2:])]
    want = [_call(c, 0) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(4):
        for c, s, g in zip(cases, streams, got):
            g.append(_call(c, 0, stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(w, one))
