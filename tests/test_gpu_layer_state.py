"""GPU checks of what MoELayer keeps between forward_train and backward."""
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import MoELayer, _abi, configs, inputs, make_fp8_weights

pytestmark = pytest.mark.gpu


def _layer(dev, T=96, **kw):
    cfg = configs.TINY.with_(name="layer_state", T=T, d=256, E=16, G=4, M=2, K=4, I=256)
    w = make_fp8_weights(cfg, dev, pow2=kw.get("pow2", False))
    layer = MoELayer(cfg, inputs.draw_centroids(cfg, dev), inputs.draw_bias(cfg, dev), *w, **kw)
    u = inputs.draw_u(cfg, dev)
    dout = torch.randn(T, cfg.d, generator=torch.Generator().manual_seed(5)).to(dev) * 0.01
    return cfg, layer, u, dout


def test_backward_wants_the_last_pass_to_be_forward_train(cuda_dev):
    """The router's gradient belongs to one forward_train: after a forward of
    other tokens its routing is gone, and mixing the two passes is refused."""
    cfg, layer, u, dout = _layer(cuda_dev, router_grad=True)
    with pytest.raises(_abi.MoEError):
        layer.backward(dout)                  # nothing to go back through
    layer.forward_train(u, update_bias=False)
    want = layer.backward(dout)
    again = layer.backward(dout)              # as often as one likes
    for k in ("du", "dgate", "dlogits", "dcentroids", "dW1", "dW2"):
        assert torch.equal(want[k], again[k]), k
    other = u.flip(0).contiguous()
    layer.forward(other, update_bias=False)   # an evaluation step on the same layer
    with pytest.raises(_abi.MoEError):
        layer.backward(dout)
    with pytest.raises(_abi.MoEError):
        layer.backward(dout, weight_grads=False)
    layer.forward_train(u, update_bias=False)
    got = layer.backward(dout)
    for k in ("du", "dgate", "dlogits", "dcentroids"):
        assert torch.equal(want[k], got[k]), k
    graph, _ = layer.capture(other, update_bias=False)
    with pytest.raises(_abi.MoEError):
        layer.backward(dout)
    del graph


def test_a_layer_without_router_gradient_is_not_asked(cuda_dev):
    """Without router_grad nothing is refused that was not: a forward of the
    same tokens in between leaves the experts' gradients as they are."""
    cfg, layer, u, dout = _layer(cuda_dev)
    layer.forward_train(u, update_bias=False)
    want = layer.backward(dout)
    layer.forward(u, update_bias=False)
    got = layer.backward(dout)
    for k in ("du", "dW1", "dW2"):
        assert torch.equal(want[k], got[k]), k


def test_a_training_step_captured_whole(cuda_dev):
    """forward_train and backward in one graph, replayed after other passes."""
    cfg, layer, u, dout = _layer(cuda_dev, router_grad=True)
    layer.forward_train(u, update_bias=False)
    want = {k: v.clone() for k, v in layer.backward(dout).items() if k in ("du", "dgate", "dlogits", "dcentroids")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_train(u, update_bias=False)
        got = layer.backward(dout)
    layer.forward(u.flip(0).contiguous(), update_bias=False)
    graph.replay()
    for k, v in want.items():
        assert torch.equal(v, got[k]), k
    del graph
