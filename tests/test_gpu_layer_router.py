"""GPU checks of MoELayer(router_grad=True) beyond one small batch: power-of-two
scales, batches on which the products are cut in parts or take half operands.

"DeepSeek_V3_Report：Annotation", eqs. (12), (13), (15) and (17)-(20),
"Low-Precision Activation".
"""
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import MoELayer, configs, inputs, make_fp8_weights
from tests.test_gpu_route_grad import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,G,M,K,pow2,S", [(264, 16, 4, 2, 4, True, 88), (1024, 32, 4, 2, 8, False, 256),
                                              (4224, 368, 1, 1, 4, True, 528)])
def test_training_step_with_the_router(cuda_dev, T, E, G, M, K, pow2, S):
    cfg = configs.TINY.with_(name="router_step", T=T, d=256, E=E, G=G, M=M, K=K, I=256)
    w = make_fp8_weights(cfg, cuda_dev, pow2=pow2)
    cent, bias = inputs.draw_centroids(cfg, cuda_dev), inputs.draw_bias(cfg, cuda_dev)
    plain = MoELayer(cfg, cent, bias.clone(), *w, pow2=pow2)
    layer = MoELayer(cfg, cent, bias.clone(), *w, pow2=pow2, balance_loss=True, seq_len=S, router_grad=True)
    u = inputs.draw_u(cfg, cuda_dev)
    dout = torch.randn(T, cfg.d, generator=torch.Generator().manual_seed(3)).to(cuda_dev) * 0.01
    dbal = torch.linspace(0.5, 1.5, T // S, device=cuda_dev)
    out = plain.forward_train(u, update_bias=False).clone()
    assert torch.equal(out, layer.forward_train(u, update_bias=False))
    r0, r1 = plain.backward(dout), layer.backward(dout, dbalance=dbal)
    layer.check()
    for k in ("dyq", "dys", "dy", "dx", "dW1", "dW2"):
        assert torch.equal(r0[k], r1[k]), k
    P = T * K
    dst = layer.perm["dst_of"].long()
    if pow2:
        assert bool((torch.frexp(layer.Ys)[0] == 0.5).all())
    y = (layer.Yq.view(torch.float8_e4m3fn).double().view(P, -1, 128) * layer.Ys.double()[..., None]).view(P, -1)[dst]
    prod = dout.double()[:, None] * y
    # d products and sums and a scale per tile, 2^-24 each
    bound = (cfg.d + 8) * 2.0 ** -24 * prod.abs().sum(2)
    assert bool(((r1["dgate"].double() - prod.sum(2)).abs() <= bound).all())
    c = dict(z=layer.logits, gate=layer.gate, dgate=r1["dgate"], idx=layer.idx, f=layer.balance.f, dloss=dbal, u=u,
             cent=cent, base=r0["du"])
    _check(c, T // S, (r1["dlogits"], r1["du"], r1["dcentroids"]), alpha=1e-4)
