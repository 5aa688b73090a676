"""GPU checks of the router's gradient at its edges: sigmoids that underflow
together, infinite centroids.

"DeepSeek_V3_Report：Annotation", eqs. (13), (15) and (17)-(20).
"""
import pytest
import torch

import tests.test_gpu_route_grad as base
import fp8_block_scaled_sigmoid_b200 as moe
from tests.test_gpu_route_grad import _call, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [16, 64, 256, 640])
def test_logits_whose_sigmoids_are_all_tiny(cuda_dev, E):
    """s' = s / sum s is a share like any other where every sigmoid is tiny or
    zero in 32 bits: rows of logits around -16 .. -1000 and the type's lowest.
    The reference takes the shares from log s.  Per share: expf within 2 ulps
    of an argument z - max(z) that is off by at most 2^-24 |z - max(z)| (16 at
    most here), a sum of E terms, a division and a few products: (E + 32)
    roundings of the magnitudes that cancel."""
    n_seq, S, d, alpha = 4, 10, 256, 0.5
    T = n_seq * S
    c = _case(T, E, d, 2, n_seq, 31, cuda_dev)
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).clamp(-3, 3)
    level = torch.tensor([-16.0, -18.0, -30.0, -60.0, -85.0, -88.0, -96.0, -103.0, -150.0, -1000.0]).repeat(n_seq)
    z = z * 2 + level[:, None]
    z[5] = torch.finfo(torch.float32).min     # the type's lowest everywhere: equal shares
    z[7, 1:] -= 70.0                          # one expert has it all
    z = z.float().to(cuda_dev)
    dz, du, dc = moe.moe_route_backward(None, z, c["idx"], c["gate"], c["u"], c["cent"], du_base=c["base"], f=c["f"],
                                        dloss=c["dloss"], alpha=alpha, seq_len=S)
    z64 = z.double()
    p = torch.softmax(torch.nn.functional.logsigmoid(z64), 1)
    rest = torch.sigmoid(-z64)
    cost = (alpha / S * c["dloss"].double()[:, None] * c["f"].double()).repeat_interleave(S, 0)
    mean = (p * cost).sum(1, keepdim=True)
    ref, mag = p * rest * (cost - mean), p * rest * (cost + mean)
    n = (E + 32) + torch.where(z64 < z64.amax(1, keepdim=True) - 16, 70.0, 0.0)
    err = (dz.double() - ref).abs()
    assert bool((err <= n * 2.0 ** -24 * mag + 1e-42).all()), float((err - n * 2.0 ** -24 * mag).max())
    dz64 = dz.double()
    ref = c["base"].double() + dz64 @ c["cent"].double()
    bound = (3 * E + 8) * 2.0 ** -23 * (dz64.abs() @ c["cent"].double().abs()) + 2.0 ** -23 * (ref.abs() + c["base"].double().abs())
    assert bool(((du.double() - ref).abs() <= bound).all())
    ref = dz64.T @ c["u"].double()
    bound = (3 * T + 8) * 2.0 ** -23 * (dz64.abs().T @ c["u"].double().abs()) + 2.0 ** -23 * ref.abs()
    assert bool(((dc.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("T,E", [(200, 144), (4100, 144), (4100, 384)])
def test_an_infinite_centroid_stays_in_its_column(cuda_dev, T, E):
    """An infinite element of a centroid reaches its own column of du alone:
    the others have the bits that they have with a zero in its place."""
    d = 384
    c = _case(T, E, d, 4, 0, 17, cuda_dev)
    c["cent"][5, 9] = 0.0
    want = _call(c, 0)
    c["cent"][5, 9] = float("inf")
    got = _call(c, 0)
    rest = torch.arange(d, device=cuda_dev) != 9
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert torch.equal(got[1][:, rest], want[1][:, rest])
    assert not bool(torch.isfinite(got[1][:, 9]).any())


@pytest.mark.parametrize("E", [384, 400])
def test_uneven_scales_with_more_experts(cuda_dev, E):
    """Where du is the product of half operands."""
    base.test_many_tokens_with_uneven_scales(cuda_dev, E)
