"""GPU checks of the checkpointed combine on buffers longer than the pairs'
rows ("DeepSeek_V3_Report：Annotation", "Low-Precision Activation")."""
import pytest
import torch

import fp8_block_scaled_sigmoid_b200 as moe
from fp8_block_scaled_sigmoid_b200 import _abi

pytestmark = pytest.mark.gpu


def test_expert_outputs_with_the_shared_experts_behind(cuda_dev):
    """Y as the layer keeps it, T*K routed rows and T shared ones in one
    buffer: the checkpoint's first T*K rows are what the backward takes."""
    T, K, d = 40, 3, 256
    P = T * K
    g = torch.Generator().manual_seed(2)
    y = torch.randn(P + T, d, generator=g).to(cuda_dev)
    dst = torch.randperm(P, generator=g).view(T, K).int().to(cuda_dev)
    gate = torch.rand(T, K, generator=g).to(cuda_dev)
    u = torch.randn(T, d, generator=g).bfloat16().to(cuda_dev)
    dout = torch.randn(T, d, generator=g).to(cuda_dev)
    out, yq, ys = moe.moe_combine_checkpoint(y, dst, gate, y[P:], u)
    out2, yq2, ys2 = moe.moe_combine_checkpoint(y[:P], dst, gate, y[P:], u)
    assert torch.equal(out, out2) and torch.equal(yq[:P], yq2) and torch.equal(ys[:P], ys2)
    with pytest.raises(_abi.MoEError):
        moe.moe_combine_checkpoint_backward(dout, dst, gate, yq, ys)
    got = moe.moe_combine_checkpoint_backward(dout, dst, gate, yq[:P], ys[:P])
    want = moe.moe_combine_checkpoint_backward(dout, dst, gate, yq2, ys2)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))
