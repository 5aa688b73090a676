"""GPU parity of the router's gradient (gates, sigmoid, balance loss, logits
product), of the same against differences, and of whole training steps.

"DeepSeek_V3_Report：Annotation", eqs. (13), (15) and (17)-(20).
"""
import numpy as np
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import MoELayer, _abi, configs, inputs, make_fp8_weights
import fp8_block_scaled_sigmoid_b200 as moe

pytestmark = pytest.mark.gpu


def _case(T, E, d, K, n_seq, seed, dev, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(T, d, generator=g).bfloat16()
    cent = (torch.randn(E, d, generator=g) / d ** 0.5).bfloat16()
    z = (u.float() @ cent.float().T) * spread
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]) if T else torch.zeros(0, K, dtype=torch.int64)
    a = torch.sigmoid(z)
    top = a.gather(1, idx)
    c = dict(u=u, cent=cent, z=z, idx=idx.int(), gate=top / top.sum(1, keepdim=True),
             dgate=torch.randn(T, K, generator=g), base=torch.randn(T, d, generator=g) * 0.01)
    c["f"] = torch.rand(n_seq, E, generator=g) * 3 if n_seq else None
    c["dloss"] = torch.rand(n_seq, generator=g) + 0.5 if n_seq else None
    return {k: None if v is None else v.to(dev) for k, v in c.items()}


def _call(c, n_seq, alpha=1e-2, **kw):
    T = c["z"].shape[0]
    return moe.moe_route_backward(c["dgate"], c["z"], c["idx"], c["gate"], c["u"], c["cent"], du_base=c["base"],
                                  f=c["f"], dloss=c["dloss"], alpha=alpha, seq_len=T // n_seq if n_seq else 0, **kw)


def _dlogits64(c, n_seq, alpha=1e-2):
    """(dlogits, sum of the magnitudes that cancel in it) in 64 bits."""
    z, g, dg = c["z"].double(), c["gate"].double(), c["dgate"].double()
    rest = torch.sigmoid(-z)
    idx = c["idx"].long()
    mean = (g * dg).sum(1, keepdim=True)
    dz = torch.zeros_like(z).scatter_add_(1, idx, g * (dg - mean)) * rest
    mag = torch.zeros_like(z).scatter_add_(1, idx, g * (dg.abs() + (g * dg.abs()).sum(1, keepdim=True))) * rest
    if n_seq:
        S = z.shape[0] // n_seq
        p = torch.sigmoid(z)
        p = p / p.sum(1, keepdim=True)
        cost = (alpha / S * c["dloss"].double()[:, None] * c["f"].double()).repeat_interleave(S, 0)
        m = (p * cost).sum(1, keepdim=True)
        dz = dz + p * rest * (cost - m)
        mag = mag + p * rest * (cost + m)
    return dz, mag


def _check(c, n_seq, out, alpha=1e-2):
    dlogits, du, dc = out
    T, E = c["z"].shape
    ref, mag = _dlogits64(c, n_seq, alpha)
    # fp32 chain: sigmoids within 4 ulps (expf 2, add, divide), the means sums
    # of at most E terms, a handful of products: (E + 32) roundings of the
    # magnitudes that cancel
    bound = (E + 32) * 2.0 ** -24 * mag + 1e-42
    err = (dlogits.double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    # the products of that dlogits: every operand exact (three bf16 terms hold
    # 24 bits), fp32 sums that may truncate (2^-23) at each of up to 3 terms
    # per depth, and one rounding of the result with the base
    dz = dlogits.double()
    ref = c["base"].double() + dz @ c["cent"].double()
    bound = (3 * E + 8) * 2.0 ** -23 * (dz.abs() @ c["cent"].double().abs()) + 2.0 ** -23 * (ref.abs() + c["base"].double().abs())
    err = (du.double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    if dc is None:
        return
    ref = dz.T @ c["u"].double()
    bound = (3 * T + 8) * 2.0 ** -23 * (dz.abs().T @ c["u"].double().abs()) + 2.0 ** -23 * ref.abs()
    err = (dc.double() - ref).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


CASES = [
    # T, E, d, K, n_seq
    (1, 16, 128, 1, 0), (1, 256, 7168, 8, 1), (37, 16, 256, 4, 0), (129, 80, 384, 6, 3), (128, 48, 640, 16, 4),
    (200, 256, 7168, 8, 0), (300, 384, 1152, 6, 2), (257, 1024, 256, 32, 1), (1000, 128, 2048, 2, 8),
    (2500, 272, 896, 8, 5), (4097, 64, 512, 4, 0), (4608, 272, 384, 8, 4),
    # dC's tiles in many equal parts, whole, two to a CTA; du in CTAs beside dC's and behind them
    (920, 384, 1024, 8, 1), (3000, 16, 128, 2, 0), (1024, 256, 7168, 8, 4), (1100, 1024, 5376, 4, 0),
    (2100, 512, 2048, 8, 0), (300, 384, 7168, 6, 1), (6000, 128, 2048, 8, 2),
]


@pytest.mark.parametrize("T,E,d,K,n_seq", CASES)
def test_against_the_formula(cuda_dev, T, E, d, K, n_seq):
    n_seq = n_seq if n_seq and T % n_seq == 0 else (1 if n_seq else 0)
    c = _case(T, E, d, K, n_seq, T + E, cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out = _call(c, n_seq, dev_err=err)
    assert int(err.item()) == 0
    _check(c, n_seq, out)
    # on the whole, well inside the worst case above: 3 T / 16 steps that each
    # lose up to 2^-23 of a partial sum, as independent errors
    # sqrt(3 * 2500 / 16) 2^-23 = 2.6e-6 of the result (with K = 1 there is
    # no gate gradient at all: both sides are zero)
    ref = _dlogits64(c, n_seq)[0].T @ c["u"].double()
    assert float((out[2].double() - ref).norm()) <= 4e-6 * float(ref.norm())
    again = _call(c, n_seq)
    assert all(torch.equal(a, b) for a, b in zip(out, again)), "not deterministic"
    # in place on the base
    du = c["base"].clone()
    c2 = dict(c, base=du)
    _call(c2, n_seq, du=du)
    assert torch.equal(du, out[1])


def test_extreme_logits(cuda_dev):
    """Saturated sigmoids: 1 - s keeps its digits, nothing is NaN."""
    c = _case(64, 64, 256, 4, 2, 9, cuda_dev, spread=30.0)
    out = _call(c, 2)
    assert all(bool(torch.isfinite(t).all()) for t in out)
    _check(c, 2, out)


@pytest.mark.parametrize("E", [48, 144])
def test_many_tokens_with_uneven_scales(cuda_dev, E):
    """Above 4096 tokens and 128 experts du is the product of scaled half operands: centroids
    and gradient rows of very different sizes, zero ones among them.  Two half
    terms hold dz within 2^-23 of a value and 2^-39 of its row's largest
    contribution top = max_e |dz_e| max|C_e| (half's smallest step is 2^-24,
    the row's largest value at least 2^14), a half centroid within 2^-39 of
    its largest element."""
    T, d, K = 4100, 384, 4
    c = _case(T, E, d, K, 4, 17, cuda_dev)
    c["cent"][3] = 0.0
    c["cent"][5] *= 2.0 ** 30
    c["cent"][7] *= 2.0 ** -60
    c["cent"][9, 100] = 3.0e4
    c["dgate"][10:20] = 0.0
    c["dgate"][20:30] *= 1e-20
    c["dgate"][30:40] *= 1e15
    c = {k: (v if k != "f" else None) for k, v in c.items()}
    c["dloss"] = None
    dlogits, du, dc = _call(c, 0)
    dz, cent = dlogits.double(), c["cent"].double()
    ref = c["base"].double() + dz @ cent.double()
    top = (dz.abs() * cent.abs().amax(1)).amax(1, keepdim=True)
    bound = ((3 * E + 8) * 2.0 ** -23 * (dz.abs() @ cent.abs()) + 2.0 ** -23 * (ref.abs() + c["base"].double().abs())
             + 3 * E * 2.0 ** -39 * top)
    assert bool(((du.double() - ref).abs() <= bound).all())
    assert torch.equal(du[10:20], c["base"][10:20])
    ref = dz.T @ c["u"].double()
    bound = (3 * T + 8) * 2.0 ** -23 * (dz.abs().T @ c["u"].double().abs()) + 2.0 ** -23 * ref.abs()
    assert bool(((dc.double() - ref).abs() <= bound).all())
    # a NaN stays in its token's row of du
    c["dgate"][50, 1] = float("nan")
    du2 = _call(c, 0)[1]
    rest = torch.arange(T, device=cuda_dev) != 50
    assert torch.equal(du2[rest], du[rest]) and bool(torch.isnan(du2[50]).all())


def test_parts_alone(cuda_dev):
    """The gates' part and the balance loss's part add up; with neither there
    is no gradient; without a base du is the product alone."""
    T, E, d, K = 96, 64, 256, 4
    c = _case(T, E, d, K, 3, 10, cuda_dev)
    gate_only = _call(dict(c, f=None, dloss=None), 0)[0]
    bal_only = moe.moe_route_backward(None, c["z"], c["idx"], c["gate"], c["u"], c["cent"], f=c["f"],
                                      dloss=c["dloss"], alpha=1e-2, seq_len=T // 3)
    both = _call(c, 3)[0]
    assert torch.allclose(gate_only + bal_only[0], both, rtol=0, atol=2.0 ** -23 * float(both.abs().max()) * 4)
    zero = moe.moe_route_backward(None, c["z"], c["idx"], c["gate"], c["u"], c["cent"])
    assert not any(bool(t.any()) for t in zero)
    ones = moe.moe_route_backward(None, c["z"], c["idx"], c["gate"], c["u"], c["cent"], f=c["f"], alpha=1e-2,
                                  seq_len=T // 3)
    one = moe.moe_route_backward(None, c["z"], c["idx"], c["gate"], c["u"], c["cent"], f=c["f"],
                                 dloss=torch.ones(3, device=cuda_dev), alpha=1e-2, seq_len=T // 3)
    assert all(torch.equal(a, b) for a, b in zip(ones, one))
    no_c = _call(c, 3, want_dcentroids=False)
    assert no_c[2] is None and torch.equal(no_c[0], both)


def test_empty_batch(cuda_dev):
    c = _case(0, 32, 256, 4, 0, 11, cuda_dev)
    dc = torch.full((32, 256), 5.0, device=cuda_dev)
    _, du, dc = _call(c, 0, dcentroids=dc)
    assert du.shape == (0, 256) and not dc.any()


def test_bad_index_is_reported(cuda_dev):
    c = _case(8, 16, 128, 2, 0, 12, cuda_dev)
    c["idx"][3, 1] = 16
    c["idx"][5, 0] = -7
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    dl, _, _ = _call(c, 0, dev_err=err)
    assert int(err.item()) == 3 and bool(torch.isfinite(dl).all())


def test_bad_index_leaves_the_rest_alone(cuda_dev):
    """A pair with a bad index is left out whatever its gradient holds."""
    c = _case(9, 32, 128, 4, 0, 21, cuda_dev)
    want = _call(dict(c, gate=c["gate"].clone().index_put_((torch.tensor([4]), torch.tensor([2])), torch.zeros(1, device=cuda_dev))), 0)
    c["idx"][4, 2] = 77
    for v in (float("nan"), float("inf")):
        c["dgate"][4, 2] = v
        err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        got = _call(c, 0, dev_err=err)
        assert int(err.item()) == 3
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T,E,K", [(1, 16, 2), (33, 48, 6), (70, 256, 32)])
def test_the_same_expert_twice(cuda_dev, T, E, K):
    """Pairs of one token that name the same expert add up."""
    c = _case(T, E, 256, K, 0, 23 + T, cuda_dev)
    c["idx"][:, 1] = c["idx"][:, 0]
    if K > 4:
        c["idx"][::2, 2:5] = c["idx"][::2, 5:6]
    out = _call(c, 0)
    _check(c, 0, out)
    assert all(torch.equal(a, b) for a, b in zip(out, _call(c, 0)))


def test_strided_tokens(cuda_dev):
    c = _case(50, 32, 256, 4, 0, 13, cuda_dev)
    want = _call(c, 0)
    wide = torch.zeros(50, 264, dtype=torch.bfloat16, device=cuda_dev)
    wide[:, :256] = c["u"]
    got = _call(dict(c, u=wide[:, :256]), 0)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_against_differences(cuda_dev):
    """Central differences in 64 bits of sum(dgate * gates(z)) + sum(dloss *
    loss(z)), with the selection and the counts f held fixed."""
    T, E, d, K, n_seq, alpha = 24, 16, 128, 3, 2, 0.3
    c = _case(T, E, d, K, n_seq, 14, cuda_dev)
    dl = _call(c, n_seq, alpha)[0].double().cpu()
    z, idx, dg, f, dloss = (c[k].cpu() for k in ("z", "idx", "dgate", "f", "dloss"))
    S = T // n_seq

    def value(z64):
        s = torch.sigmoid(z64)
        top = s.gather(1, idx.long())
        gates = top / top.sum(1, keepdim=True)
        p = (s / s.sum(1, keepdim=True)).view(n_seq, S, E).mean(1)
        loss = alpha * (f.double() * p).sum(1)
        return (dg.double() * gates).sum() + (dloss.double() * loss).sum()

    h = 1e-4
    for t, e in [(0, int(idx[0, 0])), (5, int(idx[5, 2])), (11, 7), (23, 15), (12, 0)]:
        zp, zm = z.double().clone(), z.double().clone()
        zp[t, e] += h
        zm[t, e] -= h
        diff = float((value(zp) - value(zm)) / (2 * h))
        # h^2 times the third derivative (|sigmoid'''| <= 1/8; the values are O(1)), fp32 rounding
        assert abs(diff - float(dl[t, e])) <= 1e-8 + 64 * 2.0 ** -24


def test_graph_replay(cuda_dev):
    c = _case(160, 64, 512, 4, 2, 15, cuda_dev)
    bufs = dict(dlogits=torch.empty(160, 64, device=cuda_dev), du=torch.empty(160, 512, device=cuda_dev),
                dcentroids=torch.empty(64, 512, device=cuda_dev),
                ws=torch.empty(_abi.moe_route_backward_workspace_size(160, 512, 64), dtype=torch.uint8,
                               device=cuda_dev))
    _call(c, 2, **bufs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(c, 2, **bufs)
    c["dgate"].copy_(torch.randn(160, 4))
    graph.replay()
    got = [bufs[k].clone() for k in ("dlogits", "du", "dcentroids")]
    want = _call(c, 2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del graph


def test_refusals(cuda_dev):
    E = _abi.MoEError
    c = _case(32, 32, 256, 4, 2, 16, cuda_dev)
    bad = [
        dict(dgate=c["dgate"].half()), dict(dgate=c["dgate"][:, :2]), dict(z=c["z"].double()),
        dict(idx=c["idx"].long()), dict(u=c["u"].float()), dict(u=c["u"][:16]), dict(cent=c["cent"].float()),
        dict(cent=c["cent"][:, :128].contiguous()), dict(f=c["f"][:1]), dict(dloss=c["dloss"][:1]),
        dict(base=c["base"].double()), dict(gate=c["gate"].cpu()),
    ]
    for kw in bad:
        with pytest.raises(E):
            _call(dict(c, **kw), 2)
    with pytest.raises(E):
        moe.moe_route_backward(None, c["z"], c["idx"], c["gate"], c["u"], c["cent"], f=c["f"], seq_len=5)
    with pytest.raises(E):                    # scratch too small
        _call(c, 2, ws=torch.empty(16, dtype=torch.uint8, device=cuda_dev))
    with pytest.raises(E):                    # 24 experts: not a multiple of 16
        moe.moe_route_backward(None, c["z"][:, :24].contiguous(), c["idx"], c["gate"], c["u"],
                               c["cent"][:24].contiguous())


# ------------------------------------------------------- used together -----
def test_layer_with_router_gradient(cuda_dev):
    """MoELayer(router_grad=True): the forward's output and the experts'
    gradients are those of a layer without it; the gates' gradient comes from
    the checkpoint of the very expert outputs; du gains the router's share."""
    cfg = configs.TINY.with_(name="router_grad", T=200, d=512, E=16, G=4, M=2, K=4, I=256)
    w = make_fp8_weights(cfg, cuda_dev)
    cent, bias = inputs.draw_centroids(cfg, cuda_dev), inputs.draw_bias(cfg, cuda_dev)
    S = 40
    plain = MoELayer(cfg, cent, bias.clone(), *w)
    layer = MoELayer(cfg, cent, bias.clone(), *w, balance_loss=True, seq_len=S, router_grad=True)
    u = inputs.draw_u(cfg, cuda_dev)
    dout = torch.randn(cfg.T, cfg.d, generator=torch.Generator().manual_seed(3)).to(cuda_dev) * 0.01
    dbal = torch.linspace(0.5, 1.5, cfg.T // S, device=cuda_dev)
    out0 = plain.forward_train(u, update_bias=False).clone()
    out1 = layer.forward_train(u, update_bias=False)
    assert torch.equal(out0, out1)
    r0, r1 = plain.backward(dout), layer.backward(dout, dbalance=dbal)
    layer.check()
    for k in ("dyq", "dys", "dy", "dx", "dW1", "dW2"):
        assert torch.equal(r0[k], r1[k]), k
    P = cfg.T * cfg.K
    y = layer.Yq.view(torch.float8_e4m3fn).double().view(P, -1, 128) * layer.Ys.double()[..., None]
    y = y.view(P, -1)[layer.perm["dst_of"].long()]
    prod = dout.double()[:, None] * y
    bound = (cfg.d + 8) * 2.0 ** -24 * prod.abs().sum(2)
    assert bool(((r1["dgate"].double() - prod.sum(2)).abs() <= bound).all())
    # within the checkpoint's rounding of the exact rows: 2^-4 of a value at most
    exact = layer.Y[:P].double()[layer.perm["dst_of"].long()]
    off = (dout.double()[:, None].abs() * torch.maximum(exact.abs() * 2.0 ** -4, layer.Ys.double().repeat_interleave(128, 1)[
        layer.perm["dst_of"].long()] * 2.0 ** -10)).sum(2)
    assert bool(((r1["dgate"].double() - (dout.double()[:, None] * exact).sum(2)).abs() <= off + bound).all())
    c = dict(z=layer.logits, gate=layer.gate, dgate=r1["dgate"], idx=layer.idx, f=layer.balance.f, dloss=dbal,
             u=u, cent=cent, base=r0["du"])
    _check(c, cfg.T // S, (r1["dlogits"], r1["du"], r1["dcentroids"]), alpha=1e-4)
    # no weight gradients wanted: du by the same formula (the gates' sums may
    # run in another order without dy)
    r2 = layer.backward(dout, weight_grads=False, dbalance=dbal)
    assert "dcentroids" not in r2
    assert bool(((r2["dgate"].double() - prod.sum(2)).abs() <= bound).all())
    _check(dict(c, dgate=r2["dgate"]), cfg.T // S, (r2["dlogits"], r2["du"], None), alpha=1e-4)
    with pytest.raises(_abi.MoEError):
        plain.backward(dout, dbalance=dbal)


def test_own_experts_between_sort_and_unsort(cuda_dev):
    """Route, sort, a caller's own bf16 experts, unsort, and the whole
    backward, against autograd in 64 bits on the same selection.  The experts
    here scale their rows channel by channel, so every value passes a handful
    of bf16 roundings: sorted rows exact, expert output, its gradient dy, and
    the sorted rows' gradient, 2^-8 each, over sums of a few terms."""
    T, d, E, K = 120, 256, 16, 4
    g = torch.Generator().manual_seed(7)
    u = torch.randn(T, d, generator=g).bfloat16().to(cuda_dev)
    cent = (torch.randn(E, d, generator=g) / 16).bfloat16().to(cuda_dev)
    scale = (torch.rand(E, d, generator=g) + 0.5).bfloat16().to(cuda_dev)
    dout = torch.randn(T, d, generator=g).bfloat16().to(cuda_dev)
    z = torch.empty(T, E, device=cuda_dev)
    idx, gate = moe.moe_route(u, cent, torch.zeros(E, device=cuda_dev), 1, 1, K, logits_out=z)
    p = moe.moe_permute_index(idx, E, with_shared=False)
    dst = p["dst_of"]
    xs = moe.moe_sort_rows(u, dst)
    expert = torch.repeat_interleave(torch.arange(E, device=cuda_dev), p["counts"].long())
    y = xs * scale[expert]
    out = moe.moe_unsort_rows(y, dst, gate)
    dy, dgate = moe.moe_unsort_rows_backward(dout, y, dst, gate)
    dx = moe.moe_sort_rows_backward(dy * scale[expert], dst)
    dl, du, dc = moe.moe_route_backward(dgate, z, idx, gate, u, cent, du_base=dx.float())

    u64 = u.double().requires_grad_()
    c64 = cent.double().requires_grad_()
    s = torch.sigmoid(u64 @ c64.T).gather(1, idx.long())
    g64 = s / s.sum(1, keepdim=True)
    out64 = (g64[..., None] * scale.double()[idx.long()] * u64[:, None]).sum(1)
    out64.backward(dout.double())
    for got, ref, what in ((out, out64.detach(), "out"), (du, u64.grad, "du"), (dc, c64.grad, "dcentroids")):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel < 4 * 2.0 ** -8, (what, rel)
