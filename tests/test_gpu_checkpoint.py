"""GPU parity of the combine with an 8-bit checkpoint and of its backward.

"DeepSeek_V3_Report：Annotation", eq. (12), "Low-Precision Activation".  Codes
and scales match the oracle's quantisers bit for bit; the outputs match
moe_combine / moe_combine_backward; the gates' gradient is an fp32 sum whose
bound counts one rounding of 2^-24 per term.
"""
import numpy as np
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import _abi
import fp8_block_scaled_sigmoid_b200 as moe
from oracle import moe_oracle as O
from tests._util import npraw

pytestmark = pytest.mark.gpu


def _rows(n, d, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, scale, (n, d)) * np.exp2(rng.integers(-3, 4, (n, 1)))
    x[rng.random((n, d)) < 0.002] *= 40.0
    if n > 1:
        x[n // 2, :128] = 0.0                 # a tile of zeros: the scale's floor
    return x.astype(np.float32)


def _table(T, K, drop, seed):
    rng = np.random.default_rng(seed)
    keep = rng.random((T, K)) >= drop
    if drop and T > 2:
        keep[T // 2] = False
    n = int(keep.sum())
    dst = np.full((T, K), -1, np.int32)
    dst[keep] = rng.permutation(n)
    gate = rng.uniform(0, 1, (T, K)).astype(np.float32)
    return dst, gate / gate.sum(1, keepdims=True).astype(np.float32), n


CASES = [(1, 8, 7168, 0.0), (1, 1, 128, 0.0), (37, 6, 1152, 0.2), (130, 4, 384, 0.5), (64, 32, 256, 0.1),
         (300, 8, 7168, 0.0), (20, 2, 12800, 0.0)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,K,d,drop", CASES)
def test_forward(cuda_dev, T, K, d, drop, pow2):
    dst, gate, n = _table(T, K, drop, T)
    rows = n + 2                              # two rows that no pair points at
    y = _rows(rows, d, T + 1)
    y[n:] = np.nan
    ysh, u = _rows(T, d, T + 2), torch.randn(T, d, generator=torch.Generator().manual_seed(T)).bfloat16()
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)
    yq = torch.full((rows, d), 9, dtype=torch.uint8, device=cuda_dev)
    ys = torch.full((rows, d // 128), 5.0, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    args = (up(y), up(dst), up(gate), up(ysh), u.to(cuda_dev))
    out, _, _ = moe.moe_combine_checkpoint(*args, yq=yq, ys=ys, pow2=pow2, dev_err=err)
    assert int(err.item()) == 0
    assert torch.equal(out, moe.moe_combine(*args))
    qo, so = (O.quant_1x128_pow2 if pow2 else O.quant_1x128)(y[:n])
    assert np.array_equal(npraw(ys)[:n], so) and np.array_equal(npraw(yq)[:n], qo)
    assert bool((yq[n:] == 9).all()) and bool((ys[n:] == 5.0).all())
    # no shared expert
    out2, _, _ = moe.moe_combine_checkpoint(args[0], args[1], args[2], None, args[4], pow2=pow2)
    assert torch.equal(out2, moe.moe_combine(args[0], args[1], args[2], None, args[4]))


@pytest.mark.parametrize("T,K,d,drop", CASES)
@pytest.mark.parametrize("want_dy", [False, True])
def test_backward(cuda_dev, T, K, d, drop, want_dy):
    dst, gate, n = _table(T, K, drop, T + 5)
    gate[0, 0] = 0.0                          # a gate that underflowed: a row of zeros
    dout = _rows(T, d, T + 6, 0.01)
    y = _rows(n, d, T + 7)
    yq, ys = O.quant_1x128(y)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)
    P = T * K
    kw = dict(dyq=torch.full((P + T, d), 9, dtype=torch.uint8, device=cuda_dev),
              dys=torch.full((P + T, d // 128), 5.0, device=cuda_dev))
    if want_dy:
        kw["dy"] = torch.full((P + T, d), 3.0, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    dyq, dys, dy, dgate = moe.moe_combine_checkpoint_backward(up(dout), up(dst), up(gate), up(yq), up(ys),
                                                              dev_err=err, **kw)
    assert int(err.item()) == 0
    q2, s2, y2 = _abi.moe_combine_backward(
        up(dout), up(dst), up(gate), torch.full_like(dyq, 9), torch.full_like(dys, 5.0),
        torch.full((P + T, d), 3.0, device=cuda_dev))
    assert torch.equal(dyq, q2) and torch.equal(dys, s2)
    assert (dy is None) == (not want_dy) and (dy is None or torch.equal(dy, y2))
    # dgate: d products and sums in fp32, a scale per tile
    t, k = np.nonzero(dst >= 0)
    prod = dout[t].astype(np.float64) * O.dequant_1x128(yq, ys)[dst[t, k]]
    ref, mag = np.zeros((T, K)), np.zeros((T, K))
    ref[t, k], mag[t, k] = prod.sum(1), np.abs(prod).sum(1)
    err = np.abs(npraw(dgate) - ref)
    bound = (d + d / 128 + 2) * 2.0 ** -24 * mag
    assert np.all(err <= bound), float((err - bound).max())
    assert not npraw(dgate)[dst < 0].any()


def test_backward_without_pairs(cuda_dev):
    """Every pair dropped: only the shared expert's rows are written."""
    T, K, d = 5, 3, 256
    dout = torch.randn(T, d, device=cuda_dev)
    dst = torch.full((T, K), -1, dtype=torch.int32, device=cuda_dev)
    yq = torch.zeros(0, d, dtype=torch.uint8, device=cuda_dev)
    ys = torch.zeros(0, d // 128, device=cuda_dev)
    dyq = torch.full((T * K + T, d), 9, dtype=torch.uint8, device=cuda_dev)
    dyq, dys, _, dgate = moe.moe_combine_checkpoint_backward(dout, dst, torch.ones(T, K, device=cuda_dev),
                                                            yq, ys, dyq=dyq)
    qo, so = O.quant_1x128_pow2(npraw(dout))
    assert np.array_equal(npraw(dyq)[T * K:], qo) and np.array_equal(npraw(dys)[T * K:], so)
    assert bool((dyq[:T * K] == 9).all()) and not dgate.any()


def test_infinities_and_nan(cuda_dev):
    """Non-finite values give the same bytes as the framework's quantiser and
    combine backward on the same rows, and stay in their own rows."""
    T, K, d = 6, 2, 384
    y = torch.randn(T * K, d, device=cuda_dev)
    y[1, 5], y[1, 200], y[4, 300], y[6, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
    dst = torch.arange(T * K, dtype=torch.int32, device=cuda_dev).view(T, K)
    g = torch.full((T, K), 0.5, device=cuda_dev)
    u = torch.randn(T, d, device=cuda_dev).bfloat16()
    for pow2 in (False, True):
        out, yq, ys = moe.moe_combine_checkpoint(y, dst, g, None, u, pow2=pow2)
        q, s = _abi.fp8_quant_1x128_f32(y, pow2=pow2)
        assert torch.equal(yq, q) and torch.equal(ys.view(torch.int32), s.view(torch.int32))
        want = moe.moe_combine(y, dst, g, None, u)
        assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
    dout = torch.randn(T, d, device=cuda_dev)
    dout[0, 3], dout[1, 100], dout[1, 101], dout[2, 129] = float("inf"), float("nan"), 0.0, float("-inf")
    dout[3, :128] = 1e-40
    g[4, 0], g[5, 1] = 0.0, 1e-38
    dyq, dys, dy, dgate = moe.moe_combine_checkpoint_backward(dout, dst, g, q, s, want_dy=True)
    q2, s2, y2 = _abi.moe_combine_backward(dout, dst, g, want_dy=True)
    assert torch.equal(dyq, q2) and torch.equal(dys, s2) and torch.equal(torch.nan_to_num(dy), torch.nan_to_num(y2))
    assert bool(torch.isfinite(dgate[4:]).all())


def test_bad_rows_are_reported_and_skipped(cuda_dev):
    T, K, d = 4, 2, 256
    dst = torch.arange(T * K, dtype=torch.int32, device=cuda_dev).view(T, K)
    rows = 6                                  # 6 and 7 are past the end
    y = torch.randn(rows, d, device=cuda_dev)
    u = torch.randn(T, d, device=cuda_dev).bfloat16()
    g = torch.full((T, K), 0.5, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    out, yq, ys = moe.moe_combine_checkpoint(y, dst, g, None, u, dev_err=err)
    assert int(err.item()) == 3 and torch.equal(out[3], u[3].float())
    err.zero_()
    dyq = torch.full((T * K + T, d), 9, dtype=torch.uint8, device=cuda_dev)
    _, _, _, dgate = moe.moe_combine_checkpoint_backward(u.float(), dst, g, yq, ys, dyq=dyq, dev_err=err)
    assert int(err.item()) == 3 and not dgate[3].any() and dgate[:3].all() and bool((dyq[6:8] == 9).all())


def test_gate_gradient_against_differences(cuda_dev):
    """sum(out * dout) is linear in a gate: its difference is dgate of the
    unquantised rows, so it is off by the checkpoint's rounding (2^-4 of a
    value, or half the tile's smallest step, scale * 2^-10) and the fp32
    sums."""
    T, K, d = 5, 4, 512
    dst, gate, n = _table(T, K, 0.0, 3)
    y, dout = _rows(n, d, 4), _rows(T, d, 5)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)
    u = torch.zeros(T, d, dtype=torch.bfloat16, device=cuda_dev)
    _, yq, ys = moe.moe_combine_checkpoint(up(y), up(dst), up(gate), None, u)
    dgate = npraw(moe.moe_combine_checkpoint_backward(up(dout), up(dst), up(gate), yq, ys)[3])
    s = np.repeat(npraw(ys), 128, axis=1).astype(np.float64)
    for t, k in [(0, 0), (2, 3), (4, 1)]:
        gp, gm = gate.copy(), gate.copy()
        gp[t, k] += 1.0
        gm[t, k] -= 1.0
        f = [npraw(moe.moe_combine(up(y), up(dst), up(g), None, u)).astype(np.float64) for g in (gp, gm)]
        diff = ((f[0] - f[1])[t] * dout[t]).sum() / (float(gp[t, k]) - float(gm[t, k]))
        r = dst[t, k]
        a = np.abs(dout[t].astype(np.float64))
        rounding = (a * np.maximum(np.abs(y[r]) * 2.0 ** -4, s[r] * 2.0 ** -10)).sum()
        sums = 2.0 ** -24 * (8 * K * (a * (np.abs(f[0][t]) + np.abs(f[1][t]))).sum() + 2 * d * (a * np.abs(y[r])).sum())
        assert abs(diff - dgate[t, k]) <= rounding + sums


def test_refusals(cuda_dev):
    E = _abi.MoEError
    T, K, d = 4, 2, 256
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=cuda_dev)
    dst, g, u, y = z(T, K, dt=torch.int32), z(T, K), z(T, d, dt=torch.bfloat16), z(8, d)
    yq, ys = z(8, d, dt=torch.uint8), z(8, 2)
    bad = [
        lambda: moe.moe_combine_checkpoint(y[:, :200].contiguous(), dst, g, None, u[:, :200].contiguous()),
        lambda: moe.moe_combine_checkpoint(y[:, :128], dst, g, None, u[:, :128].contiguous()),   # strided
        lambda: moe.moe_combine_checkpoint(y.half(), dst, g, None, u),
        lambda: moe.moe_combine_checkpoint(y, dst, g, None, u.float()),
        lambda: moe.moe_combine_checkpoint(y, dst, g[:3], None, u),
        lambda: moe.moe_combine_checkpoint(y, dst, g, z(3, d), u),
        lambda: moe.moe_combine_checkpoint(y, dst, g, None, u, yq=yq[:4]),
        lambda: moe.moe_combine_checkpoint(y.cpu(), dst, g, None, u),
        lambda: moe.moe_combine_checkpoint_backward(z(T, 200), dst, g, yq, ys),
        lambda: moe.moe_combine_checkpoint_backward(z(T, d), dst, g, yq.float(), ys),
        lambda: moe.moe_combine_checkpoint_backward(z(T, d), dst, g, yq, ys[:, :1]),
        lambda: moe.moe_combine_checkpoint_backward(z(T, d), dst, g, yq, ys, dyq=yq),
        lambda: moe.moe_combine_checkpoint_backward(z(T, d), dst.long(), g, yq, ys),
    ]
    for call in bad:
        with pytest.raises(E):
            call()
