"""GPU parity of the 16/32-bit sort and unsort of tokens by expert, and of
their gradients, against plain 64-bit sums.

"DeepSeek_V3_Report：Annotation", eq. (12).  Tolerances: a result of type t is
rounded once (eps(t)/2 of its value, or half its smallest subnormal); the
fp32 sum before it has one rounding of 2^-24 per term, bounded by the sum of
the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import _abi
import fp8_block_scaled_sigmoid_b200 as moe

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def _table(T, K, drop, seed, extra=0):
    """A table of distinct rows in random order with dropped pairs (-1); some
    tokens lose all of theirs.  Returns (dst_of, rows)."""
    rng = np.random.default_rng(seed)
    keep = rng.random((T, K)) >= drop
    if drop and T > 2:
        keep[T // 2] = False
    n = int(keep.sum())
    rows = n + extra
    dst = np.full((T, K), -1, np.int32)
    dst[keep] = rng.permutation(rows)[:n]
    return torch.from_numpy(dst), rows


def _mat(n, d, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, d + pad, generator=g).to(dtype)[:, :d]


def _cuda(t, dev):
    """The same values with the same strides on the device."""
    base = torch.empty(t.shape[0], t.stride(0) if t.shape[0] > 1 else t.shape[1], dtype=t.dtype, device=dev)
    out = base[:, :t.shape[1]]
    out.copy_(t)
    return out


def _near(got, ref, terms, n_terms, what):
    """|got - ref| <= half a step of got's type + n_terms fp32 roundings of the terms' magnitudes."""
    fi = torch.finfo(got.dtype)
    bound = fi.eps / 2 * ref.abs() + (n_terms + 1) * 2.0 ** -24 * terms * (1 + fi.eps) + fi.smallest_normal * fi.eps
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= bound).all()), (what, float((err - bound).max()))


CASES = [
    # T, K, d, dtype, drop, pad, extra rows
    (1, 8, 7168, BF, 0.0, 0, 0),
    (1, 1, 1, F32, 0.0, 0, 0),
    (3, 2, 5, HF, 0.0, 0, 4),
    (37, 6, 1111, HF, 0.2, 9, 3),
    (37, 6, 1111, BF, 0.2, 0, 3),
    (64, 4, 257, F32, 0.3, 0, 1),
    (130, 8, 2048, BF, 0.0, 8, 0),
    (200, 3, 4104, BF, 0.1, 4, 0),
    (129, 32, 96, F32, 0.5, 0, 7),
    (500, 8, 7168, HF, 0.0, 0, 0),
    (70, 2, 9000, F32, 0.1, 0, 0),
    (33, 12, 20000, BF, 0.0, 0, 0),
]


@pytest.mark.parametrize("T,K,d,dtype,drop,pad,extra", CASES)
def test_sort_and_its_gradient(cuda_dev, T, K, d, dtype, drop, pad, extra):
    dst, rows = _table(T, K, drop, 1 + T, extra)
    x = _mat(T, d, dtype, 2 + T, pad)
    dd = dst.to(cuda_dev)
    out = torch.full((rows, d), 7.0, dtype=dtype, device=cuda_dev)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
    xs = moe.moe_sort_rows(_cuda(x, cuda_dev), dd, rows, out=out, dev_err=err)
    ref = torch.full((rows, d), 7.0, dtype=dtype)
    t, k = torch.nonzero(dst >= 0, as_tuple=True)
    ref[dst[t, k].long()] = x[t]
    assert torch.equal(xs.cpu(), ref)        # rows that no pair points at stay as they were

    dxs = _mat(rows, d, dtype, 3 + T, pad)
    unused = torch.ones(rows, dtype=torch.bool)
    unused[dst[t, k].long()] = False
    dxs[unused] = float("nan")               # never read
    dx = moe.moe_sort_rows_backward(_cuda(dxs, cuda_dev), dd, dev_err=err)
    rows64 = torch.where((dst >= 0)[..., None], dxs.double()[dst.clamp_min(0).long()], 0.0)
    _near(dx, rows64.sum(1), rows64.abs().sum(1), K, "dx")
    assert int(err.item()) == 0


@pytest.mark.parametrize("T,K,d,dtype,drop,pad,extra", CASES)
def test_unsort_and_its_gradients(cuda_dev, T, K, d, dtype, drop, pad, extra):
    dst, rows = _table(T, K, drop, 11 + T, extra)
    g = torch.Generator().manual_seed(5)
    w = torch.rand(T, K, generator=g)
    w /= w.sum(1, keepdim=True)
    y = _mat(rows, d, dtype, 12 + T, pad)
    t, k = torch.nonzero(dst >= 0, as_tuple=True)
    r = dst[t, k].long()
    unused = torch.ones(rows, dtype=torch.bool)
    unused[r] = False
    y[unused] = float("inf")
    w_in = w.clone()
    w_in[dst < 0] = float("nan")             # a dropped pair's weight is not used
    dd, wd, yd = dst.to(cuda_dev), w_in.to(cuda_dev), _cuda(y, cuda_dev)
    out = moe.moe_unsort_rows(yd, dd, wd)
    terms = torch.where((dst >= 0)[..., None], y.double()[dst.clamp_min(0).long()], 0.0) * w.double()[..., None]
    _near(out, terms.sum(1), terms.abs().sum(1), K, "out")

    dout = _mat(T, d, dtype, 13 + T, pad)
    dy0 = torch.full((rows, d), 3.0, dtype=dtype, device=cuda_dev)
    dy, dw = moe.moe_unsort_rows_backward(_cuda(dout, cuda_dev), yd, dd, wd, dy=dy0)
    ref = torch.full((rows, d), 3.0, dtype=dtype)
    ref[r] = (w[t, k][:, None] * dout[t].float()).to(dtype)   # one fp32 product, one rounding
    assert torch.equal(dy.cpu(), ref)
    prod = dout.double()[t] * y.double()[r]
    dwr, dwm = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    dwr[t, k], dwm[t, k] = prod.sum(1), prod.abs().sum(1)
    _near(dw, dwr, dwm, d, "dweight")
    assert not dw.cpu()[dst < 0].any()
    # each alone gives the same bits
    _, dw2 = moe.moe_unsort_rows_backward(_cuda(dout, cuda_dev), yd, dd, wd, want_dy=False)
    dy3, none = moe.moe_unsort_rows_backward(_cuda(dout, cuda_dev), yd, dd, wd, want_dweight=False)
    assert torch.equal(dw, dw2) and none is None and torch.equal(dy3.cpu()[r], ref[r])


def test_weight_gradient_against_differences(cuda_dev):
    """sum(out * dout) is linear in the weights: one central difference in a
    weight, from fp32 outputs, is its gradient up to the outputs' rounding."""
    T, K, d = 9, 4, 640
    dst, rows = _table(T, K, 0.1, 21)
    y, dout = _mat(rows, d, F32, 22).to(cuda_dev), _mat(T, d, F32, 23).to(cuda_dev)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(24)).to(cuda_dev)
    dd = dst.to(cuda_dev)
    _, dw = moe.moe_unsort_rows_backward(dout, y, dd, w)
    h = 0.5                                   # linear: any step is exact but for rounding
    for t, k in [(0, 0), (4, 3), (8, 1)]:
        wp, wm = w.clone(), w.clone()
        wp[t, k] += h
        wm[t, k] -= h
        span = (wp[t, k] - wm[t, k]).double()
        fp, fm = moe.moe_unsort_rows(y, dd, wp).double(), moe.moe_unsort_rows(y, dd, wm).double()
        diff = ((fp - fm) * dout.double()).sum() / span
        # each out value is off by at most (K + 1) 2^-24 of its terms, both sides
        mag = (fp.abs() + fm.abs())[t] @ dout.double().abs()[t] + 1.0
        assert abs(float(diff - dw[t, k])) <= float((K + 1) * 4 * 2.0 ** -24 * mag / span) + d * 2.0 ** -24 * float(
            (dout.double()[t].abs() * y.double()[dst[t, k].clamp_min(0)].abs()).sum())


def test_empty_batches_and_no_pairs(cuda_dev):
    z = torch.empty(0, 4, dtype=torch.int32, device=cuda_dev)
    x = torch.empty(0, 64, dtype=BF, device=cuda_dev)
    assert moe.moe_sort_rows(x, z).shape == (0, 64)
    assert moe.moe_sort_rows_backward(x, z).shape == (0, 64)
    # every pair dropped: zero rows come back, nothing is written
    none = torch.full((5, 3), -1, dtype=torch.int32, device=cuda_dev)
    y = torch.full((4, 64), float("nan"), dtype=BF, device=cuda_dev)
    w = torch.ones(5, 3, device=cuda_dev)
    assert not moe.moe_unsort_rows(y, none, w).any()
    assert not moe.moe_sort_rows_backward(y, none).any()
    tok = torch.ones(5, 64, dtype=BF, device=cuda_dev)
    dy = torch.full((4, 64), 2.0, dtype=BF, device=cuda_dev)
    _, dw = moe.moe_unsort_rows_backward(tok, y, none, w, dy=dy)
    assert not dw.any() and bool((dy == 2.0).all())
    # K = 0
    k0 = torch.empty(5, 0, dtype=torch.int32, device=cuda_dev)
    assert not moe.moe_sort_rows_backward(y, k0).any()


def test_bad_rows_are_reported_and_skipped(cuda_dev):
    """An entry past the sorted rows records the error and counts as dropped
    (the kernels check every row before using it)."""
    T, K, d, rows = 6, 2, 72, 9
    dst, _ = _table(T, K, 0.0, 31)
    dd = dst.to(cuda_dev)                     # rows 0..11, of which 9..11 are past the end
    ok = dst < rows
    x = _mat(T, d, F32, 32).to(cuda_dev)
    for call in (lambda e: moe.moe_sort_rows(x, dd, rows, dev_err=e),
                 lambda e: moe.moe_sort_rows_backward(xs, dd, dev_err=e),
                 lambda e: moe.moe_unsort_rows(xs, dd, torch.ones(T, K, device=cuda_dev), dev_err=e),
                 lambda e: moe.moe_unsort_rows_backward(x, xs, dd, torch.ones(T, K, device=cuda_dev),
                                                        dev_err=e)[1]):
        err = torch.zeros(1, dtype=torch.int32, device=cuda_dev)
        got = call(err)
        assert int(err.item()) == 3
        if got.shape[0] == rows:
            xs = got
            t, k = torch.nonzero(ok, as_tuple=True)
            assert torch.equal(xs[dd[t, k].long()], x[t])
    assert not got.cpu()[~ok].any()


def test_rows_past_two_billion_elements(cuda_dev):
    """Sorted rows whose element offset passes 32 bits."""
    d, rows = 7168, 300_001                   # 2.15e9 elements, 4.3 GB
    xs = torch.empty(rows, d, dtype=BF, device=cuda_dev)
    x = _mat(2, d, BF, 41).to(cuda_dev)
    dd = torch.tensor([[rows - 1, 0], [rows - 2, 1]], dtype=torch.int32, device=cuda_dev)
    moe.moe_sort_rows(x, dd, rows, out=xs)
    assert torch.equal(xs[rows - 1], x[0]) and torch.equal(xs[rows - 2], x[1]) and torch.equal(xs[1], x[1])
    w = torch.tensor([[1.0, 2.0], [0.5, 0.25]], device=cuda_dev)
    out = moe.moe_unsort_rows(xs, dd, w)
    assert torch.equal(out, torch.stack([3.0 * x[0].float(), 0.75 * x[1].float()]).to(BF))
    _, dw = moe.moe_unsort_rows_backward(x, xs, dd, w, want_dy=False)
    assert torch.equal(dw[:, 0], dw[:, 1])


def test_graph_replay_and_side_stream(cuda_dev):
    """Captured calls replay on new contents, and a call on another stream
    gives the same bits."""
    T, K, d = 100, 4, 1024
    dst, rows = _table(T, K, 0.1, 51)
    dd = dst.to(cuda_dev)
    x, w = _mat(T, d, BF, 52).to(cuda_dev), torch.rand(T, K, device=cuda_dev)
    xs = torch.zeros(rows, d, dtype=BF, device=cuda_dev)
    out, dy = torch.empty(T, d, dtype=BF, device=cuda_dev), torch.zeros(rows, d, dtype=BF, device=cuda_dev)
    dw = torch.empty(T, K, device=cuda_dev)

    def step():
        moe.moe_sort_rows(x, dd, rows, out=xs)
        moe.moe_unsort_rows(xs, dd, w, out=out)
        moe.moe_unsort_rows_backward(out, xs, dd, w, dy=dy, dweight=dw)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(_mat(T, d, BF, 53))
    graph.replay()
    got = [t.clone() for t in (xs, out, dy, dw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, (xs, out, dy, dw)):
        assert torch.equal(a, b)
    # given as an argument: new outputs belong to that stream
    s.wait_stream(torch.cuda.current_stream())
    out2 = moe.moe_unsort_rows(xs, dd, w, stream=s)
    dy2, dw2 = moe.moe_unsort_rows_backward(out2, xs, dd, w, stream=s)
    xs2 = moe.moe_sort_rows(x, dd, rows, stream=s)
    dx2 = moe.moe_sort_rows_backward(xs2, dd, stream=s)
    s.synchronize()
    used = dd[dd >= 0].long()
    assert torch.equal(out2, out) and torch.equal(dy2[used], dy[used]) and torch.equal(dw2, dw)
    assert torch.equal(xs2[used], xs[used]) and dx2.shape == (T, d)
    del graph


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("d,ld,shift", [(64, 64, 1), (130, 131, 3), (96, 104, 4), (1024, 1032, 0), (7, 9, 2)])
def test_rows_at_any_element_offset(cuda_dev, dtype, d, ld, shift):
    """Views whose rows start at any element, and outputs that are such views:
    the columns between rows stay as they were."""
    T, K = 33, 3
    dst, rows = _table(T, K, 0.2, 61)
    dd = dst.to(cuda_dev)

    def view(n, seed=None):
        flat = torch.full((n * ld + 16,), 9.0, dtype=dtype, device=cuda_dev)
        v = flat[shift:shift + n * ld].view(n, ld)[:, :d]
        if seed is not None:
            v.copy_(_mat(n, d, dtype, seed))
        return flat, v

    _, x = view(T, 62)
    flat, xs = view(rows)
    moe.moe_sort_rows(x, dd, rows, out=xs)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(63)).to(cuda_dev)
    fo, out = view(T)
    moe.moe_unsort_rows(xs, dd, w, out=out)
    fd, dy = view(rows)
    _, dw = moe.moe_unsort_rows_backward(x, xs, dd, w, dy=dy)
    fx, dx = view(T)
    moe.moe_sort_rows_backward(xs, dd, dx=dx)
    cx, cxs = x.clone(), xs.clone()
    used = dd[dd >= 0].long()
    assert torch.equal(cxs[used], moe.moe_sort_rows(cx, dd, rows)[used])
    assert torch.equal(out, moe.moe_unsort_rows(cxs, dd, w))
    dy2, dw2 = moe.moe_unsort_rows_backward(cx, cxs, dd, w)
    assert torch.equal(dy[used], dy2[used])
    assert torch.equal(dx, moe.moe_sort_rows_backward(cxs, dd))
    # two access widths sum a dot product in two orders: d roundings of its terms each
    t, k = torch.nonzero(dst >= 0, as_tuple=True)
    mag = torch.zeros(T, K, dtype=torch.float64)
    mag[t, k] = (cx.double().abs().cpu()[t] * cxs.double().abs().cpu()[dst[t, k].long()]).sum(1)
    assert bool(((dw - dw2).double().cpu().abs() <= 2 * d * 2.0 ** -24 * mag).all())
    for f, v, n in ((flat, xs, rows), (fo, out, T), (fd, dy, rows), (fx, dx, T)):
        gap = torch.ones_like(f, dtype=torch.bool)
        gap[shift:shift + n * ld].view(n, ld)[:, :d] = False
        assert bool((f[gap] == 9.0).all())


def test_refusals(cuda_dev):
    E = _abi.MoEError
    dd = torch.zeros(4, 2, dtype=torch.int32, device=cuda_dev)
    x = torch.zeros(4, 64, dtype=BF, device=cuda_dev)
    w = torch.zeros(4, 2, device=cuda_dev)
    bad = [
        lambda: moe.moe_sort_rows(x.double(), dd),                        # type
        lambda: moe.moe_sort_rows(x[:3], dd),                             # tokens
        lambda: moe.moe_sort_rows(x, dd.long()),                          # table type
        lambda: moe.moe_sort_rows(x, dd[:, ::2]),                         # table strides
        lambda: moe.moe_sort_rows(x.t().contiguous().t(), dd),            # columns not contiguous
        lambda: moe.moe_sort_rows(x.cpu(), dd),                           # device
        lambda: moe.moe_sort_rows(x[:1].expand(4, 64), dd),               # rows over one another
        lambda: moe.moe_sort_rows(x, dd, out=torch.zeros(8, 64, device=cuda_dev)),
        lambda: moe.moe_sort_rows(x, torch.zeros(4, 33, dtype=torch.int32, device=cuda_dev)),
        lambda: moe.moe_unsort_rows(x, dd, w.half()),                     # weight type
        lambda: moe.moe_unsort_rows(x, dd, w[:, :1]),                     # weight shape
        lambda: moe.moe_unsort_rows_backward(x, x.half(), dd, w),         # types differ
        lambda: moe.moe_unsort_rows_backward(x, x, dd, w, want_dy=False, want_dweight=False),
    ]
    for call in bad:
        with pytest.raises(E):
            call()
