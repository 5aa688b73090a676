"""CPU checks of the training operators' C entry points: bad arguments are
refused on the host before any launch, and empty batches do nothing (these
calls never reach a GPU)."""
import ctypes

import pytest

from fp8_block_scaled_sigmoid_b200 import _abi

F = ctypes.c_float
BF, HF, F32 = 0, 1, 2


def sort(L, x=16, dt=BF, ldx=64, dst=16, T=4, K=2, d=64, xs=16, ldxs=64, rows=8):
    return L.moe_sort_rows(x, dt, ldx, dst, T, K, d, xs, ldxs, rows, None, None)


def sort_bwd(L, g=16, dt=BF, ldg=64, rows=8, dst=16, T=4, K=2, d=64, dx=16, ldx=64):
    return L.moe_sort_rows_backward(g, dt, ldg, rows, dst, T, K, d, dx, ldx, None, None)


def unsort(L, y=16, dt=BF, ldy=64, rows=8, dst=16, w=16, T=4, K=2, d=64, out=16, ldo=64):
    return L.moe_unsort_rows(y, dt, ldy, rows, dst, w, T, K, d, out, ldo, None, None)


def unsort_bwd(L, g=16, dt=BF, ldg=64, y=16, ldy=64, dst=16, w=16, T=4, K=2, d=64, dy=16, lddy=64, rows=8, dw=16):
    return L.moe_unsort_rows_backward(g, dt, ldg, y, ldy, dst, w, T, K, d, dy, lddy, rows, dw, None, None)


def ck(L, Y=16, rows=8, dst=16, g=16, Ysh=None, u=16, T=4, K=2, d=128, out=16, yq=16, ys=16):
    return L.moe_combine_checkpoint(Y, rows, dst, g, Ysh, u, T, K, d, 0, out, yq, ys, None, None)


def ck_bwd(L, dout=16, dst=16, g=16, yq=16, ys=16, rows=8, T=4, K=2, d=128, dyq=16, dys=16, dy=None, dg=16):
    return L.moe_combine_checkpoint_backward(dout, dst, g, yq, ys, rows, T, K, d, dyq, dys, dy, dg, None, None)


def route(L, dg=16, z=16, idx=16, gate=16, u=16, ldu=128, cent=16, T=8, d=128, E=16, K=2, f=None, dl=None, S=0,
          base=None, dz=16, du=16, dc=16, ws=16, nws=1 << 30):
    return L.moe_route_backward(dg, z, idx, gate, u, ldu, cent, T, d, E, K, f, dl, S, F(1e-4), base, dz, du, dc, ws,
                                nws, None, None)


@pytest.mark.parametrize("call,kw,code", [
    (sort, dict(T=-1), 1), (sort, dict(d=0), 1), (sort, dict(rows=-1), 1), (sort, dict(dt=3), 1),
    (sort, dict(x=None), 1), (sort, dict(xs=None), 1), (sort, dict(dst=None), 1),
    (sort, dict(ldx=63), 2), (sort, dict(ldxs=63), 2),
    (sort, dict(x=17), 3), (sort, dict(dt=F32, xs=18), 3), (sort, dict(dst=18), 3),
    (sort, dict(K=33), 4), (sort, dict(d=(1 << 30) + 1, ldx=1 << 31, ldxs=1 << 31), 4), (sort, dict(rows=1 << 31), 4),
    (sort_bwd, dict(K=-1), 1), (sort_bwd, dict(g=None), 1), (sort_bwd, dict(dx=None), 1),
    (sort_bwd, dict(ldg=10), 2), (sort_bwd, dict(ldx=10), 2), (sort_bwd, dict(dx=17), 3), (sort_bwd, dict(K=40), 4),
    (unsort, dict(w=None), 1), (unsort, dict(dt=-1), 1), (unsort, dict(ldo=10), 2), (unsort, dict(w=18), 3),
    (unsort, dict(dt=F32, y=18), 3), (unsort, dict(K=33), 4),
    (unsort_bwd, dict(dy=None, dw=None), 1), (unsort_bwd, dict(y=None), 1), (unsort_bwd, dict(w=None), 1),
    (unsort_bwd, dict(lddy=10), 2), (unsort_bwd, dict(ldy=10), 2), (unsort_bwd, dict(ldg=10), 2),
    (unsort_bwd, dict(dw=18), 3), (unsort_bwd, dict(dy=17), 3), (unsort_bwd, dict(K=33), 4),
    (ck, dict(T=-1), 1), (ck, dict(u=None), 1), (ck, dict(yq=None), 1), (ck, dict(g=None), 1),
    (ck, dict(d=200), 2), (ck, dict(Y=20), 3), (ck, dict(Ysh=20), 3), (ck, dict(ys=18), 3), (ck, dict(K=33), 4),
    (ck, dict(rows=1 << 31), 4),
    (ck_bwd, dict(dout=None), 1), (ck_bwd, dict(dg=None), 1), (ck_bwd, dict(yq=None), 1), (ck_bwd, dict(rows=-1), 1),
    (ck_bwd, dict(d=64), 2), (ck_bwd, dict(dyq=20), 3), (ck_bwd, dict(dy=20), 3), (ck_bwd, dict(K=33), 4),
    (ck_bwd, dict(T=1 << 28, K=8), 4),
    (route, dict(T=-1), 1), (route, dict(K=0), 1), (route, dict(z=None), 1), (route, dict(idx=None), 1),
    (route, dict(cent=None), 1), (route, dict(u=None), 1), (route, dict(f=16, S=0), 1),
    (route, dict(E=24), 2), (route, dict(d=192), 2), (route, dict(K=17), 2), (route, dict(ldu=64), 2),
    (route, dict(f=16, S=3), 2), (route, dict(E=2048), 4), (route, dict(E=64, K=33), 4),
    (route, dict(z=20), 3), (route, dict(ldu=132), 3), (route, dict(du=20), 3), (route, dict(f=20, S=4), 3), (route, dict(dg=18), 3),
    (route, dict(nws=0), 6), (route, dict(ws=None), 6), (route, dict(ws=20), 3),
])
def test_refused_on_the_host(call, kw, code):
    assert call(_abi.lib(), **kw) == code


def test_empty_batches_do_nothing():
    L = _abi.lib()
    assert sort(L, x=None, dst=None, xs=None, T=0, rows=0) == 0
    assert sort(L, dst=None, K=0) == 0
    assert sort_bwd(L, g=None, dst=None, dx=None, T=0, rows=0) == 0
    assert unsort(L, y=None, dst=None, w=None, out=None, T=0, rows=0) == 0
    assert unsort_bwd(L, g=None, y=None, dst=None, w=None, dy=None, dw=None, T=0, rows=0) == 0
    assert ck(L, Y=None, dst=None, g=None, u=None, out=None, yq=None, ys=None, T=0, rows=0) == 0
    assert ck_bwd(L, dout=None, dst=None, g=None, yq=None, ys=None, dyq=None, dys=None, dg=None, T=0, rows=0) == 0
    assert route(L, T=0, dc=None) == 0


def test_workspace_size():
    L = _abi.lib()
    n = ctypes.c_size_t(0)
    assert L.moe_route_backward_workspace_size(4096, 7168, 256, ctypes.byref(n)) == 0 and n.value > 0
    assert L.moe_route_backward_workspace_size(4096, 7168, 250, ctypes.byref(n)) == 2
    assert L.moe_route_backward_workspace_size(4096, 7168, 2048, ctypes.byref(n)) == 4
    assert L.moe_route_backward_workspace_size(-1, 7168, 256, ctypes.byref(n)) == 1
    assert L.moe_route_backward_workspace_size(1, 7168, 256, None) == 1
