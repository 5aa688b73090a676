"""CPU checks of limits that the training operators' entry points have to keep
(these calls never reach a GPU)."""
import ctypes

import pytest
import torch

from fp8_block_scaled_sigmoid_b200 import _abi


def _checkpoint_backward(rows, T=4, K=2):
    return _abi.lib().moe_combine_checkpoint_backward(16, 16, 16, 16, 16, rows, T, K, 128, 16, 16, None, 16, None, None)


@pytest.mark.parametrize("rows", [9, 12, 1 << 30])
def test_a_checkpoint_of_more_rows_than_pairs_is_refused_by_its_backward(rows):
    """The gradient rows of T*K pairs are followed by the shared expert's, so a
    pair at a sorted row behind T*K has no place there: the forward takes such
    tables, and their backward would lose the pair without a sign."""
    assert _checkpoint_backward(rows) == 2
    assert _checkpoint_backward(1 << 31) == 4      # and what was out of range stays so


def test_without_pairs_the_checkpoint_may_have_any_rows():
    assert _checkpoint_backward(9, T=0) == 0


def test_the_python_call_says_what_to_do():
    z = torch.zeros
    T, K, d = 4, 2, 128
    with pytest.raises(_abi.MoEError, match=r"pass the first T\*K rows"):
        _abi.moe_combine_checkpoint_backward(z(T, d), z(T, K, dtype=torch.int32), z(T, K), z(T * K + T, d, dtype=torch.uint8),
                                             z(T * K + T, 1))


def test_launches_of_the_router_gradient():
    L, n = _abi.lib(), ctypes.c_int(-1)
    call = lambda T, d, E, du=1, dc=1: L.moe_route_backward_launches(T, d, E, du, dc, ctypes.byref(n))
    assert call(0, 256, 32) == 0 and n.value == 0
    assert call(40, 256, 32, 0, 0) == 0 and n.value == 1       # dlogits alone
    assert call(4608, 384, 400, 1, 0) == 0 and n.value == 3    # half operands: the centroids' conversion too
    assert call(40, 256, 2048) == 4 and call(40, 250, 32) == 2 and call(-1, 256, 32) == 1
    assert L.moe_route_backward_launches(40, 256, 32, 1, 1, None) == 1


@pytest.mark.parametrize("T,E,half", [(4096, 1024, 0), (4097, 272, 1), (4100, 256, 0), (8192, 256, 0), (8200, 256, 1),
                                      (16384, 128, 0), (14000, 144, 0), (16384, 144, 1)])
def test_where_the_input_gradient_takes_half_operands(T, E, half):
    """Three terms where halves do not pay: their conversion is a kernel more."""
    n = ctypes.c_int(-1)
    assert _abi.lib().moe_route_backward_launches(T, 384, E, 1, 0, ctypes.byref(n)) == 0
    assert n.value == 2 + half
