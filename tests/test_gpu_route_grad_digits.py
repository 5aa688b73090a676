"""GPU check of the digits that the router's gradient keeps of dlogits.

Centroids and tokens with a single power of two in each column make every
element of du and dC one dlogits value, so that nothing but the split into
16-bit terms and the tensor core's additions is left:

  three bf16 terms hold all 24 bits; adding them (smallest first) to an fp32
  accumulator may truncate twice, 2^-23 each:             2^-22 |v|
  two half terms, each within half a step of 2^-10:       2^-22 |v|, with the
  additions 2^-21 |v|; half's smallest step loses at most 2^-39 of the row's
  largest contribution max_e |dz_e| max|C_e|

A lost last term is 2^-17 (bf16) or 2^-11 (half) of a value at most: the test
first makes sure that most values would show it.
"""
import pytest
import torch

import fp8_block_scaled_sigmoid_b200 as moe
from tests.test_gpu_route_grad import _case

pytestmark = pytest.mark.gpu


def _one_per_column(rows, d, step, start, dev):
    """[rows][d] bf16 with +-2^(-2..2) at row (step j + start) % rows of column j; the rows."""
    at = (torch.arange(d) * step + start) % rows
    m = torch.zeros(rows, d)
    m[at, torch.arange(d)] = torch.exp2(torch.arange(d).float() % 5 - 2) * (1 - 2 * (torch.arange(d) % 2)).float()
    return m.bfloat16().to(dev), at.to(dev)


def _lost(v, dtype, terms):
    """What is left of v after some terms of a type."""
    for _ in range(terms):
        v = v - v.to(dtype).float()
    return v.abs()


@pytest.mark.parametrize("T,E,d,n_seq", [(300, 80, 512, 3), (1, 16, 128, 1), (920, 384, 1024, 4), (4096, 144, 512, 4),
                                         (4100, 144, 512, 4), (4100, 384, 512, 4), (8192, 400, 768, 8),
                                         (14600, 144, 256, 4)])
def test_every_digit_of_dlogits_counts(cuda_dev, T, E, d, n_seq):
    c = _case(T, E, d, 4, n_seq, T + E, cuda_dev)
    cent, e_of = _one_per_column(E, d, 7, 3, cuda_dev)
    u, t_of = _one_per_column(T, d, 13, 5, cuda_dev)
    dz, du, dc = moe.moe_route_backward(c["dgate"], c["z"], c["idx"], c["gate"], u, cent, f=c["f"], dloss=c["dloss"],
                                        alpha=0.5, seq_len=T // n_seq)
    half = T > 4096 and (E > 256 or T * E > 1 << 21)   # the operands that du takes
    worth = _lost(dz, torch.float16 if half else torch.bfloat16, 1 if half else 2) > 2.0 ** -21 * dz.abs()
    assert T * E < 100 or float(worth.float().mean()) > 0.5
    assert T * E < 100 or float((_lost(dz, torch.bfloat16, 2) > 2.0 ** -22 * dz.abs()).float().mean()) > 0.5
    cols = torch.arange(d, device=cuda_dev)
    v = dz.double()[:, e_of] * cent.double()[e_of, cols]
    bound = 2.0 ** -22 * v.abs()
    if half:
        top = (dz.double().abs() * cent.double().abs().amax(1)).amax(1, keepdim=True)
        bound = 2.0 ** -21 * v.abs() + 2.0 ** -39 * top
    err = (du.double() - v).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    v = dz.double()[t_of].T * u.double()[t_of, cols]
    err = (dc.double() - v).abs()
    assert bool((err <= 2.0 ** -22 * v.abs()).all()), float((err / v.abs().clamp_min(1e-300)).max())
