"""The router's sigmoid gate where it is used and where it is steep: choices by sigmoid + bias of one size, weights and gradients of
logits far from zero, against the definition in 64 bits.

Tolerance.  u = 2^-24, z = 2^-149 (the smallest float32).  With e = exp(-|l|), off by at most 2 ulp (4 u, below 2^-126 2 z), s and
1 - s are r = 1 / (1 + e) and e r: the sum, the reciprocal and the product round once each, so both are off by at most 7 u of
themselves and 3 z.  The score s + bias rounds once more: two scores further apart than 2 (7 u + u max |score|) keep their order.
  weight, not renormalized: the factor's product once more, 8 u.
  gradient factor g s (1 - s): 2 * 7 u and three products: 17 u, 18 u with the terms of second order; each of s, 1 - s and
the products loses 3 z at most where it is that small: 8 z (|g| + 1).
  renormalized q = s / sum: the sum of k positive terms over five exchanges 5 u + 7 u, the quotient u, s itself 7 u: 20 u of q; the
terms' 3 z are 3 z / sum of q each, and 3 z k q / sum by the sum: dq = 3 z (1 + k q) / sum.
  mean = sum g q: |err| <= 26 u sum |g| q + sum |g| dq (the product and five exchanges on top).
  gradient q (g - mean) (1 - s), with m = sum |g| q: q (|g| + m) (20 + 7 + 3 + 1) u + q (26 u m + sum |g| dq) + dq (|g| + m), all
times 1 - s; 58 u q (|g| + m) bounds the first terms; and 8 z (|g| + 1) as above.
The output's type adds half a step: 2^-8 of a BF16 value, and 2^-134 below 2^-126, where BF16 numbers lie 2^-133 apart.
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu

U, Z = 2.0 ** -24, 2.0 ** -149
BF16, F32 = torch.bfloat16, torch.float32


def both(x):
    """(s, 1 - s) of a float64 array, each to its own last bits."""
    e = np.exp(-np.abs(x))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(x >= 0, big, small), np.where(x >= 0, small, big)


def check(x, ids, grad, renorm, factor):
    """The weights and the gradient of logits x [T, E] with the choice ids [T, k] against 64 bits."""
    ids = torch.as_tensor(ids, dtype=torch.int32)
    got = bsq.route_backward(x.cuda(), ids.cuda(), grad.cuda(), gate="sigmoid", renormalize=renorm, factor=factor)
    got = got.cpu().double().numpy()
    at = ids.long().numpy()
    s, rest = both(np.take_along_axis(x.double().numpy(), at, axis=1))
    g = float(np.float32(factor)) * grad.double().numpy()
    k = at.shape[1]
    if renorm:
        total = s.sum(axis=1, keepdims=True)
        q = s / total
        size, mean = (abs(g) * q).sum(axis=1, keepdims=True), (g * q).sum(axis=1, keepdims=True)
        ref = q * (g - mean) * rest
        dq = 3 * Z * (1 + k * q) / total
        bound = rest * (58 * U * q * (abs(g) + size) + q * (abs(g) * dq).sum(axis=1, keepdims=True) + dq * (abs(g) + size))
    else:
        ref = g * s * rest
        bound = 18 * U * abs(ref)
    bound = bound + 8 * Z * (abs(g) + 1) + (np.maximum(2.0 ** -8 * abs(ref), 2.0 ** -134) if x.dtype == BF16 else 0)
    err = np.abs(np.take_along_axis(got, at, axis=1) - ref)
    assert np.isfinite(got).all() and (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()
    other = np.ones(x.shape, bool)
    np.put_along_axis(other, at, False, axis=1)
    assert not got[other].any()


def distinct(T, E, k, seed):
    return torch.rand((T, E), generator=torch.Generator().manual_seed(seed)).argsort(dim=1)[:, :k]

@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("low", [-30.0, -88.0, -90.0, -95.0, -100.0])
def test_weights_of_small_sigmoids(low, renorm):
    """Sigmoids are those of float32 as far as it has numbers, down to a logit of -103."""
    x = low + torch.rand((9, 12), generator=torch.Generator().manual_seed(5))
    ids, w = (t.cpu() for t in bsq.route(x.cuda(), 3, gate="sigmoid", renormalize=renorm))
    s = both(np.take_along_axis(x.double().numpy(), ids.long().numpy(), axis=1))[0]
    total = s.sum(axis=1, keepdims=True) if renorm else np.ones((9, 1))
    bound = (20 if renorm else 8) * U * s / total + 3 * Z * (1 + 3 * s / total * renorm) / total
    assert (np.abs(w.double().numpy() - s / total) <= bound).all()


@pytest.mark.parametrize("factor", [1.0, 1e3])
@pytest.mark.parametrize("low", [-70.0, -80.0, -82.0, -86.0, -87.5, -88.6])
def test_renormalized_gradient_of_small_sigmoids(low, factor):
    """Sums of sigmoids down to 1e-38, large gradients: the quotients are of the size of one."""
    T, E, k = 16, 40, 4
    g = torch.Generator().manual_seed(int(-10 * low))
    x = low + 0.7 * torch.rand((T, E), generator=g)
    ids = distinct(T, E, k, 1)
    x[torch.arange(0, T, 2), ids[::2, 1].long()] = -100.0
    x[3, ids[3, 0]] = 2.0
    check(x, ids, 5 * torch.randn((T, k), generator=g), True, factor)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("low,high", [(8, 12), (12, 20), (20, 60), (60, 88), (88, 104)])
def test_gradient_of_large_logits(low, high, renorm):
    """1 - s far below a step of s."""
    T, E, k = 24, 33, 5
    g = torch.Generator().manual_seed(low)
    for dtype in (F32, BF16):
        x = (low + (high - low) * torch.rand((T, E), generator=g)).to(dtype)
        check(x, distinct(T, E, k, 2), torch.randn((T, k), generator=g), renorm, 2.5)
        check(-x, distinct(T, E, k, 2), torch.randn((T, k), generator=g), renorm, 2.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,k", [(64, 96, 6), (40, 256, 8), (7, 12, 12), (16, 600, 4)])
def test_choice_by_sigmoids_and_biases_of_one_size(dtype, T, E, k):
    g = torch.Generator().manual_seed(E)
    x = (1.5 * torch.randn((T, E), generator=g)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g)
    x[:, 1::4], bias[1::4] = x[:, 0::4], bias[0::4]        # pairs of equal scores
    ids, w = (t.cpu() for t in bsq.route(x.cuda(), k, gate="sigmoid", bias=bias.cuda()))
    s = both(x.double().numpy())[0]
    score = s + bias.double().numpy()
    far = 2 * (7 * U + U * np.abs(score).max())
    assert len(set(np.argsort(-s, axis=1)[:, 0]) & set(np.argsort(-score, axis=1)[:, 0])) < T or T < 8      # the bias changes choices
    for t in range(T):
        row = ids[t].tolist()
        assert len(set(row)) == k
        mine = score[t, row]
        assert (mine[:-1] >= mine[1:] - far).all()
        rest = np.delete(score[t], row)
        assert rest.size == 0 or rest.max() <= mine[-1] + far
        for e in row:
            if e % 4 == 1:                                  # of two equal ones the lower index comes first
                assert row.index(e - 1) == row.index(e) - 1
    v = np.take_along_axis(s, ids.long().numpy(), axis=1)
    assert (np.abs(w.double().numpy() - v / v.sum(axis=1, keepdims=True)) <= 21 * U).all()
