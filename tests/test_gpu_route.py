"""The router and its gradient (bsq_route, bsq_route_backward) against their definition in 64 bits.

Choice.  The score is a float32 sum at most, so the ids have one value each: they are compared
exactly, with ties (BF16 logits of few values) to the lowest index.

Tolerance.  u = 2^-24.  A weight is e / sum e with e = exp(l - m): the difference l - m is rounded
once (an error of R u in the exponent, R = max |l - m|), expf is off by at most 2 ulp (4 u), the sum of E terms over
V = E / 32 per lane and five exchanges adds (V + 5) u, its terms' own R u + 4 u, the
division and the factor 2 u: rel = (2 R + V + 15) u, sigmoid likewise with R = max |l| (1 + e rounded: u).
A gradient p (g - sum g p) is two such p's, a sum over k <= 32 (10 u) and three
operations: |err| <= 2 rel + 16 u relative to p (|g| + sum |g| p), plus half a step of the
output's type (BF16: 2^-8 of the value).
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def draw(T, E, dtype, seed, coarse=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, E), generator=g) * 2
    if coarse:
        x = (x * 2).round() / 2          # many ties
    return x.to(dtype)


def choose(score, k):
    """int [T, k] of float32 scores, by falling score, ties to the lowest index; -1 where there is none."""
    T, E = score.shape
    ids = np.full((T, k), -1, np.int32)
    for t in range(T):
        s = score[t]
        able = [e for e in range(E) if s[e] > -np.inf]
        able.sort(key=lambda e: (-s[e], e))
        ids[t, :min(k, len(able))] = able[:k]
    return ids


def scores(x, gate, bias):
    x = x.float().numpy()
    if bias is None:
        return x
    with np.errstate(invalid="ignore", over="ignore"):
        return (1 / (1 + np.exp(-x.astype(np.float64))) if gate == "sigmoid" else x.astype(np.float64)) .astype(np.float32) + bias.numpy()


def parts(x, ids, gate, renorm):
    """(p over all experts or the chosen, zero elsewhere; sigmoid sums) in float64, [T, E]."""
    x = x.double().numpy()
    mask = np.zeros(x.shape, bool)
    for t, row in enumerate(ids):
        mask[t, row[row >= 0]] = True
    if gate == "softmax":
        over = np.where(mask, x, -np.inf) if renorm else x
        m = over.max(axis=1, keepdims=True)
        e = np.exp(over - np.where(np.isfinite(m), m, 0))
        s = e.sum(axis=1, keepdims=True)
        return e / np.where(s > 0, s, 1), mask
    s = np.where(mask, 1 / (1 + np.exp(-x)), 0)
    return (s / np.where(s.sum(axis=1, keepdims=True) > 0, s.sum(axis=1, keepdims=True), 1) if renorm else s), mask


def reference(x, ids, gate, renorm, factor, grad=None):
    """(weights [T, k], grad_logits [T, E], its scale [T, E]) in float64."""
    p, mask = parts(x, ids, gate, renorm)
    pick = np.take_along_axis(p, np.maximum(ids, 0), axis=1) * (ids >= 0)
    if grad is None:
        return factor * pick, None, None
    g = np.zeros(p.shape)
    for t, row in enumerate(ids):
        for j, e in enumerate(row):
            if e >= 0:
                g[t, e] += factor * float(grad[t, j])
    mean, size = (p * g).sum(axis=1, keepdims=True), (p * abs(g)).sum(axis=1, keepdims=True)
    if gate == "softmax":
        some = mask.any(axis=1, keepdims=True)
        return factor * pick, p * (g - mean) * some, p * (abs(g) + size) * some
    s = 1 / (1 + np.exp(-x.double().numpy()))
    if renorm:
        return factor * pick, p * (1 - s) * (g - mean), p * (abs(g) + size)
    return factor * pick, g * s * (1 - s), abs(g)


def rel_of(x, E):
    f = x.double()
    f = f[torch.isfinite(f)]
    span = float(f.max() - f.min()) if f.numel() else 0.0
    return (2 * max(span, float(f.abs().max()) if f.numel() else 0.0) + -(-E // 32) + 15) * U


def check(x, k, gate, renorm, bias=None, factor=1.0, seed=0):
    T, E = x.shape
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    ids, w = bsq.route(d(x), k, gate=gate, renormalize=renorm, bias=d(bias), factor=factor)
    grad = torch.randn((T, k), generator=torch.Generator().manual_seed(seed + 1))
    gl = bsq.route_backward(d(x), ids, d(grad), gate=gate, renormalize=renorm, factor=factor)
    torch.cuda.synchronize()
    want = choose(scores(x, gate, bias), k)
    assert np.array_equal(ids.cpu().numpy(), want)
    ref, g_ref, g_size = reference(x, want, gate, renorm, factor, grad.numpy())
    rel = rel_of(x, E)
    assert w.dtype == F32 and gl.dtype == x.dtype and gl.shape == x.shape
    err = np.abs(w.cpu().double().numpy() - ref)
    assert (err <= rel * np.abs(ref) + 1e-38).all(), (err / np.maximum(np.abs(ref), 1e-30)).max() / rel
    half = 2.0 ** -8 if x.dtype == BF16 else U
    bound = (2 * rel + 16 * U) * g_size + half * np.abs(g_ref) + 1e-38
    err = np.abs(gl.cpu().double().numpy() - g_ref)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 33, 3), (37, 8, 8), (130, 128, 6), (3, 1000, 32), (9, 1024, 2), (65, 257, 4)])
def test_route_and_gradient(gate, renorm, dtype, T, E, k):
    check(draw(T, E, dtype, T + E, coarse=dtype == BF16), k, gate, renorm, factor=2.5, seed=E)


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_a_bias_does_not_unmask(gate):
    x = torch.linspace(-1, 1, 40).repeat(3, 1)
    x[0, 3:] = -float("inf")                # three experts left of five slots
    x[1] = -float("inf")
    x[2, :34] = -float("inf")
    bias = torch.full((40,), 9.0)
    bias[[0, 1, 2, 34, 35, 36, 37, 38, 39]] = -9.0
    ids, w = bsq.route(x.cuda(), 5, gate=gate, bias=bias.cuda())
    assert ids.cpu().tolist() == [[2, 1, 0, -1, -1], [-1] * 5, [39, 38, 37, 36, 35]]
    w = w.cpu()
    assert not w[0, 3:].any() and not w[1].any() and (w[2] > 0).all() and (w[0, :3] > 0).all()


@pytest.mark.parametrize("renorm", [False, True])
def test_bias_takes_part_in_the_choice_alone(renorm):
    x, bias = draw(64, 96, F32, 3), torch.randn(96, generator=torch.Generator().manual_seed(4))
    check(x, 5, "softmax", renorm, bias=bias, factor=-1.5)
    # sigmoids are computed: a bias far from any near tie
    far = torch.arange(96, dtype=F32).flip(0)
    ids, w = bsq.route(x.cuda(), 5, gate="sigmoid", renormalize=renorm, bias=far.cuda())
    assert np.array_equal(ids.cpu().numpy(), np.tile(np.arange(5, dtype=np.int32), (64, 1)))
    ref = reference(x, ids.cpu().numpy(), "sigmoid", renorm, 1.0)[0]
    assert (np.abs(w.cpu().double().numpy() - ref) <= rel_of(x, 96) * ref).all()


def test_masked_rows_and_experts():
    x = draw(6, 40, F32, 5)
    x[0] = -float("inf")                    # a padding row
    x[1, 2:] = -float("inf")                # two experts left of four slots
    x[2, ::2] = -float("inf")
    x[3] = torch.finfo(F32).min             # a mask of the type's lowest value is a tie of all
    x[4, 7] = torch.finfo(F32).min
    for gate in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = bsq.route(x.cuda(), 4, gate=gate, renormalize=renorm)
            gl = bsq.route_backward(x.cuda(), ids, torch.ones((6, 4), device="cuda"), gate=gate, renormalize=renorm)
            ids, w, gl = ids.cpu(), w.cpu(), gl.cpu()
            assert ids[0].tolist() == [-1] * 4 and w[0].tolist() == [0] * 4 and not gl[0].any()
            assert sorted(ids[1, :2].tolist()) == [0, 1] and ids[1, 2:].tolist() == [-1, -1] and w[1, 2:].tolist() == [0, 0]
            assert (ids[2] % 2 == 1).all() and ids[3].tolist() == [0, 1, 2, 3]
            assert torch.isfinite(w).all() and torch.isfinite(gl).all()
            if gate == "softmax":
                assert torch.allclose(w[3], torch.full((4,), 0.25 if renorm else 1 / 40), rtol=40 * U)
            else:
                assert not w[3].any() and not gl[3].any()      # sigmoids of zero
            assert (gl[1, 2:] == 0).all()


def test_nan_and_infinity():
    x = draw(5, 33, F32, 6)
    x[0, 3] = float("nan")
    x[1] = float("nan")
    x[2, 32] = float("inf")
    ids, w = (t.cpu() for t in bsq.route(x.cuda(), 3))
    assert 3 not in ids[0].tolist() and w[0].isnan().all()
    assert ids[1].tolist() == [-1, -1, -1] and w[1].tolist() == [0, 0, 0]
    assert ids[2, 0] == 32 and w[2].isnan().all()
    assert torch.isfinite(w[3:]).all()
    ids, w = (t.cpu() for t in bsq.route(x.cuda(), 3, gate="sigmoid", renormalize=False))
    assert ids[2, 0] == 32 and w[2, 0] == 1 and torch.isfinite(w[2]).all() and w[0].isnan().all()


def test_zeros_of_both_signs_are_equal():
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -1.0]])
    assert bsq.route(x.cuda(), 4)[0].cpu().tolist() == [[0, 1, 2, 3]]


def test_ids_of_the_caller():
    """Outside 0..E-1: nothing; the same one twice counts twice."""
    x, g = draw(3, 20, F32, 7), torch.randn((3, 4), generator=torch.Generator().manual_seed(8))
    for gate, renorm in (("softmax", False), ("sigmoid", False)):
        got = bsq.route_backward(x.cuda(), torch.tensor([[4, 4, -1, 20], [-5, 99, 2, 1], [-1, -1, -1, -1]], dtype=torch.int32, device="cuda"),
                                 g.cuda(), gate=gate, renormalize=renorm).cpu()
        once = torch.stack([torch.tensor([g[0, 0] + g[0, 1], 0]), torch.tensor([g[1, 2], g[1, 3]]), torch.zeros(2)])
        ref = bsq.route_backward(x.cuda(), torch.tensor([[4, -1], [2, 1], [-1, -1]], dtype=torch.int32, device="cuda"), once.cuda(),
                                 gate=gate, renormalize=renorm).cpu()
        assert torch.allclose(got, ref, rtol=1e-5, atol=1e-7) and not got[2].any()


@pytest.mark.parametrize("gate,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_gradient_against_differences(gate, renorm):
    """Central differences of the 64-bit weights with the choice held: truncation h^2 / 6 |f'''| <= 1e-8 |grad|, rounding
    2^-53 / h = 1.1e-12; the gradient's own float32 error is at most 1e-5 of the row's largest."""
    x, k, h = draw(4, 24, F32, 9), 3, 1e-4
    g = torch.randn((4, k), generator=torch.Generator().manual_seed(10))
    ids, _ = bsq.route(x.cuda(), k, gate=gate, renormalize=renorm, factor=1.7)
    got = bsq.route_backward(x.cuda(), ids, g.cuda(), gate=gate, renormalize=renorm, factor=1.7).cpu().double().numpy()
    ids, xd = ids.cpu().numpy(), x.double()
    f = lambda z: (reference(z, ids, gate, renorm, 1.7)[0] * g.double().numpy()).sum(axis=1)  # noqa: E731
    for e in range(24):
        d = torch.zeros_like(xd)
        d[:, e] = h
        num = (f(xd + d) - f(xd - d)) / (2 * h)
        assert (np.abs(num - got[:, e]) <= 1e-5 * np.abs(got).max(axis=1) + 1e-7).all()


def test_no_tokens_and_given_outputs():
    ids, w = bsq.route(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == w.shape == (0, 2)
    assert bsq.route_backward(torch.zeros((0, 8), device="cuda"), ids, w).shape == (0, 8)
    x = draw(7, 16, BF16, 11).cuda()
    mine = torch.full((9, 2), 77, dtype=torch.int32, device="cuda")
    ids, w = bsq.route(x, 2, ids=mine[1:8])
    assert ids.data_ptr() == mine[1:8].data_ptr() and mine[0].tolist() == mine[8].tolist() == [77, 77]
    assert torch.equal(ids, bsq.route(x, 2)[0])


def test_factor_zero_passes_nothing():
    x = draw(3, 16, F32, 12).cuda()
    ids, w = bsq.route(x, 4, factor=0.0)
    assert (ids >= 0).all() and not w.any()
    assert not bsq.route_backward(x, ids, torch.ones((3, 4), device="cuda"), factor=0.0).any()
