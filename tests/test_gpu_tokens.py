"""Tokens to their experts' rows and back (bsq_sort_experts, bsq_dispatch, bsq_combine,
bsq_combine_backward) against plain forms: whole numbers, copies and codes exactly, sums in 64 bits.

Tolerance.  u = 2^-24.  A combined element is a float32 sum of k fused products: at most (k + 1) u of
sum |w y|, and half a BF16 step, 2^-8, of itself.  A weighted row is one float32 product, rounded to
BF16: the same two roundings here, so it is compared exactly.  A gradient of a weight is a sum of N products: a
lane adds ceil(N / 256) * 8 of them at most, then 5 + 8 partial sums: that many + 1 times u of sum |g y|.
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, I32 = torch.bfloat16, torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def draw_ids(T, k, E, seed, bad=0.0):
    g = gen(seed)
    ids = torch.randint(0, E, (T, k), generator=g)
    if bad:
        miss = torch.rand((T, k), generator=g) < bad
        ids = torch.where(miss, torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 4, (T, k), generator=g)], ids)
    return ids.to(I32)


def sorted_plain(ids, E):
    """(offsets, rows, slots) by a stable sort on the host."""
    flat = ids.reshape(-1).numpy().astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    kept = int((key < E).sum())
    rows, slots = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    rows[order[:kept]] = np.arange(kept)
    slots[:kept] = order[:kept]
    return np.cumsum(np.bincount(key, minlength=E + 1)[:E]).astype(np.int32), rows.reshape(ids.shape), slots


# ---------------------------------------------------------------- sort
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (7, 3, 5), (33, 2, 1024), (100, 32, 1000), (1024, 8, 128), (1025, 8, 64),
                                   (5000, 4, 257), (16384, 8, 256), (40001, 8, 1024), (3, 5, 1), (131072, 1, 3), (1366, 6, 64), (2047, 8, 31), (8191, 8, 64), (30000, 8, 1024)])
@pytest.mark.parametrize("bad", [0.0, 0.3])
def test_sort(T, k, E, bad):
    ids = draw_ids(T, k, E, T + E, bad)
    offsets, rows, slots = bsq.sort_experts(ids.cuda(), E)
    want = sorted_plain(ids, E)
    for got, ref in zip((offsets, rows, slots), want):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("ids,E", [(torch.zeros((5000, 4), dtype=I32), 64), (torch.full((300, 3), -1, dtype=I32), 7),
                                   (torch.arange(40000, dtype=I32).view(-1, 1) % 2 * 63, 64), (torch.full((9, 2), 63, dtype=I32), 64)])
def test_sort_of_one_sided_ids(ids, E):
    offsets, rows, slots = bsq.sort_experts(ids.cuda(), E)
    for got, ref in zip((offsets, rows, slots), sorted_plain(ids, E)):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_sort_of_nothing_and_without_slots():
    offsets, rows, slots = bsq.sort_experts(torch.zeros((0, 4), dtype=I32, device="cuda"), 9)
    assert offsets.cpu().tolist() == [0] * 9 and rows.shape == (0, 4) and slots.shape == (0,)
    ids = draw_ids(50, 4, 9, 1).cuda()
    a, b = bsq.sort_experts(ids, 9), bsq.sort_experts(ids, 9, want_slots=False)
    assert b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- dispatch
def tokens(T, K, seed):
    x = torch.randn((T, K), generator=gen(seed)) * torch.exp2(torch.randint(-8, 8, (T, 1), generator=gen(seed + 1)).float())
    return x.to(BF16)


def weights_of(T, k, seed):
    return torch.randn((T, k), generator=gen(seed))     # negative ones too


def expect_rows(x, rows, w, S, fill):
    """BF16 rows of the definition, `fill` where no slot owns one."""
    out = torch.full((S, x.shape[1]), fill, dtype=BF16)
    for t in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            r = int(rows[t, j])
            if 0 <= r < S:
                out[r] = x[t] if w is None else (x[t].float() * w[t, j]).to(BF16)
    return out


CASES = [(1, 8, 1, 1), (3, 128, 2, 4), (5, 144, 3, 2), (17, 264, 4, 8), (9, 520, 32, 16), (2, 7168, 8, 64), (33, 1040, 1, 3), (64, 2064, 5, 7)]


@pytest.mark.parametrize("T,K,k,E", CASES)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("bad", [0.0, 0.4])
def test_dispatch(T, K, k, E, weighted, bad):
    x, ids = tokens(T, K, K), draw_ids(T, k, E, T, bad)
    w = weights_of(T, k, 5) if weighted else None
    S = T * k
    _, rows, _ = bsq.sort_experts(ids.cuda(), E)
    e4m3 = K % 16 == 0
    out = torch.full((S, K), 7.0, dtype=BF16, device="cuda")
    codes = torch.full((S, K), 0x55, dtype=torch.uint8, device="cuda") if e4m3 else None
    scale = torch.full((S, -(-K // 128)), -3.0, device="cuda") if e4m3 else None
    wd = None if w is None else w.cuda()
    bsq.dispatch(x.cuda(), rows, wd, out=out, codes=codes, scale=scale)
    h = rows.cpu()
    assert torch.equal(out.cpu().view(torch.int16), expect_rows(x, h, w, S, 7.0).view(torch.int16))
    if not e4m3:
        return
    qc, qs = (t.cpu() for t in bsq.quantize_e4m3(x.cuda()))
    want_c, want_s = torch.full((S, K), 0x55, dtype=torch.uint8), torch.full((S, -(-K // 128)), -3.0)
    for t in range(T):
        for j in range(k):
            if h[t, j] >= 0:
                want_c[h[t, j]] = qc[t]
                want_s[h[t, j]] = qs[t] if w is None else qs[t] * w[t, j]
    assert torch.equal(codes.cpu(), want_c) and torch.equal(scale.cpu(), want_s)
    # each type alone gives the same
    assert torch.equal(bsq.dispatch(x.cuda(), rows, wd, out=out.clone())[0].view(torch.int16), out.view(torch.int16))
    only = bsq.dispatch(x.cuda(), rows, wd, bf16=False, codes=codes.clone(), scale=scale.clone())
    assert only[0] is None and torch.equal(only[1], codes) and torch.equal(only[2], scale)


def test_dispatched_values_in_64_bits():
    """A row's codes times its scale are w x to half a step of E4M3, 2^-4 of a value in its normal range, else 2^-10 of the scale."""
    T, K, k = 20, 400, 3
    x, w = tokens(T, K, 1), weights_of(T, k, 2)
    _, rows, _ = bsq.sort_experts(draw_ids(T, k, 6, 3).cuda(), 6)
    _, codes, scale = bsq.dispatch(x.cuda(), rows, w.cuda(), bf16=False, e4m3=True)
    v = codes.cpu().view(torch.float8_e4m3fn).double()
    s = scale.cpu().double().repeat_interleave(128, 1)[:, :K]
    for t in range(T):
        for j in range(k):
            r = int(rows[t, j])
            ref = x[t].double() * float(w[t, j])
            assert ((v[r] * s[r] - ref).abs() <= 2.0 ** -4 * ref.abs() * (1 + 2.0 ** -20) + 2.0 ** -10 * s[r].abs()).all()


def test_rows_outside_are_left_out():
    x = tokens(4, 128, 9)
    rows = torch.tensor([[0, 5], [-1, 2], [2 ** 31 - 1, -2 ** 31], [1, 3]], dtype=I32)
    out = torch.full((6, 128), 7.0, dtype=BF16, device="cuda")
    got = bsq.dispatch(x.cuda(), rows.cuda(), out=out[:4])[0].cpu()       # rows 5 and beyond are not of this call
    assert torch.equal(got, expect_rows(x, rows, None, 4, 7.0)) and (out[4:] == 7).all()
    y = bsq.combine(out[:4], rows.cuda()).cpu().double()
    o = out.cpu().double()
    assert torch.equal(y, torch.stack([o[0], o[2], torch.zeros(128).double(), o[1] + o[3]]).to(BF16).double())
    g = bsq.combine_backward(x.cuda(), out[:4], rows.cuda())[3].cpu()
    assert g[0, 1] == 0 and g[1, 0] == 0 and not g[2].any() and g[0, 0] != 0


def test_special_values():
    x = tokens(4, 256, 11)
    x[0, 3], x[1, 200], x[2] = float("nan"), float("inf"), 0.0
    rows = torch.arange(4, dtype=I32).view(4, 1)
    out, codes, scale = (t.cpu() for t in bsq.dispatch(x.cuda(), rows.cuda(), e4m3=True))
    qc, qs = (t.cpu() for t in bsq.quantize_e4m3(x.cuda()))
    assert torch.equal(out.view(torch.int16), x.view(torch.int16))
    assert torch.equal(codes, qc) and torch.equal(scale.view(torch.int32), qs.view(torch.int32))
    assert scale[0, 0].isnan() and torch.isinf(scale[1, 1]) and (scale[2] == 1).all()
    # a weight of zero, and NaN where no row is
    w = torch.tensor([[0.0], [1.0], [float("nan")], [2.0]])
    rows[2] = -1
    y = bsq.combine(x.cuda(), rows.cuda(), w.cuda()).cpu()
    assert y[0, 3].isnan() and y[0, 4] == 0 and torch.isinf(y[1, 200]) and not y[2].any() and torch.equal(y[3], (2 * x[3].float()).to(BF16))


def test_far_rows():
    """Rows whose elements lie beyond 2^31."""
    K, S = 8192, 2 ** 18 + 10
    x, rows = tokens(2, K, 13), torch.tensor([[S - 1, 5], [0, S - 2]], dtype=I32)
    out, codes, scale = bsq.dispatch(x.cuda(), rows.cuda(), S=S, e4m3=True)
    for t in range(2):
        for j in range(2):
            assert torch.equal(out[rows[t, j].item()].cpu(), x[t])
    qc, qs = bsq.quantize_e4m3(x.cuda())
    assert torch.equal(codes[S - 1], qc[0]) and torch.equal(scale[S - 2], qs[1])
    y = bsq.combine(out, rows.cuda()).cpu()
    assert torch.equal(y, (2 * x.float()).to(BF16))
    grad, _, _, gw = bsq.combine_backward(x.cuda(), out, rows.cuda())
    assert torch.equal(grad[S - 1].cpu(), x[0]) and torch.equal(gw[0, 0], gw[0, 1])


# ---------------------------------------------------------------- combine and its gradient
@pytest.mark.parametrize("T,N,k,E", CASES + [(3000, 264, 3, 9), (2500, 648, 2, 5), (2600, 1808, 5, 9), (610, 1040, 4, 8)])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("bad", [0.0, 0.4])
def test_combine_and_gradient(T, N, k, E, weighted, bad):
    S = T * k
    y = torch.randn((S, N), generator=gen(N)).to(BF16)
    w = weights_of(T, k, 5) if weighted else None
    wd = None if w is None else w.cuda()
    _, rows, _ = bsq.sort_experts(draw_ids(T, k, E, T, bad).cuda(), E)
    h = rows.cpu()
    at, have = h.long().clamp(min=0), (h >= 0).double()
    got = bsq.combine(y.cuda(), rows, wd).cpu().double()
    one = have if w is None else have * w.double()
    ref, size = torch.zeros((T, N)).double(), torch.zeros((T, N)).double()
    for j in range(k):
        term = one[:, j, None] * y[at[:, j]].double()
        ref += term
        size += term.abs()
    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (k + 1) * U * size).all()

    g = torch.randn((T, N), generator=gen(N + 1)).to(BF16)
    e4m3 = N % 16 == 0
    gy = torch.full((S, N), 7.0, dtype=BF16, device="cuda")
    codes = torch.full((S, N), 0x55, dtype=torch.uint8, device="cuda") if e4m3 else None
    scale = torch.full((S, -(-N // 128)), -3.0, device="cuda") if e4m3 else None
    _, _, _, gw = bsq.combine_backward(g.cuda(), y.cuda(), rows, wd, grad_y=gy, codes=codes, scale=scale)
    # the rows are those that dispatch writes
    same = bsq.dispatch(g.cuda(), rows, wd, out=torch.full_like(gy, 7.0), e4m3=False,
                        codes=None if codes is None else torch.full_like(codes, 0x55), scale=None if scale is None else torch.full_like(scale, -3.0))
    assert torch.equal(gy.view(torch.int16), same[0].view(torch.int16))
    if e4m3:
        assert torch.equal(codes, same[1]) and torch.equal(scale, same[2])
    steps = -(-N // 256) * 8 + 14
    for j in range(k):
        prod = g.double() * y[at[:, j]].double() * have[:, j, None]
        assert ((gw.cpu().double()[:, j] - prod.sum(1)).abs() <= steps * U * prod.abs().sum(1)).all()
    # what is asked for alone is the same
    assert torch.equal(bsq.combine_backward(g.cuda(), y.cuda(), rows, wd, bf16=False)[3], gw)
    alone = bsq.combine_backward(g.cuda(), None, rows, wd, want_weights=False, grad_y=torch.full_like(gy, 7.0))
    assert alone[3] is None and torch.equal(alone[0].view(torch.int16), gy.view(torch.int16))
    if e4m3:
        part = bsq.combine_backward(g.cuda(), y.cuda(), rows, wd, bf16=False, codes=torch.full_like(codes, 0x55), scale=torch.full_like(scale, -3.0))
        assert torch.equal(part[1], codes) and torch.equal(part[2], scale) and torch.equal(part[3], gw)


def test_combine_of_one_row_by_several_slots():
    y = torch.randn((2, 128), generator=gen(1)).to(BF16)
    rows = torch.tensor([[1, 1, 0], [1, -1, 1]], dtype=I32)
    got = bsq.combine(y.cuda(), rows.cuda()).cpu()
    assert torch.equal(got[1], (2 * y[1].float()).to(BF16))
    ref = 2 * y[1].double() + y[0].double()
    assert ((got[0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 4 * U * (2 * y[1].double().abs() + y[0].double().abs())).all()


def test_gradients_against_differences():
    """f = <g, combine(y, w)> is bilinear: its differences are exact in 64 bits but for rounding (2^-45 here), its gradients off by
    half a BF16 step (rows) and the dot product's float32 rounding (weights, see above)."""
    T, N, k, E = 6, 48, 3, 4
    _, rows, _ = bsq.sort_experts(draw_ids(T, k, E, 3, 0.2).cuda(), E)
    y, g, w = torch.randn((T * k, N), generator=gen(4)).to(BF16), torch.randn((T, N), generator=gen(5)).to(BF16), weights_of(T, k, 6)
    gy = torch.zeros((T * k, N), dtype=BF16, device="cuda")
    gw = bsq.combine_backward(g.cuda(), y.cuda(), rows, w.cuda(), grad_y=gy)[3].cpu().double()
    h, gy = rows.cpu().long(), gy.cpu().double()

    def f(yy, ww):
        have = (h >= 0).double()
        return (g.double() * ((ww * have)[:, :, None] * yy[h.clamp(min=0)]).sum(1)).sum()

    yd, wd = y.double(), w.double()
    for r in range(T * k):
        d = torch.zeros_like(yd)
        d[r, r % N] = 0.5
        num = f(yd + d, wd) - f(yd - d, wd)
        assert abs(num - gy[r, r % N]) <= 2.0 ** -8 * abs(num) + 1e-9
    for t in range(T):
        for j in range(k):
            d = torch.zeros_like(wd)
            d[t, j] = 0.5
            assert abs(f(yd, wd + d) - f(yd, wd - d) - gw[t, j]) <= 22 * U * float(g[t].double().abs() @ yd[h[t, j].clamp(min=0)].abs()) + 1e-9


def test_empty_calls():
    z = lambda *s, d=BF16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    out, _, _ = bsq.dispatch(z(0, 64), z(0, 3, d=I32))
    assert out.shape == (0, 64)
    assert bsq.combine(z(5, 64), z(0, 3, d=I32)).shape == (0, 64)
    y = bsq.combine(z(0, 64), torch.zeros((4, 2), dtype=I32, device="cuda"))       # no rows at all: every slot's is outside
    assert y.shape == (4, 64) and not y.any()
    gw = bsq.combine_backward(z(4, 64), z(0, 64), torch.zeros((4, 2), dtype=I32, device="cuda"))[3]
    assert gw.shape == (4, 2) and not gw.any()


def test_large_sorts_side_by_side():
    """Clusters of sixteen CTAs, captured in two graphs that run on two streams at once, on other slots than they were captured with."""
    held, graphs, outs = [], [], []
    for s in range(2):
        held.append(draw_ids(3000, 8, 256, s, 0.1).cuda())
        bsq.sort_experts(held[s], 256)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[s]):
            outs.append([bsq.sort_experts(held[s], 256) for _ in range(20)])
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    new = [draw_ids(3000, 8, 256, 7 + s, 0.1) for s in range(2)]
    for s in range(2):
        held[s].copy_(new[s])
    torch.cuda.synchronize()
    for s in range(2):
        with torch.cuda.stream(side[s]):
            graphs[s].replay()
    torch.cuda.synchronize()
    for s in range(2):
        want = sorted_plain(new[s], 256)
        for got in outs[s]:
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
