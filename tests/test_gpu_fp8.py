"""Products of E4M3 operands on their own codes (bsq_fp8_forward, bsq_fp8_dgrad and their grouped
forms) against the float64 definition

    y[m, n]  = sum_b xs[m, b] ws[n/128, b] sum_{k in b} xc[m, k] wc[n, k]
    gx[m, k] = sum_b gs[m, b] ws[b, k/128] sum_{n in b} gc[m, n] wc[n, k]

Tolerance.  A code product has 8 mantissa bits and is exact in FP32; the scale xs * ws and
its product with a partial sum are rounded to float32 (2^-24 each), the sums run in FP32;
the result is rounded to BF16 once, at most 2^-9 of it.  The elementwise bound is that of
every product of the library (2e-2 sqrt(Kc) rms rms, plus 2^-8 |ref|); over the matrix the
relative error is the BF16 rounding's alone, at most 2^-9, so 2.5e-3 leaves 28 % for FP32
accumulation.  One-hot operands leave a single product, whose result has one value bit for
bit.
"""

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth
from oracle import formats as F
from oracle import gemm as Gm
from tests._util import bf16_vals

pytestmark = pytest.mark.gpu

REL = 2.5e-3
E4M3 = np.arange(256, dtype=np.uint8)


def e4m3_values(codes):
    t = torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).to(torch.float64)
    return t.numpy()


def draw_rows(M, K, seed):
    """Random finite codes [M, K] and a positive scale per 128 columns of each row."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (M, K)).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1
    s = (rng.uniform(0.5, 1.5, (M, -(-K // 128))) * 2.0 ** rng.integers(-6, 3, (M, -(-K // 128)))).astype(np.float32)
    return c, s


def draw_weight(E, N, K, seed):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (E, N, K)).astype(np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1
    shape = (E, -(-N // 128), -(-K // 128))
    s = (rng.uniform(0.5, 1.5, shape) * 2.0 ** rng.integers(-8, 0, shape)).astype(np.float32)
    return c, s


def packed(c, s):
    E, N, K = c.shape
    return synth.Packed(synth.FMT_FP8, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), None, E, N, K)


def row_values(c, s):
    return e4m3_values(c) * np.repeat(s.astype(np.float64), 128, axis=1)[:, :c.shape[1]]


def weight_values(c, s):
    v = np.repeat(np.repeat(s.astype(np.float64), 128, axis=1), 128, axis=2)[:, :c.shape[1], :c.shape[2]]
    return e4m3_values(c) * v


def check(out, ref, a, b, kc, what):
    got = bf16_vals(out)
    ok, err, rel = Gm.check(got, ref, Gm.tolerance(kc, a, b), rel_fro=REL)
    assert ok, f"{what}: max|err|={err:.4g} relF={rel:.3g}"


DENSE = [(1, 8, 16), (1, 128, 128), (3, 40, 144), (8, 256, 512), (9, 1000, 400), (16, 264, 2064), (17, 520, 1024),
         (32, 128, 4096), (33, 256, 128), (64, 8, 640), (129, 264, 96), (256, 256, 1024), (257, 776, 1168), (600, 1320, 2064),
         (100, 1024, 5136), (40, 136, 4112)]   # the last two: tiles split over a cluster, uneven parts


@pytest.mark.parametrize("M,N,K", DENSE)
def test_forward(M, N, K):
    xc, xs = draw_rows(M, K, 1)
    wc, ws = draw_weight(1, N, K, 2)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.fp8_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws), out=y)
    x, w = row_values(xc, xs), weight_values(wc, ws)[0]
    check(y, x @ w.T, x, w, K, "forward")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 128, 128), (5, 144, 48), (16, 2064, 272), (129, 96, 256), (256, 512, 512),
                                   (300, 1168, 784), (520, 256, 2064), (70, 4112, 528)])
def test_dgrad(M, N, K):
    gc, gs = draw_rows(M, N, 3)
    wc, ws = draw_weight(1, N, K, 4)
    gx = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.fp8_dgrad(torch.from_numpy(gc).cuda(), torch.from_numpy(gs).cuda(), packed(wc, ws), out=gx)
    g, w = row_values(gc, gs), weight_values(wc, ws)[0]
    check(gx, g @ w, g, w, N, "dgrad")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_first_operand_beyond_l2_share(direction):
    """54 MB of first operand: its row tiles go in groups.  Every output is written, and rows and
    columns from every tile, the last ones and both sides of the groups' border, are right."""
    M, inner, outer = 3301, 16384, 528
    xc, xs = draw_rows(M, inner, 18)
    wc, ws = draw_weight(1, *((outer, inner) if direction == "forward" else (inner, outer)), 19)
    y = torch.full((M, outer), float("nan"), dtype=torch.bfloat16, device="cuda")
    call = bsq.fp8_forward if direction == "forward" else bsq.fp8_dgrad
    call(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws), out=y)
    assert torch.isfinite(y).all()
    rows = np.unique(np.concatenate([np.arange(5, M, 97), [0, 1663, 1664, M - 1]]))
    cols = np.unique(np.concatenate([np.arange(3, outer, 41), [0, 255, 256, outer - 1]]))
    x, w = row_values(xc[rows], xs[rows]), weight_values(wc, ws)[0]
    w = w[cols] if direction == "forward" else w[:, cols]
    check(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], x @ (w.T if direction == "forward" else w), x, w,
          inner, direction)
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


ROUTING = [[0, 5, 0, 0, 1], [1, 1, 1, 1], [256, 0, 257, 1, 0, 130], [0, 0, 700], [3] * 40, [64, 0, 8, 15, 2, 33, 128, 300]]


@pytest.mark.parametrize("counts", ROUTING)
@pytest.mark.parametrize("N,K", [(264, 400), (512, 256)])
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_grouped(direction, N, K, counts):
    """Ragged experts, empty ones, and trailing rows that belong to none: their codes are NaN codes
    and their outputs keep what they held."""
    if direction == "dgrad" and N % 16:
        N += 8
    E, used, S = len(counts), sum(counts), sum(counts) + 5
    offs = synth.offsets_from_counts(counts)
    inner, outer = (K, N) if direction == "forward" else (N, K)
    xc, xs = draw_rows(S, inner, 5)
    xc[used:] = 0x7F
    xs[used:] = np.nan
    wc, ws = draw_weight(E, N, K, 6)
    y = torch.full((S, outer), 7.0, dtype=torch.bfloat16, device="cuda")
    call = bsq.fp8_grouped_forward if direction == "forward" else bsq.fp8_grouped_dgrad
    call(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws), torch.from_numpy(offs).cuda(), out=y)
    assert (y[used:] == 7.0).all()
    x, w = row_values(xc[:used], xs[:used]), weight_values(wc, ws)
    for e in range(E):
        r0, r1 = Gm.expert_rows(offs, e)
        if r1 > r0:
            ref = x[r0:r1] @ (w[e].T if direction == "forward" else w[e])
            check(y[r0:r1], ref, x[r0:r1], w[e], inner, f"{direction} expert {e}")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("counts", [[0, 1, 0, 2, 0, 0, 0, 0], [0] * 20 + [1, 0, 19, 0, 0, 9], [1] * 13])
def test_grouped_few_rows(counts):
    """No more rows than experts: an expert has none, one, or more than one pass over W takes."""
    N, K = 264, 400
    E, S = len(counts), len(counts)
    used, offs = sum(counts), synth.offsets_from_counts(counts)
    if used > S:
        E = S = used
        offs = np.concatenate([offs, np.full(used - len(counts), used, dtype=offs.dtype)])
    xc, xs = draw_rows(S, K, 16)
    xc[used:] = 0x7F
    wc, ws = draw_weight(E, N, K, 17)
    y = torch.full((S, N), 7.0, dtype=torch.bfloat16, device="cuda")
    bsq.fp8_grouped_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws),
                            torch.from_numpy(offs).cuda(), out=y)
    assert (y[used:] == 7.0).all()
    x, w = row_values(xc[:used], xs[:used]), weight_values(wc, ws)
    for e in range(E):
        r0, r1 = Gm.expert_rows(offs, e)
        if r1 > r0:
            check(y[r0:r1], x[r0:r1] @ w[e].T, x[r0:r1], w[e], K, f"expert {e}")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("M", [4, 20, 300])
@pytest.mark.parametrize("direction", ["forward", "dgrad"])
def test_one_hot_is_one_product(direction, M):
    """Row i holds one code at column k_i: every output is code * code * (xs * ws), with the float32
    roundings of xs * ws and of its product, then BF16: compared bit for bit.  W's scales reach
    2^-100 and 2^60, subnormal codes included."""
    N, K = 400, 656
    inner, outer = (K, N) if direction == "forward" else (N, K)
    rng = np.random.default_rng(7)
    xc = np.zeros((M, inner), np.uint8)
    ks = rng.integers(0, inner, M)
    ks[:3] = [0, inner - 1, inner // 2]
    xc[np.arange(M), ks] = rng.integers(1, 0x7F, M)
    _, xs = draw_rows(M, inner, 8)
    wc, ws = draw_weight(1, N, K, 9)
    ws[0, 0, 0], ws[0, 1, 2], ws[0, 2, 1] = 2.0 ** -100, 2.0 ** 60, 1e-3
    call = bsq.fp8_forward if direction == "forward" else bsq.fp8_dgrad
    y = call(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws))
    w, s = e4m3_values(wc[0]), np.repeat(np.repeat(ws[0], 128, 0), 128, 1)[:N, :K]
    if direction == "dgrad":
        w, s = w.T, s.T                                     # [outer, inner]
    scale = xs[np.arange(M), ks // 128][:, None] * s[:, ks].T               # float32
    prod = (e4m3_values(xc)[np.arange(M), ks][:, None] * w[:, ks].T).astype(np.float32)   # exact
    np.testing.assert_array_equal(bf16_vals(y) + 0.0, F.bf16_round((prod * scale).astype(np.float64)) + 0.0)


def test_nan_and_infinite_scales_stay_in_their_rows():
    M, N, K = 40, 256, 512
    for rows in (M, 300):
        xc, xs = draw_rows(rows, K, 10)
        wc, ws = draw_weight(1, N, K, 11)
        xs[3, 1] = np.nan
        xc[5, 300] = 0x7F
        xs[7, 0] = np.inf
        y = bf16_vals(bsq.fp8_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws)))
        assert np.isnan(y[3]).all() and np.isnan(y[5]).all() and not np.isfinite(y[7]).any()
        rest = np.delete(y, [3, 5, 7], axis=0)
        assert np.isfinite(rest).all()


@pytest.mark.parametrize("S", [6, 700])
def test_bad_offsets_write_nothing(S):
    N = K = 256
    xc, xs = draw_rows(S, K, 12)
    wc, ws = draw_weight(3, N, K, 13)
    for offs in ([4, 2, S], [1, 3, S + 1], [-1, 2, 3]):
        for call in (bsq.fp8_grouped_forward, bsq.fp8_grouped_dgrad):
            y = torch.full((S, K), 3.0, dtype=torch.bfloat16, device="cuda")
            call(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws),
                 torch.tensor(offs, dtype=torch.int32, device="cuda"), out=y)
            st, code = bsq.get_device_error()
            assert (st, code) == (bsq.BSQ_ERR_INVALID_ARG, 2)
            assert (y == 3.0).all()


@pytest.mark.parametrize("K", [16, 400, 2064])
def test_grouped_many_experts_of_few_rows(K):
    """CTAs enough for the small ones of a short contraction: most experts empty, one with 11 rows."""
    E, N = 200, 136
    counts = np.zeros(E, dtype=np.int64)
    counts[[3, 50, 51, 120]], counts[77], counts[199] = 1, 11, 4
    used = int(counts.sum())
    offs = synth.offsets_from_counts(list(counts))
    xc, xs = draw_rows(used, K, 20)
    wc, ws = draw_weight(E, N, K, 21)
    y = torch.full((used, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    bsq.fp8_grouped_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws),
                            torch.from_numpy(offs).cuda(), out=y)
    x = row_values(xc, xs)
    for e in np.flatnonzero(counts):
        r0, r1 = Gm.expert_rows(offs, int(e))
        w = weight_values(wc[e:e + 1], ws[e:e + 1])[0]
        check(y[r0:r1], x[r0:r1] @ w.T, x[r0:r1], w, K, f"expert {e}")
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("offs", [[4, 2, 3, 3, 6, 6], [1, 3, 3, 3, 3, 7], [-1, 2, 2, 2, 2, 3]])
def test_bad_offsets_of_few_rows_write_nothing(offs):
    """The same with no more rows than experts."""
    S, N, K = 6, 256, 256
    xc, xs = draw_rows(S, K, 12)
    wc, ws = draw_weight(6, N, K, 13)
    y = torch.full((S, K), 3.0, dtype=torch.bfloat16, device="cuda")
    bsq.fp8_grouped_forward(torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws),
                            torch.tensor(offs, dtype=torch.int32, device="cuda"), out=y)
    assert bsq.get_device_error() == (bsq.BSQ_ERR_INVALID_ARG, 2)
    assert (y == 3.0).all()


def test_results_repeat_and_streams():
    """The same call twice, and on another stream than the default one: the same bits."""
    for M in (12, 900):
        xc, xs = draw_rows(M, 1040, 14)
        wc, ws = draw_weight(1, 776, 1040, 15)
        x, s, w = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws)
        first = bsq.fp8_forward(x, s, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        second = bsq.fp8_forward(x, s, w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), second.view(torch.int16))


def test_dgrad_is_the_gradient_of_forward():
    """<G, forward(X + d) - forward(X)> = <dgrad(G), d> for operands whose values, differences and
    products are exact: small integers with unit scales."""
    M, N, K = 70, 256, 384
    rng = np.random.default_rng(16)
    code = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    ones = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    x, d = rng.integers(-2, 3, (M, K)), rng.integers(-1, 2, (M, K))
    g, w = rng.integers(-1, 2, (M, N)), rng.integers(-1, 2, (1, N, K))
    keep = rng.random((1, N, K)) < 0.1   # sparse, so that every output is an integer below 2^8
    w = w * keep
    W = synth.Packed(synth.FMT_FP8, code(w), ones(1, 2, 3), None, 1, N, K)
    y0 = bf16_vals(bsq.fp8_forward(code(x), ones(M, 3), W))
    y1 = bf16_vals(bsq.fp8_forward(code(x + d), ones(M, 3), W))
    gx = bf16_vals(bsq.fp8_dgrad(code(g), ones(M, 2), W))
    assert np.abs(y0).max() < 256 and np.abs(y1).max() < 256 and np.abs(gx).max() < 256
    assert (g * (y1 - y0)).sum() == (gx * d).sum()


def test_empty_sizes():
    wc, ws = draw_weight(1, 128, 256, 17)
    w = packed(wc, ws)
    assert bsq.fp8_forward(torch.empty((0, 256), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda"), w).shape == (0, 128)
    e = synth.Packed(synth.FMT_FP8, torch.empty((1, 128, 0), dtype=torch.uint8, device="cuda"), torch.empty((1, 1, 0), device="cuda"),
                     None, 1, 128, 0)
    y = bsq.fp8_forward(torch.empty((3, 0), dtype=torch.uint8, device="cuda"), torch.empty((3, 0), device="cuda"), e)
    assert (y == 0).all() and y.shape == (3, 128)


def test_binding_refuses():
    xc, xs = draw_rows(20, 256, 18)
    wc, ws = draw_weight(2, 128, 256, 19)
    x, s, w = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda(), packed(wc, ws)
    one = synth.Packed(synth.FMT_FP8, w.data[:1], w.scale[:1], None, 1, 128, 256)
    offs = torch.tensor([5, 20], dtype=torch.int32, device="cuda")
    for bad in (lambda: bsq.fp8_forward(x, s, w),                                   # two weights, no offsets
                lambda: bsq.fp8_forward(x[:, :128], s, one),                        # strided codes
                lambda: bsq.fp8_forward(x, s[:, :1].contiguous(), one),             # scales of another width
                lambda: bsq.fp8_forward(x.cpu(), s, one),
                lambda: bsq.fp8_forward(x, s.double(), one),
                lambda: bsq.fp8_forward(x, s, one, out=torch.empty((20, 64), dtype=torch.bfloat16, device="cuda")),
                lambda: bsq.fp8_grouped_forward(x, s, w, offs.long()),
                lambda: bsq.fp8_grouped_forward(x, s, w, offs[:1])):
        with pytest.raises(ValueError):
            bad()
    mx = synth.Packed(synth.FMT_MXFP4, one.data, one.scale, None, 1, 128, 256)
    with pytest.raises(bsq.BsqError):
        bsq.fp8_forward(x, s, mx)
