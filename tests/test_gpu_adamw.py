"""bsq_adamw against the formula in float64, in 32- and 8-bit states.

Tolerances.  A step has at most ten float32 roundings between its inputs and any output, each
2^-24 of a value no larger than the terms summed: 2^-20 of the sum of the terms' magnitudes
bounds them with room.  An 8-bit code is the E4M3 value below or above the exact one (up to
2^-20 of it), so it is less than one step of the E4M3 grid away; rounding at random makes
the mean error of N codes less than 5 standard deviations of N uniform steps, 5 / sqrt(3 N)
steps (a step rounded with probability p has variance p (1 - p) <= 1/4 < 1/3).
"""

import math

import numpy as np
import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq

pytestmark = pytest.mark.gpu

B = 128
LR, BETAS, EPS = 1e-2, (0.9, 0.95), 1e-8


def value(codes, scale):
    return codes.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(B)[:codes.numel()]


def make(n, grad, bits, seed, offset=0):
    """One tensor's buffers; `offset` elements into their storage (alignment)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = -(-n // B)

    def put(t):
        s = torch.empty(n + offset, dtype=t.dtype, device="cuda")[offset:]
        return s.copy_(t)

    d = dict(p=put(torch.randn(n, generator=g, device="cuda")), g=put((torch.randn(n, generator=g, device="cuda") * 1e-2).to(grad)),
             copy=put(torch.zeros(n, dtype=torch.bfloat16, device="cuda")), ms=None, vs=None)
    if bits == 32:
        d["m"] = put(torch.randn(n, generator=g, device="cuda") * 1e-3)
        d["v"] = put((torch.randn(n, generator=g, device="cuda") * 1e-2).square())
    else:
        d["m"] = put(torch.randint(0, 0x7F, (n,), generator=g, device="cuda").to(torch.uint8))
        d["v"] = put(torch.randint(1, 0x7F, (n,), generator=g, device="cuda").to(torch.uint8))
        d["ms"] = torch.rand(blocks, generator=g, device="cuda") * 1e-5
        d["vs"] = torch.rand(blocks, generator=g, device="cuda") * 1e-4 + 1e-6
    return d


def table(ts, wd=0.0, copies=True):
    pick = lambda k: [t[k] for t in ts]  # noqa: E731
    s8 = ts[0]["ms"] is not None
    return bsq.adamw_table(pick("p"), pick("g"), pick("m"), pick("v"), pick("ms") if s8 else None, pick("vs") if s8 else None,
                           copies=pick("copy") if copies else None, weight_decay=wd)


def exact(t, step, wd, gs):
    m, r = (t["m"].double(), t["v"].double().sqrt()) if t["ms"] is None else (value(t["m"], t["ms"]), value(t["v"], t["vs"]))
    g = t["g"].double() * gs
    b1, b2 = BETAS
    m, v = b1 * m + (1 - b1) * g, b2 * r * r + (1 - b2) * g * g
    u = LR * (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + EPS)
    return t["p"].double() * (1 - LR * wd) - u, m, v, t["p"].double().abs() + u.abs()


def close(got, ref, size):
    assert ((got.double() - ref).abs() <= 2.0 ** -20 * size + 1e-300).all(), (got.double() - ref).abs().max()


def grid(q):
    return torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)


def check_codes(codes, scale, ref):
    """Scales are the blocks' maxima / 448; codes are neighbours of the exact values."""
    n = ref.numel()
    pad = torch.zeros(-(-n // B) * B, dtype=torch.float64, device="cuda")
    pad[:n] = ref.abs()
    a = pad.view(-1, B).amax(1)
    a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
    close(scale, a / 448, a / 448)
    q = ref / (a / 448).repeat_interleave(B)[:n]
    v = codes.view(torch.float8_e4m3fn).double()
    assert ((v - q).abs() <= grid(q) * (1 + 2.0 ** -10)).all()
    return (v - q) / grid(q)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("wd,step", [(0.0, 1), (0.1, 7), (0.3, 100000)])
def test_one_step(bits, grad, offset, wd, step):
    """Lengths from nothing to several chunks, aligned and not, in one call."""
    sizes = [1, 0, 7, 8, 127, 128, 129, 1000, 4096, 4097, 20011]
    ts = [make(n, grad, bits, 10 + i, offset) for i, n in enumerate(sizes)]
    refs = [exact(t, step, wd, 0.5) for t in ts]
    bsq.adamw(table(ts, wd), step, LR, BETAS, EPS, grad_scale=torch.full((1,), 0.5, device="cuda"), seed=3)
    for t, (p, m, v, size) in zip(ts, refs):
        close(t["p"], p, size)
        assert torch.equal(t["copy"], t["p"].to(torch.bfloat16))
        if bits == 32:
            g = t["g"].double().abs()
            close(t["m"], m, m.abs() + g)
            close(t["v"], v, v)
        elif t["p"].numel():
            check_codes(t["m"], t["ms"], m)
            check_codes(t["v"], t["vs"], v.sqrt())


def in_float32(t, step, gs, seed):
    """The states after a step in float32 tensor operations, each rounded by itself: (m, v) or (m
    codes, m scales, v codes, v scales) of a tensor whose counter starts at 0."""
    b1, b2 = BETAS
    g = t["g"].float() * gs
    f = lambda c, s: c.view(torch.float8_e4m3fn).float() * s.repeat_interleave(B)[:c.numel()]  # noqa: E731
    m, v = (t["m"], t["v"]) if t["ms"] is None else (f(t["m"], t["ms"]), f(t["v"], t["vs"]).square())
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    if t["ms"] is None:
        return m, v
    mask, n = 0xFFFFFFFF, m.numel()
    x = (torch.arange(n, device="cuda") * 0x9E3779B1 + ((seed + step * 0x7F4A7C15) & mask)) & mask
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & mask
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & mask
    x = x ^ (x >> 16)
    got = []
    for y, bits, keep in ((m, x & 0xFFFF, False), (v.sqrt(), x >> 16, True)):
        pad = torch.zeros(-(-n // B) * B, device="cuda")
        pad[:n] = y
        a = pad.view(-1, B).abs().amax(1)
        a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
        top = torch.full_like(a, 448.0)
        q = y * (top / a).repeat_interleave(B)[:n]
        w = q.abs()
        big = ((w.view(torch.int32).long() + (bits << 4)) & ~0xFFFFF).to(torch.int32).view(torch.float32)
        r = torch.where(w >= 2.0 ** -6, big, torch.floor(w * 512 + bits.float() * 2.0 ** -16) * 2.0 ** -9).clamp(max=448.0)
        if keep:
            r = torch.where((q > 0) & (r == 0), torch.full_like(r, 2.0 ** -9), r)
        got += [torch.copysign(r, q), a / top]
    return got


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_states_follow_float32_bit_for_bit(bits, grad, offset):
    """No operation of the states is fused with another: they equal the same formula in float32
    tensor operations (the 8-bit codes by value: a zero has two)."""
    t = make(300001, grad, bits, 90, offset)
    want = in_float32(t, 5, 0.75, 11)
    bsq.adamw(table([t]), 5, LR, BETAS, EPS, grad_scale=torch.full((1,), 0.75, device="cuda"), seed=11)
    got = (t["m"], t["v"]) if bits == 32 else (t["m"].view(torch.float8_e4m3fn).float(), t["ms"],
                                               t["v"].view(torch.float8_e4m3fn).float(), t["vs"])
    for a, b in zip(got, want):
        assert torch.equal(a + 0.0, b + 0.0), (a != b).sum()


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch(bits):
    ts = [make(5 + 37 * i % 300, torch.float32, bits, i) for i in range(600)]
    wds = [0.1 * (i % 3) for i in range(600)]
    refs = [exact(t, 2, wd, 1.0) for t, wd in zip(ts, wds)]
    bsq.adamw(table(ts, wds, copies=False), 2, LR, BETAS, EPS)
    for t, (p, _, _, size) in zip(ts, refs):
        close(t["p"], p, size)
        assert (t["copy"] == 0).all()


def test_codes_are_right_on_average_and_repeat():
    n = 1 << 20
    runs = []
    for seed in (5, 5, 6):
        t = make(n, torch.float32, 8, 20)
        _, m, v, _ = exact(t, 3, 0.0, 1.0)
        bsq.adamw(table([t]), 3, LR, BETAS, EPS, seed=seed)
        for codes, scale, ref in ((t["m"], t["ms"], m), (t["v"], t["vs"], v.sqrt())):
            err = check_codes(codes, scale, ref)
            assert abs(err.mean().item()) <= 5 / math.sqrt(3 * n)
        runs.append((t["m"].clone(), t["v"].clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert not torch.equal(runs[0][0], runs[2][0])


def test_8bit_second_moment_decays():
    """With no gradient v falls by beta2 a step: a rounding to nearest would hold its root still."""
    n, steps, b2 = 1 << 16, 200, 0.995
    t = make(n, torch.float32, 8, 30)
    t["g"].zero_()
    before = value(t["v"], t["vs"])
    tab = table([t])
    for s in range(1, steps + 1):
        bsq.adamw(tab, s, 0.0, (0.9, b2), EPS, seed=1)
    after, want = value(t["v"], t["vs"]), before * b2 ** (steps / 2)
    assert abs((after.sum() / want.sum()).item() - 1) < 0.02
    assert (after > 0).all()


def test_8bit_from_zero_states():
    """Zero codes, any scale: the first step is that of 32-bit zero states; nothing divides by zero."""
    a, b = make(5000, torch.bfloat16, 8, 40), make(5000, torch.bfloat16, 32, 40)
    a["m"].zero_(), a["v"].zero_(), b["m"].zero_(), b["v"].zero_()
    b["p"].copy_(a["p"]), b["g"].copy_(a["g"])
    a["g"][:1000] = 0
    b["g"][:1000] = 0
    bsq.adamw(table([a]), 1, LR, BETAS, EPS)
    bsq.adamw(table([b]), 1, LR, BETAS, EPS)
    assert torch.equal(a["p"], b["p"]) and torch.isfinite(a["p"]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_nan_and_infinite_gradients_show(bits):
    t = make(1000, torch.float32, bits, 50)
    t["g"][3] = float("nan")
    t["g"][500] = float("inf")
    bsq.adamw(table([t]), 2, LR, BETAS, EPS)
    bad = ~torch.isfinite(t["p"])
    assert bad[3] and bad[500] and bad.sum() == 2
    m = t["m"].double() if bits == 32 else value(t["m"], t["ms"])
    assert not torch.isfinite(m[3]) and not torch.isfinite(m[500])
    if bits == 32:
        assert (~torch.isfinite(m)).sum() == 2


def test_other_stream():
    t, u = make(9000, torch.bfloat16, 8, 60), make(9000, torch.bfloat16, 8, 60)
    bsq.adamw(table([t]), 4, LR, BETAS, EPS, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bsq.adamw(table([u]), 4, LR, BETAS, EPS, seed=9, stream=side)
    torch.cuda.synchronize()
    for k in ("p", "m", "v", "ms", "vs", "copy"):
        assert torch.equal(t[k], u[k]), k


def test_refusals():
    t = make(100, torch.float32, 8, 70)
    args = lambda **k: bsq.adamw_table(**{**dict(params=[t["p"]], grads=[t["g"]], ms=[t["m"]], vs=[t["v"]], m_scales=[t["ms"]],  # noqa: E731
                                               v_scales=[t["vs"]]), **k})
    args()
    for bad in (dict(params=[t["p"].half()]), dict(grads=[t["g"][:50]]), dict(grads=[]), dict(m_scales=None), dict(ms=[t["p"]]),
                dict(m_scales=[torch.empty(2, device="cuda")]), dict(grads=[t["g"].cpu()]), dict(weight_decay=[0.1, 0.1]),
                dict(copies=[t["p"]]), dict(vs=[t["v"][::2]])):
        with pytest.raises(ValueError):
            args(**bad)
    for bad in (dict(step=0), dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0)):
        with pytest.raises(bsq.BsqError):
            bsq.adamw(args(), **{**dict(step=1, lr=LR), **bad})
    with pytest.raises(ValueError):
        bsq.adamw(args(), 1, LR, grad_scale=torch.ones(2, device="cuda"))
    assert np.isfinite(t["p"].cpu().numpy()).all()
