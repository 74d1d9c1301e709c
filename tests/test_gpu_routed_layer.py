"""The router, the sort, dispatch, the experts' products and combine together, as a mixture layer runs them: forward and
gradients against 64 bits, single tokens through 4-bit experts, captured graphs and other streams.

Tolerances.  A product's rows are off by the BF16 rounding, 2.5e-3 over a matrix (test_gpu_fp8.py); combine adds one
more rounding of its own result and passes the rows' on: 2.5e-3 of the norm of the weighted rows and as much of the sum's.
A quantized gradient is off by half a step of E4M3, 2^-4 of a value at most; so are sums of its products over a matrix.
"""

import os
import sys

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq, synth

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def dequantized(codes, scale, block):
    v = codes.view(torch.float8_e4m3fn).double()
    s = scale.double().repeat_interleave(block, -2)[..., :v.shape[-2], :].repeat_interleave(128, -1)[..., :v.shape[-1]]
    return v * s


def tokens(T, K, seed):
    return synth.randn((T, K), 1.0, seed, "cuda", BF16)


@pytest.mark.parametrize("T,experts,n,k,slots", [(1, 4, 128, 256, 2), (37, 5, 272, 400, 3), (300, 16, 256, 512, 4)])
def test_forward_and_gradients(T, experts, n, k, slots):
    from routed_layer import RoutedLayer
    layer = RoutedLayer(experts, n, k, slots, seed=T)
    layer.gate *= 5
    x, g = tokens(T, k, 1), tokens(T, n, 2)
    y, saved = layer.forward(x)
    grad_x, grad_gate = layer.backward(g, saved)
    _, logits, ids, weights, offsets, rows, held, ry = saved
    assert int(offsets[-1]) == T * slots
    # 64 bits, on the quantized operands
    w = dequantized(layer.experts.w.data, layer.experts.w.scale, 128)
    xq = dequantized(*bsq.quantize_e4m3(x), 1)
    gate = layer.gate.double().requires_grad_()
    leaf = x.double().requires_grad_()
    p = torch.softmax((leaf @ gate.T).gather(1, ids.long()), dim=1)
    terms = torch.einsum("tk,tjnk->tjn", leaf, w[ids.long()])
    exact_terms = p.detach()[:, :, None] * torch.einsum("tk,tjnk->tjn", xq, w[ids.long()])
    ref = exact_terms.sum(1)
    assert (y.double() - ref).norm() <= 2.5e-3 * (exact_terms.norm() + ref.norm())
    # gradients of the layer without its quantization: off by that of g and x, 2^-4 of each product's operand at most
    ((p[:, :, None] * terms).sum(1) * g.double()).sum().backward()
    assert (grad_x.double() - leaf.grad).norm() <= 2.0 ** -4 * leaf.grad.norm() + 2.0 ** -4 * g.double().norm() * w.norm() / experts ** 0.5 * 0.1
    size = (p.detach() * (g.double()[:, None, :] * terms.detach()).norm(dim=2)).norm() * x.double().norm(dim=1).max()
    assert (grad_gate.double() - gate.grad).norm() <= 2.0 ** -4 * size
    # the weight gradient of each expert, from the rows that were dispatched
    r0 = 0
    gy, _, _, _ = bsq.combine_backward(g, ry, rows, weights)
    for e, r1 in enumerate(offsets.tolist()):
        want = gy[r0:r1].double().T @ held[r0:r1].double()
        got = layer.experts.grad[e].double()
        assert (got - want).norm() <= 2.5e-3 * want.norm() if r1 > r0 else not got.any()
        r0 = r1
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


@pytest.mark.parametrize("fmt", [synth.FMT_MXFP4, synth.FMT_NVFP4])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_decoding_through_4_bit_experts(fmt, T):
    from routed_layer import Fp4Layer, RoutedLayer
    layer = Fp4Layer(RoutedLayer(12, 264, 512, 3, seed=5), fmt)
    x = tokens(T, 512, 6)
    y = layer.forward(x)
    ids, weights = bsq.route(x.float() @ layer.gate.T, 3)
    w = bsq.dequant(layer.w).double()
    terms = weights.double()[:, :, None] * torch.einsum("tk,tjnk->tjn", x.double(), w[ids.long()])
    assert (y.double() - terms.sum(1)).norm() <= 2.5e-3 * (terms.norm() + terms.sum(1).norm())
    # the last token alone: another kernel of the same sums
    one, last = layer.forward(x[T - 1:].contiguous()).double(), terms[T - 1:]
    assert (one - last.sum(1)).norm() <= 2.5e-3 * (last.norm() + last.sum(1).norm())


def parts(layer, x, stream=None):
    logits = x[0] @ layer.gate.T
    ids, w = bsq.route(logits, 2, stream=stream)
    offsets, rows, slots = bsq.sort_experts(ids, layer.w.batch, stream=stream)
    held, codes, scale = bsq.dispatch(x[1], rows, w, e4m3=True, stream=stream)
    y = bsq.fp4_grouped_forward(held, layer.w, offsets, stream=stream)
    out = bsq.combine(y, rows, w, stream=stream)
    gy, gc, gs, gw = bsq.combine_backward(out, y, rows, w, e4m3=True, stream=stream)
    gl = bsq.route_backward(logits, ids, gw, stream=stream)
    return [ids, w, offsets, rows, slots, held, codes, scale, y, out, gy, gc, gs, gw, gl]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_captured_graphs_follow_their_inputs():
    """Two graphs of the whole chain, replayed in turn and side by side on other tokens than they were captured with."""
    from routed_layer import Fp4Layer, RoutedLayer
    layer = Fp4Layer(RoutedLayer(8, 128, 256, seed=9))
    draw = lambda s: (synth.randn((50, 256), 1.0, s, "cuda"), tokens(50, 256, s + 1))  # noqa: E731
    held, graphs, outs = [], [], []
    for s in (20, 30):
        x = draw(s)
        parts(layer, x)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(parts(layer, x))
        held.append(x)
        graphs.append(gr)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for round_ in range(3):
        want = []
        for i in range(2):
            new = draw(100 * round_ + 10 * i)
            for dst, src in zip(held[i], new):
                dst.copy_(src)
            want.append([t.clone() for t in parts(layer, new)])
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1])
    assert bsq.get_device_error() == (bsq.BSQ_OK, 0)


def test_another_stream_gives_the_same():
    from routed_layer import Fp4Layer, RoutedLayer
    layer = Fp4Layer(RoutedLayer(8, 128, 256, seed=9))
    x = (synth.randn((50, 256), 1.0, 3, "cuda"), tokens(50, 256, 4))
    want = parts(layer, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = parts(layer, x, side)
    side.synchronize()
    assert same(got, want)


def test_a_padded_batch():
    """Tokens whose logits are all minus infinity have no rows, give zeros and get zero gradients."""
    from routed_layer import Fp4Layer, RoutedLayer
    layer = Fp4Layer(RoutedLayer(8, 128, 256, seed=9))
    logits, x = synth.randn((20, 8), 1.0, 3, "cuda"), tokens(20, 256, 4)
    logits[13:] = -float("inf")
    ids, w = bsq.route(logits, 2)
    offsets, rows, slots = bsq.sort_experts(ids, 8)
    held = torch.full((40, 256), 7.0, dtype=BF16, device="cuda")
    bsq.dispatch(x, rows, out=held)
    y = torch.full((40, 128), 5.0, dtype=BF16, device="cuda")
    bsq.fp4_grouped_forward(held, layer.w, offsets, out=y)
    out = bsq.combine(y, rows, w)
    gw = bsq.combine_backward(out, y, rows, w)[3]
    gl = bsq.route_backward(logits, ids, gw)
    assert int(offsets[-1]) == 26 and (held[26:] == 7).all() and (y[26:] == 5).all() and (slots[26:] == -1).all()
    assert not out[13:].any() and not gw[13:].any() and not gl[13:].any() and out[:13].any(dim=1).all()


def test_training_runs_and_its_gradients_are_finite():
    from routed_layer import RoutedLayer, train
    layer = RoutedLayer(8, 256, 512, seed=3)
    before = layer.gate.clone(), layer.experts.master.clone()
    losses = train(layer, 4, tokens=128)
    assert all(torch.isfinite(torch.tensor(losses))) and torch.isfinite(layer.gate).all() and torch.isfinite(layer.experts.master).all()
    assert not torch.equal(layer.gate, before[0]) and not torch.equal(layer.experts.master, before[1])
