"""A mixture layer, trained in FP8 and served with 4-bit weights by the library's operators.

    python examples/routed_layer.py         # trains on synthetic data, then decodes with MXFP4 experts

Tokens choose their experts (route), go to the experts' rows as E4M3 codes and as BF16 (sort_experts,
dispatch), are multiplied there, and come back with the gate's weights (combine).  The backward
goes the same way in reverse: the gradient reaches the rows (combine_backward), the tokens
(combine), the gate's weights and through them the router.  Serving keeps 4-bit codes of the
experts and takes few tokens at a time.
"""

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [HERE, os.path.join(HERE, "..")]

from block_scaled_gemm_fp8_gb300 import bsq, synth  # noqa: E402
from fp8_experts import Fp8Experts  # noqa: E402


class RoutedLayer:
    """y[t] = sum_j w[t, j] W[ids[t, j]] x[t], with ids and w from the softmax of x @ gate^T over the k best."""

    def __init__(self, experts, n, k, slots=2, seed=0, device="cuda"):
        self.experts = Fp8Experts(experts, n, k, seed=seed, device=device)
        self.gate = synth.randn((experts, k), 0.02, seed + 1, device)
        self.slots, self.lr = slots, 0.05

    def forward(self, x):
        """The output of BF16 tokens x [T, k], and what the backward needs."""
        logits = x.float() @ self.gate.T
        ids, weights = bsq.route(logits, self.slots)
        offsets, rows, _ = bsq.sort_experts(ids, self.experts.experts, want_slots=False)
        held, codes, scale = bsq.dispatch(x, rows, e4m3=True)
        y = bsq.fp8_grouped_forward(codes, scale, self.experts.w, offsets)
        return bsq.combine(y, rows, weights), (x, logits, ids, weights, offsets, rows, held, y)

    def backward(self, grad_out, saved):
        """(gradient of x, of the gate); the experts' goes to their .grad."""
        x, logits, ids, weights, offsets, rows, held, y = saved
        e = self.experts
        grad_y, codes, scale, grad_weights = bsq.combine_backward(grad_out, y, rows, weights, e4m3=True)
        grad_rows = bsq.fp8_grouped_dgrad(codes, scale, e.w, offsets)
        packed = synth.Packed(synth.FMT_BF16, held, None, None, 1, held.shape[0], e.k)
        bsq.grouped_wgrad(grad_y, packed, offsets, e.experts, out=e.grad)
        grad_logits = bsq.route_backward(logits, ids, grad_weights)
        grad_x = bsq.combine(grad_rows, rows).float() + grad_logits @ self.gate
        return grad_x, grad_logits.T @ x.float()

    def update(self, lr, grad_gate):
        self.experts.update(lr)
        self.gate -= self.lr * grad_gate


class Fp4Layer:
    """The same layer for a few tokens, its experts' weights in MXFP4 or NVFP4."""

    def __init__(self, layer, fmt=synth.FMT_MXFP4):
        self.w, self.gate, self.slots = synth.quantize(fmt, layer.experts.master), layer.gate, layer.slots

    def forward(self, x):
        ids, weights = bsq.route(x.float() @ self.gate.T, self.slots)
        offsets, rows, _ = bsq.sort_experts(ids, self.w.batch, want_slots=False)
        held, _, _ = bsq.dispatch(x, rows)
        return bsq.combine(bsq.fp4_grouped_forward(held, self.w, offsets), rows, weights)


def train(layer, steps, tokens=512, lr=2e-3, seed=1, device="cuda"):
    """Teaches the layer a second one's outputs; the loss of every step."""
    teacher = RoutedLayer(layer.experts.experts, layer.experts.n, layer.experts.k, layer.slots, seed + 100, device)
    losses = []
    for i in range(steps):
        x = synth.randn((tokens, layer.experts.k), 1.0, seed + i, device, torch.bfloat16)
        y, saved = layer.forward(x)
        diff = y.float() - teacher.forward(x)[0].float()
        losses.append(diff.square().mean())
        _, grad_gate = layer.backward((2.0 / tokens * diff).to(torch.bfloat16), saved)
        layer.update(lr, grad_gate)
    return torch.stack(losses).tolist()


def main():
    torch.cuda.set_device(0)
    layer = RoutedLayer(8, 512, 1024)
    losses = train(layer, 60)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    token = synth.randn((3, layer.experts.k), 1.0, 7, "cuda", torch.bfloat16)
    print("three tokens through MXFP4 experts:", Fp4Layer(layer).forward(token).float().norm(dim=1).tolist())
    status, code = bsq.get_device_error()
    assert status == bsq.BSQ_OK and code == 0, (status, code)


if __name__ == "__main__":
    main()
