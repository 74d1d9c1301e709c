"""A layer of experts trained and served in FP8 with the library's operators.

    python examples/fp8_experts.py          # trains on synthetic data, then decodes single tokens

Master weights stay in float32.  Every step quantizes them in 128 x 128 blocks and the
activations in 1 x 128 blocks, multiplies the E4M3 codes per expert (forward and input
gradient), takes the weight gradient from the BF16 activations, and updates the masters with
AdamW, whose states are 8-bit codes.  Serving keeps the codes of the weights and quantizes
the tokens alone.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from block_scaled_gemm_fp8_gb300 import bsq, synth  # noqa: E402


class Fp8Experts:
    """y[r0:r1] = x[r0:r1] @ W[e]^T for the rows of each expert e (cumulative int32 end offsets)."""

    def __init__(self, experts, n, k, std=0.02, seed=0, device="cuda"):
        self.master = synth.randn((experts, n, k), std, seed, device)
        self.experts, self.n, self.k, self.step = experts, n, k, 0
        self.grad = torch.zeros((experts, n, k), dtype=torch.bfloat16, device=device)
        codes = lambda: torch.zeros((experts, n, k), dtype=torch.uint8, device=device)  # noqa: E731
        scales = lambda: torch.ones((experts, -(-n * k // 128)), device=device)  # noqa: E731
        self.m, self.v, self.m_scale, self.v_scale = codes(), codes(), scales(), scales()
        # one tensor per expert, so that an optimizer may treat them one by one
        self.table = bsq.adamw_table(self.master.unbind(), self.grad.unbind(), self.m.unbind(), self.v.unbind(),
                                     self.m_scale.unbind(), self.v_scale.unbind(), weight_decay=0.01)
        self.quantize_weights()

    def quantize_weights(self):
        codes, scale = bsq.quantize_e4m3(self.master, block_rows=128)
        self.w = synth.Packed(synth.FMT_FP8, codes, scale, None, self.experts, self.n, self.k)

    def forward(self, x, offsets):
        codes, scale = bsq.quantize_e4m3(x)
        return bsq.fp8_grouped_forward(codes, scale, self.w, offsets)

    def backward(self, grad_y, x, offsets):
        """The input gradient; the weight gradient goes to self.grad."""
        codes, scale = bsq.quantize_e4m3(grad_y)
        grad_x = bsq.fp8_grouped_dgrad(codes, scale, self.w, offsets)
        rows = synth.Packed(synth.FMT_BF16, x, None, None, 1, x.shape[0], self.k)
        bsq.grouped_wgrad(grad_y, rows, offsets, self.experts, out=self.grad)
        return grad_x

    def update(self, lr):
        self.step += 1
        bsq.adamw(self.table, step=self.step, lr=lr, betas=(0.9, 0.95), seed=self.step)
        self.quantize_weights()


def train(layer, steps, rows=512, lr=2e-3, seed=1, device="cuda"):
    """Teaches the layer a second one's outputs; the loss of every step."""
    teacher = Fp8Experts(layer.experts, layer.n, layer.k, seed=seed + 100, device=device)
    losses = []
    for i in range(steps):
        counts = synth.zipf_counts(rows, layer.experts, 1.1, seed + i, force_empty=(0,))
        offsets = torch.from_numpy(synth.offsets_from_counts(counts)).to(device)
        x = synth.randn((rows, layer.k), 1.0, seed + i, device, torch.bfloat16)
        y = layer.forward(x, offsets)
        diff = y.float() - teacher.forward(x, offsets).float()
        losses.append(diff.square().mean())
        layer.backward((2.0 / rows * diff).to(torch.bfloat16), x, offsets)
        layer.update(lr)
    return torch.stack(losses).tolist()


def main():
    torch.cuda.set_device(0)
    layer = Fp8Experts(8, 512, 1024)
    losses = train(layer, 120)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    offsets = torch.tensor([0, 1, 1, 1, 2, 2, 3, 3], dtype=torch.int32, device="cuda")
    token = synth.randn((3, layer.k), 1.0, 7, "cuda", torch.bfloat16)
    print("three tokens decoded by experts 1, 4 and 6:", layer.forward(token, offsets).float().norm(dim=1).tolist())
    status, code = bsq.get_device_error()
    assert status == bsq.BSQ_OK and code == 0, (status, code)


if __name__ == "__main__":
    main()
