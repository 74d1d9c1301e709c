"""Timed cases of the FP8 training and serving operators: block-scaled E4M3 quantization, the
products of E4M3 operands on their own codes (dense and per expert, forward and dgrad), and
the AdamW step over many tensors.

``own`` selects who computes: False, elementary torch operations in float32 (`plain_*`);
True, the framework's entry points.  The definitions, with B = 128:

  quantize  a block is 1 x B (activations, gradients) or B x B (weights) elements;
            a = max |x| over it (a zero block takes 448, a smaller one than 2^-100 takes 2^-100),
            scale = a / 448, code = E4M3(x * (448 / a)), nearest even, saturating
  forward   y[m, n]  = sum_b xs[m, b] ws[n/B, b] sum_{k in block b} xc[m, k] wc[n, k]
  dgrad     gx[m, k] = sum_b gs[m, b] ws[b, k/B] sum_{n in block b} gc[m, n] wc[n, k]
  grouped   the same with W[e] for the token rows of expert e (cumulative int32 end offsets)
  adamw     g = grad * grad_scale;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
            p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps);
            8-bit states hold m and r = sqrt(v) as E4M3 codes with a scale per B elements of
            the tensor, rounded at random by 16 bits each of a hash of (seed, element);
            an r above zero keeps at least the smallest code above zero
"""

import math
import random
from types import SimpleNamespace

import torch

own = False

B = 128
BETAS, EPS, LR = (0.9, 0.95), 1e-8, 1e-3
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode batch's activations: nothing but latency
        dict(name="quantize_decode_rows", op="quantize", batch=1, rows=16, cols=4096, block=1, dtype="bf16"),
        # the activations of the FFN workload, odd row count
        dict(name="quantize_ffn_rows", op="quantize", batch=1, rows=8191, cols=5120, block=1, dtype="bf16"),
        # expert master weights after an optimizer step, requantized for the next forward
        dict(name="quantize_expert_weights", op="quantize", batch=64, rows=2816, cols=2048, block=128, dtype="f32"),
        # a few token rows through one layer: bound by reading W once
        dict(name="forward_m16_4096", op="forward", M=16, N=4096, K=4096),
        # a ragged prompt: sizes that end inside every tile and scale block
        dict(name="forward_ragged_1000", op="forward", M=1000, N=2824, K=2064),
        # the FFN workload's forward, the largest product
        dict(name="forward_ffn", op="forward", M=8192, N=14336, K=5120),
        # its input gradient on the square workload
        dict(name="dgrad_4096", op="dgrad", M=4096, N=4096, K=4096),
        # 64 routed tokens over 64 experts: one decode step of a mixture layer
        dict(name="grouped_forward_decode", op="grouped_forward", E=64, S=64, N=2816, K=2048, skew=1.1, mix=3),
        # the mixture workload's prompt: Zipf routing with empty experts
        dict(name="grouped_forward_zipf", op="grouped_forward", E=64, S=16384, N=2816, K=2048, skew=1.1, mix=1),
        # the gradient through wide experts
        dict(name="grouped_dgrad_wide", op="grouped_dgrad", E=32, S=8192, N=2048, K=7168, skew=0.7, mix=2),
        # many tensors of all sizes (adapters, norms, biases), 32-bit states: launch count matters
        dict(name="adamw_many_small", op="adamw", count=300, low=1, high=200000, bits=32, grad="f32", mix=4),
        # whole layers, states in 8 bits, gradients as the wgrad writes them
        dict(name="adamw_layers_8bit", op="adamw", count=24, low=2000000, high=12000000, bits=8, grad="bf16", mix=5),
    ]


def _log(rng, low, high, step=1):
    return max(1, round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step


def draw(rng):
    op = rng.choice(["quantize", "forward", "dgrad", "grouped_forward", "grouped_dgrad", "adamw"])
    if op == "quantize":
        block, dtype = rng.choice([1, 128]), rng.choice(["bf16", "f32"])
        return dict(op=op, batch=_log(rng, 1, 16), rows=_log(rng, 1, 8192), cols=_log(rng, 128, 7168, 16), block=block, dtype=dtype)
    if op == "forward":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 128, 14336, 8), K=_log(rng, 128, 5120, 16))
    if op == "dgrad":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 128, 7168, 16), K=_log(rng, 128, 7168, 16))
    if op == "adamw":
        low = _log(rng, 1, 100000)
        return dict(op=op, count=_log(rng, 1, 200), low=low, high=low + _log(rng, 100, 1000000), bits=rng.choice([8, 32]),
                    grad=rng.choice(["bf16", "f32"]), mix=rng.randrange(1 << 20))
    return dict(op=op, E=_log(rng, 1, 64), S=_log(rng, 1, 16384), N=_log(rng, 128, 2816, 16), K=_log(rng, 128, 7168, 16),
                skew=round(rng.uniform(0.0, 1.2), 2), mix=rng.randrange(1 << 20))


def counts_of(case):
    """Rows of each expert: S draws from r^-skew over experts in a drawn order; every eighth expert gets none."""
    rng, E = random.Random(case["mix"]), case["E"]
    open_ = [e for e in range(E) if E < 8 or e % 8 != 3]
    rng.shuffle(open_)
    p = [(r + 1) ** -case["skew"] for r in range(len(open_))]
    got = [0] * E
    for e in rng.choices(open_, weights=p, k=case["S"]):
        got[e] += 1
    return got


def sizes_of(case):
    """Lengths of the tensors, spread over the logarithm of the range."""
    rng = random.Random(case["mix"])
    return [_log(rng, case["low"], case["high"]) for _ in range(case["count"])]


def work(case):
    op = case["op"]
    if op == "quantize":
        n, r = case["batch"] * case["rows"] * case["cols"], case["rows"] if case["block"] == 1 else -(-case["rows"] // B)
        scales = case["batch"] * r * -(-case["cols"] // B)
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + n + 4 * scales, "flops": 2 * n}
    if op == "adamw":
        n = sum(sizes_of(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / B
        return {"bytes": n * (8 + 2 + state + (2 if case["grad"] == "bf16" else 4)), "flops": 16 * n}
    N, K = case["N"], case["K"]
    rows = case["M"] if "M" in case else case["S"]
    experts = 1 if "M" in case else sum(c > 0 for c in counts_of(case))
    inner, outer = (K, N) if "forward" in op else (N, K)
    weight = experts * (N * K + 4 * -(-N // B) * -(-K // B))
    return {"bytes": rows * (inner + 4 * -(-inner // B) + 2 * outer) + weight, "flops": 2 * rows * N * K}


# ---------------------------------------------------------------- inputs
def _blocks(x, block):
    """x [b, r, c] as [b, r', block, c', B], zero-padded to whole blocks."""
    b, r, c = x.shape
    pr, pc = -r % block, -c % B
    if pr or pc:
        x = torch.nn.functional.pad(x, (0, pc, 0, pr))
    return x.view(b, (r + pr) // block, block, (c + pc) // B, B)


def _divided(a, b):
    return a / b if torch.is_tensor(b) else a / torch.full_like(a, b)


def plain_quantize(x, block):
    """(E4M3 values [b, r, c], float32 scales [b, r / block, c / B]) of x."""
    b, r, c = x.shape
    t = _blocks(x.float(), block)
    a = t.abs().amax(dim=(2, 4))
    a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
    scale = _divided(a, 448.0)
    q = t * _divided(torch.full_like(a, 448.0), a)[:, :, None, :, None]
    q = q.clamp(-448.0, 448.0).to(FP8).view(b, t.shape[1] * block, -1)[:, :r, :c]
    return q.contiguous(), scale


def _activations(shape, g):
    """N(0, 1) with a few loud channels, as activations have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 20.0, 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        shape = (case["batch"], case["rows"], case["cols"])
        x = _activations(shape, g) if case["block"] == 1 else torch.randn(shape, generator=g, device="cuda") * 0.02
        return dict(op=op, block=case["block"], x=x.to(torch.bfloat16) if case["dtype"] == "bf16" else x)
    if op == "adamw":
        return _prepare_adamw(case, seed, g)
    N, K, E = case["N"], case["K"], case.get("E", 1)
    rows = case["M"] if "M" in case else case["S"]
    x = _activations((1, rows, K if "forward" in op else N), g)
    codes, scale = plain_quantize(x, 1)
    w = [plain_quantize(torch.randn((1, N, K), generator=g, device="cuda") * 0.02, B) for _ in range(E)]
    wc, ws = torch.cat([c for c, _ in w]), torch.cat([s for _, s in w])
    state = dict(op=op, codes=codes[0].view(torch.uint8), scale=scale[0], N=N, K=K, E=E,
                 w=SimpleNamespace(fmt=1, data=wc.view(torch.uint8), scale=ws, tensor_scale=None, batch=E, rows=N, cols=K))
    if "S" in case:
        ends, at = [], 0
        for c in counts_of(case):
            at += c
            ends.append(at)
        state["ends"] = ends
        state["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    return state


def _prepare_adamw(case, seed, g):
    """One flat buffer each for parameters, gradients and states; every tensor starts at a multiple of B."""
    sizes = sizes_of(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // B) * B
    blocks = total // B
    tensor_of_block = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"),
                                              torch.tensor([-(-n // B) for n in sizes], device="cuda"))
    at = torch.arange(total, device="cuda")
    ends = torch.tensor([s + n for s, n in zip(starts, sizes)], device="cuda")
    real = (at < ends[tensor_of_block].repeat_interleave(B)).float()
    draw_ = lambda std: torch.randn(total, generator=g, device="cuda") * std * real  # noqa: E731
    s = dict(op="adamw", bits=case["bits"], step=9, seed=seed & 0xFFFFFFFF, p=draw_(0.02),
             grad=draw_(1e-3) * torch.exp(2 * torch.randn(blocks, generator=g, device="cuda")).repeat_interleave(B),
             copy=torch.zeros(total, dtype=torch.bfloat16, device="cuda"),
             grad_scale=torch.full((1,), 0.5, device="cuda"),
             wd=torch.tensor([0.1 if n > 4096 else 0.0 for n in sizes], device="cuda")[tensor_of_block])
    s["copy"].copy_(s["p"])
    if case["grad"] == "bf16":
        s["grad"] = s["grad"].to(torch.bfloat16)
    m, v = draw_(3e-4), draw_(1e-3).square() + 1e-9 * real
    if case["bits"] == 32:
        s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
    else:
        (s["m"], s["ms"]), (s["v"], s["vs"]) = _state_codes(m), _state_codes(v.sqrt())
    if own:
        from block_scaled_gemm_fp8_gb300 import bsq
        cut = lambda t: [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
        scales = lambda t: None if t is None else [t[a // B:a // B + -(-n // B)] for a, n in zip(starts, sizes)]  # noqa: E731
        s["table"] = bsq.adamw_table(cut(s["p"]), cut(s["grad"]), cut(s["m"]), cut(s["v"]), scales(s["ms"]), scales(s["vs"]),
                                     copies=cut(s["copy"]), weight_decay=[0.1 if n > 4096 else 0.0 for n in sizes])
    return s


def _state_codes(x):
    t = x.view(-1, B)
    a = t.abs().amax(dim=1)
    a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
    q = (t * _divided(torch.full_like(a, 448.0), a)[:, None]).clamp(-448.0, 448.0)
    return q.to(FP8).view(-1).view(torch.uint8), _divided(a, 448.0)


# ---------------------------------------------------------------- plain forms
def _weights(state):
    """W in float32 [E, N, K]: the codes' values times their block's scale."""
    w = state["w"]
    s = w.scale.repeat_interleave(B, 1)[:, :w.rows].repeat_interleave(B, 2)[:, :, :w.cols]
    return w.data.view(FP8).float() * s


def plain_product(state):
    x = state["codes"].view(FP8).float()
    x = x * state["scale"].repeat_interleave(B, 1)[:, :x.shape[1]]
    w = _weights(state)
    if "forward" in state["op"]:
        w = w.transpose(1, 2)
    if "ends" not in state:
        return (x @ w[0]).to(torch.bfloat16)
    # the experts' row counts differ: one product for each, on its own rows
    y = torch.empty((x.shape[0], w.shape[2]), dtype=torch.bfloat16, device=x.device)
    r0 = 0
    for e, r1 in enumerate(state["ends"]):
        if r1 > r0:
            y[r0:r1] = (x[r0:r1] @ w[e]).to(torch.bfloat16)
        r0 = r1
    return y


def _random_bits(n, seed, step):
    """(low, high) 16 bits of a 32-bit hash of each element's place: Weyl step, then MurmurHash3's finalizer (Appleby)."""
    mask = 0xFFFFFFFF
    x = (torch.arange(n, device="cuda") * 0x9E3779B1 + ((seed + step * 0x7F4A7C15) & mask)) & mask
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & mask
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & mask
    x = x ^ (x >> 16)
    return x & 0xFFFF, x >> 16


def _round_at_random(a, bits):
    """E4M3 magnitude of a in [0, 448.0001]: the next one below or above, the latter with the probability of the rest."""
    big = ((a.view(torch.int32).to(torch.int64) + (bits << 4)) & ~0xFFFFF).to(torch.int32).view(torch.float32)
    small = torch.floor(a * 512.0 + bits.float() * 2.0 ** -16) * 2.0 ** -9
    return torch.where(a >= 2.0 ** -6, big, small).clamp(max=448.0)


def _store(x, bits, keep):
    t = x.view(-1, B)
    a = t.abs().amax(dim=1)
    a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
    q = (t * _divided(torch.full_like(a, 448.0), a)[:, None]).view(-1)
    r = _round_at_random(q.abs(), bits)
    if keep:
        r = torch.where((q > 0) & (r == 0), torch.full_like(r, 2.0 ** -9), r)
    return torch.copysign(r, q).to(FP8).view(torch.uint8), _divided(a, 448.0)


def plain_adamw(s):
    s["step"] += 1
    t, (b1, b2) = s["step"], BETAS
    c1, c2 = LR / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
    g = s["grad"].float() * s["grad_scale"]
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        value = lambda c, k: (s[c].view(FP8).float().view(-1, B) * s[k][:, None]).view(-1)  # noqa: E731
        m, v = value("m", "ms"), value("v", "vs").square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = v.sqrt()
    p = (s["p"].view(-1, B) * (1 - LR * s["wd"].double()).float()[:, None]).view(-1) - (m * c1) / (r * c2 + EPS)
    s["p"].copy_(p)
    s["copy"].copy_(p)
    if s["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        low, high = _random_bits(p.numel(), s["seed"], t)
        for (codes, scale), c, k in ((_store(m, low, False), "m", "ms"), (_store(r, high, True), "v", "vs")):
            s[c].copy_(codes)
            s[k].copy_(scale)


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if own:
        from block_scaled_gemm_fp8_gb300 import bsq
    if op == "quantize":
        if not own:
            return plain_quantize(state["x"], state["block"])
        codes, scale = bsq.quantize_e4m3(state["x"], block_rows=state["block"])
        return codes.view(FP8), scale
    if op == "adamw":
        if own:
            state["step"] += 1
            bsq.adamw(state["table"], step=state["step"], lr=LR, betas=BETAS, eps=EPS, grad_scale=state["grad_scale"], seed=state["seed"])
        else:
            plain_adamw(state)
        out = dict(p=state["p"], copy=state["copy"])
        if state["bits"] == 32:
            return dict(out, m=state["m"], v=state["v"])
        return dict(out, m=state["m"].view(FP8), v=state["v"].view(FP8), ms=state["ms"], vs=state["vs"])
    if not own:
        return plain_product(state)
    if "ends" not in state:
        return getattr(bsq, "fp8_" + op)(state["codes"], state["scale"], state["w"])
    return getattr(bsq, "fp8_" + op)(state["codes"], state["scale"], state["w"], state["offsets"])


# ---------------------------------------------------------------- 64 bits
def _scale64(a):
    return torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100)) / 448.0


def _grid(a):
    """Distance of E4M3 magnitudes at a."""
    return torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        b, r, c = s["x"].shape
        t = s["x"].double()
        # blocks by index, one flat segment each
        rows = torch.arange(r, device="cuda") // s["block"]
        nr, nc = -(-r // s["block"]), -(-c // B)
        seg = (rows[:, None] * nc + (torch.arange(c, device="cuda") // B)[None, :]).reshape(1, -1).expand(b, -1)
        a = torch.zeros((b, nr * nc), dtype=torch.float64, device="cuda").scatter_reduce(1, seg, t.abs().reshape(b, -1), "amax")
        scale = _scale64(a)
        q = t / scale.gather(1, seg).view(b, r, c)
        u = _grid(q.abs())
        return (torch.round(q / u) * u).clamp(-448.0, 448.0), scale.view(b, nr, nc)
    if op == "adamw":
        t, (b1, b2) = s["step"] + 1, BETAS
        f = lambda c, k: s[c].view(FP8).double() * s[k].double().repeat_interleave(B)  # noqa: E731
        m, r = (s["m"].double(), s["v"].double().sqrt()) if s["bits"] == 32 else (f("m", "ms"), f("v", "vs"))
        g = s["grad"].double() * s["grad_scale"].double()
        m = b1 * m + (1 - b1) * g
        v = b2 * r ** 2 + (1 - b2) * g ** 2
        p = s["p"].double() * (1 - LR * s["wd"].double().repeat_interleave(B))
        p = p - LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
        out = dict(p=p, copy=p)
        if s["bits"] == 32:
            return dict(out, m=m, v=v)
        # the codes are drawn by the random numbers: their scales alone have a value of their own
        top = lambda x: _scale64(x.abs().view(-1, B).amax(1))  # noqa: E731
        return dict(out, m=None, v=None, ms=top(m), vs=top(v.sqrt()))
    # products: integer multiples of powers of two, summed in 64 bits
    x = s["codes"].view(FP8).double() * s["scale"].double().repeat_interleave(B, 1)[:, :s["codes"].shape[1]]
    n, k = torch.arange(s["N"], device="cuda") // B, torch.arange(s["K"], device="cuda") // B
    y = torch.zeros((x.shape[0], s["N"] if "forward" in op else s["K"]), dtype=torch.float64, device="cuda")
    r0 = 0
    for e, r1 in enumerate(s.get("ends", [x.shape[0]])):
        if r1 > r0:
            w = s["w"].data[e].view(FP8).double() * s["w"].scale[e].double()[n][:, k]
            y[r0:r1] = x[r0:r1] @ (w.T if "forward" in op else w)
        r0 = r1
    return y
