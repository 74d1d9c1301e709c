"""Timed cases of the operators around a mixture layer's products: the router with its gradient,
tokens sorted by expert and sent to their experts' rows (BF16 or block-scaled E4M3), the rows
combined back with weights, both with their gradients, and products of a few BF16 token rows
with 4-bit weights, dense and per expert.

``own`` selects who computes: False, elementary torch operations in float32 (`plain_*`);
True, the framework's entry points.  The definitions, with T tokens, k slots each, B = 128:

  route     score = logit (+ bias); the k experts of the highest score, ties to the lowest
            index; weight = f softmax(logits)[chosen], renormalized: f softmax(chosen logits);
            or f sigmoid(logit), renormalized: divided by its sum over the chosen
  sort      rows[t, j] = place of slot (t, j) when slots are sorted by expert, stable; -1 where
            the id is no expert's; offsets = cumulative ends; slots = the inverse, -1 behind it
  dispatch  out[rows[t, j]] = w[t, j] x[t]; E4M3: the codes of x[t] in blocks of B columns
            (a = max |x|, scale = a / 448, code = E4M3(x * (448 / a))), scale times w[t, j]
  combine   out[t] = sum_j w[t, j] y[rows[t, j]]; gradients: w[t, j] g[t] to the row (as
            dispatch does) and g[t] . y[rows[t, j]] to the weight
  fp4       y = x deq(W)^T, deq = bf16(code * bf16(scale)): MXFP4 scale 2^(e - 127) per 32
            elements, NVFP4 scale float32(E4M3 * tensor scale) per 16; per expert as grouped
"""

import math
import random
from types import SimpleNamespace

import torch

own = False

B = 128
FP8 = torch.float8_e4m3fn
MXFP4, NVFP4 = 2, 3
FACTOR = 2.5


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the gate of one decode batch: nothing but latency
        dict(name="route_decode", op="route", T=16, E=64, k=4, dtype="bf16", gate="softmax", renorm=True, bias=False, train=False),
        # the gate over a training batch, with its gradient; scores carry a balancing bias
        dict(name="route_train", op="route", T=16384, E=128, k=8, dtype="f32", gate="softmax", renorm=False, bias=True, train=True),
        # one decode batch to its experts' FP8 rows
        dict(name="dispatch_decode", op="dispatch", T=16, K=2048, E=64, k=4, pad=0, bf16=False, e4m3=True, weighted=False, train=False),
        # a training batch: FP8 rows for the product, BF16 rows for the weight gradient, and the gradient of the tokens
        dict(name="dispatch_train", op="dispatch", T=4096, K=2048, E=64, k=4, pad=0, bf16=True, e4m3=True, weighted=False, train=True),
        # a padded prompt of wide tokens, odd count
        dict(name="dispatch_wide_padded", op="dispatch", T=8191, K=7168, E=128, k=4, pad=500, bf16=False, e4m3=True, weighted=False, train=False),
        # the decode batch's rows back to their tokens
        dict(name="combine_decode", op="combine", T=16, N=2816, E=64, k=4, pad=0, weighted=True, train=False, bf16=False, e4m3=False),
        # a training batch's rows back, and the gradients of rows (both types) and weights
        dict(name="combine_train", op="combine", T=4096, N=2816, E=64, k=4, pad=0, weighted=True, train=True, bf16=True, e4m3=True),
        # the largest: eight wide rows a token, odd count
        dict(name="combine_wide", op="combine", T=8191, N=7168, E=128, k=8, pad=0, weighted=True, train=False, bf16=False, e4m3=False),
        # one token through one layer: bound by reading W once
        dict(name="fp4_token", op="fp4", M=1, N=4096, K=4096, fmt=MXFP4),
        # a decode batch, odd count, through the wide layer
        dict(name="fp4_batch_wide", op="fp4", M=13, N=14336, K=5120, fmt=NVFP4),
        # 64 routed rows over 128 wide experts: one decode step of a mixture layer
        dict(name="fp4_experts_decode", op="fp4", E=128, S=64, N=2048, K=7168, fmt=MXFP4, skew=0.7, mix=2),
        # a larger batch: every expert several rows
        dict(name="fp4_experts_batch", op="fp4", E=64, S=509, N=2816, K=2048, fmt=NVFP4, skew=0.7, mix=3),
    ]


def _log(rng, low, high, step=1):
    return max(1, round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "fp4", "fp4_experts"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "route":
        E, gate = _log(rng, 2, 512), rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=rng.randint(1, min(8, E)), dtype=rng.choice(["bf16", "f32"]), gate=gate,
                    renorm=flip(), bias=gate == "softmax" and flip(), train=flip())
    if op in ("dispatch", "combine"):
        T, k, train = _log(rng, 1, 8191), rng.randint(1, 8), flip()
        types = rng.choice([(True, False), (False, True), (True, True)]) if train or op == "dispatch" else (False, False)
        d = dict(op=op, T=T, E=_log(rng, 1, 256), k=k, pad=rng.choice([0, T // 10]), weighted=flip(), train=train, bf16=types[0], e4m3=types[1])
        d["K" if op == "dispatch" else "N"] = _log(rng, 128, 7168 if T * k <= 32768 else 2816, 16)
        return d
    if op == "fp4":
        return dict(op=op, M=_log(rng, 1, 64), N=_log(rng, 128, 14336, 8), K=_log(rng, 128, 7168, 32), fmt=rng.choice([MXFP4, NVFP4]))
    return dict(op="fp4", E=_log(rng, 1, 128), S=_log(rng, 1, 512), N=_log(rng, 128, 2816, 8), K=_log(rng, 128, 5120, 32),
                fmt=rng.choice([MXFP4, NVFP4]), skew=round(rng.uniform(0.0, 1.2), 2), mix=rng.randrange(1 << 20))


def ends_of(case):
    """Cumulative ends of the experts' rows: S draws from r^-skew over experts in a drawn order."""
    rng, E = random.Random(case["mix"]), case["E"]
    order = list(range(E))
    rng.shuffle(order)
    got = [0] * E
    for e in rng.choices(order, weights=[(r + 1) ** -case["skew"] for r in range(E)], k=case["S"]):
        got[e] += 1
    ends, at = [], 0
    for c in got:
        at += c
        ends.append(at)
    return ends


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, s = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * s + 8 * T * k + 4 * E * case["bias"] + case["train"] * (T * E * s + 4 * T * k), "flops": 5 * T * E}
    if op == "fp4":
        N, K, rows = case["N"], case["K"], case["M"] if "M" in case else case["S"]
        ends = ends_of(case) if "S" in case else [rows]
        experts = sum(b > a for a, b in zip([0] + ends, ends))
        weight = experts * (N * K // 2 + N * K // (32 if case["fmt"] == MXFP4 else 16))
        return {"bytes": weight + 2 * rows * (K + N), "flops": 2 * rows * N * K}
    T, k = case["T"], case["k"]
    slots, rows = T * k, (T - case["pad"]) * k
    wide = case["K"] if op == "dispatch" else case["N"]
    row = wide * (2 * case["bf16"] + case["e4m3"]) + 4 * -(-wide // B) * case["e4m3"]
    if op == "dispatch":
        n = 12 * slots + 4 * case["E"] + 2 * T * wide + 4 * slots * case["weighted"] + rows * row
        if case["train"]:
            n += 2 * rows * wide + 2 * T * wide + 4 * slots * case["weighted"]
        return {"bytes": n, "flops": rows * wide * (1 + 2 * case["train"])}
    n = 4 * slots * (1 + case["weighted"]) + 2 * rows * wide + 2 * T * wide
    if case["train"]:
        n += 2 * T * wide + rows * row + 4 * slots
    return {"bytes": n, "flops": 2 * rows * wide * (1 + 2 * case["train"])}


# ---------------------------------------------------------------- inputs
def _activations(shape, g):
    """N(0, 1) with a few loud channels, as activations have them."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 20.0, 1.0)


def _choices(T, E, k, pad, g):
    """int32 [T, k]: distinct experts of a skewed popularity where there are k of them; -1 for the last `pad` tokens."""
    like = torch.randn(E, generator=g, device="cuda")
    noise = torch.rand((T, E), generator=g, device="cuda").clamp(min=1e-9)
    ids = (like - (-noise.log()).log()).argsort(dim=1, descending=True)[:, :k].to(torch.int32)
    if k > E:
        ids = ids.repeat(1, -(-k // E))[:, :k]
    if pad:
        ids[T - pad:] = -1
    return ids.contiguous()


def _weights(T, k, g):
    w = torch.rand((T, k), generator=g, device="cuda") + 0.05
    return (w / w.sum(dim=1, keepdim=True)).contiguous()


# halves between neighbouring magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 of E2M1
_E2M1_HALVES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _encode_fp4(w, fmt):
    """(packed codes [N, K / 2], scale bytes, tensor scale or None) of w [N, K]."""
    n, k = w.shape
    t = w.view(n, -1, 32 if fmt == MXFP4 else 16)
    a = t.abs().amax(dim=2)
    top = None
    if fmt == MXFP4:
        e = torch.ceil(torch.log2(a / 6)).clamp(-126, 126)
        scale, value = (e + 127).to(torch.uint8), torch.exp2(e)
    else:
        top = w.abs().amax() / (6 * 448)
        code = (a / (6 * top)).clamp(max=448).to(FP8)
        scale, value = code.view(torch.uint8), code.float() * top
    q = (t / value.clamp(min=1e-30)[:, :, None]).view(n, k)
    code = torch.bucketize(q.abs(), torch.tensor(_E2M1_HALVES, device="cuda"), out_int32=True) + 8 * (q < 0)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale, top


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["bias_"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["grad"] = 1e-2 * torch.randn((T, k), generator=g, device="cuda")
        return s
    if op == "fp4":
        N, K, E = case["N"], case["K"], case.get("E", 1)
        rows = case["M"] if "M" in case else case["S"]
        s["x"] = _activations((rows, K), g).to(torch.bfloat16)
        w = [_encode_fp4(torch.randn((N, K), generator=g, device="cuda") * 0.02, case["fmt"]) for _ in range(E)]
        top = torch.stack([t for _, _, t in w]) if case["fmt"] == NVFP4 else None
        s["w"] = SimpleNamespace(fmt=case["fmt"], data=torch.stack([c for c, _, _ in w]), scale=torch.stack([c for _, c, _ in w]),
                                 tensor_scale=top, batch=E, rows=N, cols=K)
        if "S" in case:
            s["ends"] = ends_of(case)
            s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device="cuda")
        return s
    T, E, k = case["T"], case["E"], case["k"]
    S, wide = T * k, case["K"] if op == "dispatch" else case["N"]
    s["ids"] = _choices(T, E, k, case["pad"], g)
    s["weights"] = _weights(T, k, g) if case["weighted"] else None
    if op == "dispatch":
        s["x"] = _activations((T, wide), g).to(torch.bfloat16)
        if case["train"]:
            s["grad"] = (1e-2 * torch.randn((S, wide), generator=g, device="cuda")).to(torch.bfloat16)
    else:
        s["y"] = torch.randn((S, wide), generator=g, device="cuda").to(torch.bfloat16)
        s["rows"] = plain_sort(s["ids"], E)[1]
        if case["train"]:
            s["grad"] = (1e-2 * torch.randn((T, wide), generator=g, device="cuda")).to(torch.bfloat16)
    # rows of a padded batch: the program's own buffers, of which the last are left as they are
    s["out"] = torch.zeros((S, wide), dtype=torch.bfloat16, device="cuda") if case["bf16"] and case["pad"] else None
    s["codes"] = torch.zeros((S, wide), dtype=torch.uint8, device="cuda") if case["e4m3"] and case["pad"] else None
    s["scale"] = torch.zeros((S, -(-wide // B)), device="cuda") if case["e4m3"] and case["pad"] else None
    return s


# ---------------------------------------------------------------- plain forms
def plain_route(s):
    x = s["logits"].float()
    score = x if s["bias_"] is None else x + s["bias_"]
    ids = score.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    chosen = x.gather(1, ids)
    soft = s["gate"] == "softmax"
    over = x if soft and not s["renorm"] else chosen          # what the softmax runs over
    if soft:
        p = (over - over.amax(dim=1, keepdim=True)).exp()
        p = p / p.sum(dim=1, keepdim=True)
        v = p if s["renorm"] else p.gather(1, ids)
    else:
        p = 1 / (1 + (-chosen).exp())
        total = p.sum(dim=1, keepdim=True) if s["renorm"] else torch.ones_like(p[:, :1])
        v = p / total
    out = dict(ids=ids.to(torch.int32), weights=FACTOR * v)
    if s["train"]:
        g = FACTOR * s["grad"]
        mean = (g * v).sum(dim=1, keepdim=True)
        if soft and not s["renorm"]:
            full = (-p * mean).scatter_add(1, ids, g * v)
        else:
            d = v * (g - mean) if soft else (g - mean if s["renorm"] else g) / total * p * (1 - p)
            full = torch.zeros_like(x).scatter(1, ids, d)
        out["grad_logits"] = full.to(s["logits"].dtype)
    return out


def plain_sort(ids, E):
    """(offsets, rows, slots) of int32 ids [T, k]."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    ordered, order = key.sort(stable=True)
    n = torch.arange(flat.numel(), device="cuda")
    rows = torch.empty_like(n).scatter(0, order, n)
    ends = torch.searchsorted(ordered, torch.arange(E, device="cuda"), right=True)
    rows = torch.where(key < E, rows, torch.full_like(rows, -1)).view(ids.shape)
    slots = torch.where(ordered < E, order, torch.full_like(order, -1))
    return ends.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32)


def plain_codes(x):
    """(E4M3 values [r, c], float32 scales [r, c / B]) of x [r, c]."""
    r, c = x.shape
    t = torch.nn.functional.pad(x.float(), (0, -c % B)).view(r, -1, B)
    a = t.abs().amax(dim=2)
    a = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100))
    top = torch.full_like(a, 448.0)
    q = (t * (top / a)[:, :, None]).clamp(-448.0, 448.0).to(FP8)
    return q.view(r, -1)[:, :c], a / top


def plain_scatter(x, rows, weights, s):
    """Rows [S, c] of tokens x [T, c] in the types that the case asks for."""
    T, k = rows.shape
    flat = rows.reshape(-1).long()
    held = flat >= 0
    if s["pad"]:
        to, token = flat[held], torch.arange(T, device="cuda").repeat_interleave(k)[held]
        w = None if weights is None else weights.reshape(-1)[held]
    else:
        to, token, w = flat, torch.arange(T, device="cuda").repeat_interleave(k), None if weights is None else weights.reshape(-1)
    out = {}
    if s["bf16"]:
        out["out"] = s["out"] if s["out"] is not None else torch.empty((T * k, x.shape[1]), dtype=torch.bfloat16, device="cuda")
        v = x.float()[token]
        out["out"][to] = (v if w is None else v * w[:, None]).to(torch.bfloat16)
    if s["e4m3"]:
        codes, scale = plain_codes(x)
        out["codes"] = s["codes"] if s["codes"] is not None else torch.empty((T * k, x.shape[1]), dtype=torch.uint8, device="cuda")
        out["scale"] = s["scale"] if s["scale"] is not None else torch.empty((T * k, scale.shape[1]), device="cuda")
        out["codes"][to] = codes.contiguous().view(torch.uint8)[token]
        out["scale"][to] = scale[token] if w is None else scale[token] * w[:, None]
    return out


def plain_gather(y, rows, weights):
    """sum_j w[t, j] y[rows[t, j]], and the rows [T, k, c] in float32 (zero where there is none)."""
    v = y[rows.long().clamp(min=0)].float() * (rows >= 0)[:, :, None]
    return (v if weights is None else v * weights[:, :, None]).sum(dim=1).to(torch.bfloat16), v


def plain_dispatch(s):
    offsets, rows, slots = plain_sort(s["ids"], s["E"])
    out = dict(plain_scatter(s["x"], rows, s["weights"], s), offsets=offsets, rows=rows, slots=slots)
    if s["train"]:
        out["grad_x"], v = plain_gather(s["grad"], rows, s["weights"])
        if s["weighted"]:
            out["grad_weights"] = (v * s["x"].float()[:, None, :]).sum(dim=2)
    return out


def plain_combine(s):
    out = {}
    out["y"], v = plain_gather(s["y"], s["rows"], s["weights"])
    if s["train"]:
        out.update(plain_scatter(s["grad"], s["rows"], s["weights"], s))
        out["grad_weights"] = (v * s["grad"].float()[:, None, :]).sum(dim=2)
    return out


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decoded(w, which):
    """The values of W's experts `which`, float32 [len, N, K]."""
    one = torch.tensor(_E2M1, device="cuda")
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], dim=1)
    codes = pair[w.data[which].int()].view(len(which), w.rows, w.cols)
    if w.fmt == MXFP4:
        scale = torch.exp2(w.scale[which].float() - 127)
    else:
        scale = w.scale[which].view(FP8).float() * w.tensor_scale[which][:, None, None]
    scale = scale.to(torch.bfloat16).float()
    return (codes.view(*scale.shape, -1) * scale[..., None]).to(torch.bfloat16).float().view(len(which), w.rows, w.cols)


def plain_fp4(s):
    x = s["x"].float()
    if "ends" not in s:
        return (x @ _decoded(s["w"], [0])[0].T).to(torch.bfloat16)
    # the routed experts' rows, padded to the longest
    counts = [b - a for a, b in zip([0] + s["ends"], s["ends"])]
    which = [e for e, c in enumerate(counts) if c]
    size = torch.tensor([counts[e] for e in which], device="cuda")
    expert = torch.arange(len(which), device="cuda").repeat_interleave(size, output_size=len(x))
    place = torch.arange(len(x), device="cuda") - (size.cumsum(0) - size)[expert]
    padded = torch.zeros((len(which), max(counts), x.shape[1]), device="cuda")
    padded[expert, place] = x
    return (padded @ _decoded(s["w"], which).transpose(1, 2))[expert, place].to(torch.bfloat16)


# ---------------------------------------------------------------- one pass
def own_run(s):
    from block_scaled_gemm_fp8_gb300 import bsq
    op = s["op"]
    if op == "route":
        how = dict(gate=s["gate"], renormalize=s["renorm"], factor=FACTOR)
        ids, weights = bsq.route(s["logits"], s["k"], bias=s["bias_"], **how)
        out = dict(ids=ids, weights=weights)
        if s["train"]:
            out["grad_logits"] = bsq.route_backward(s["logits"], ids, s["grad"], **how)
        return out
    if op == "fp4":
        return bsq.fp4_grouped_forward(s["x"], s["w"], s["offsets"]) if "ends" in s else bsq.fp4_forward(s["x"], s["w"])
    types, given = dict(bf16=s["bf16"], e4m3=s["e4m3"]), dict(codes=s["codes"], scale=s["scale"])
    named = lambda rows, codes, scale: {n: t for n, t in (("out", rows), ("codes", codes), ("scale", scale)) if t is not None}  # noqa: E731
    if op == "dispatch":
        offsets, rows, slots = bsq.sort_experts(s["ids"], s["E"])
        out = dict(named(*bsq.dispatch(s["x"], rows, s["weights"], out=s["out"], **types, **given)), offsets=offsets, rows=rows, slots=slots)
        if s["train"]:
            out["grad_x"] = bsq.combine(s["grad"], rows, s["weights"])
            if s["weighted"]:
                out["grad_weights"] = bsq.combine_backward(s["x"], s["grad"], rows, s["weights"], bf16=False)[3]
        return out
    out = dict(y=bsq.combine(s["y"], s["rows"], s["weights"]))
    if s["train"]:
        rows, codes, scale, out["grad_weights"] = bsq.combine_backward(s["grad"], s["y"], s["rows"], s["weights"], grad_y=s["out"], **types, **given)
        out.update(named(rows, codes, scale))
    return out


def run(state):
    if own:
        out = own_run(state)
    else:
        out = {"route": plain_route, "dispatch": plain_dispatch, "combine": plain_combine, "fp4": plain_fp4}[state["op"]](state)
    if isinstance(out, dict) and "codes" in out:
        out["codes"] = out["codes"].view(FP8)
    return out


# ---------------------------------------------------------------- 64 bits
def _codes64(x):
    """E4M3 values and scales of float64 x [r, c]: blocks by index, values on the grid of their magnitude."""
    r, c = x.shape
    nb = -(-c // B)
    block = (torch.arange(c, device="cuda") // B)[None, :].expand(r, -1)
    a = torch.zeros((r, nb), dtype=torch.float64, device="cuda").scatter_reduce(1, block, x.abs(), "amax")
    scale = torch.where(a == 0, torch.full_like(a, 448.0), a.clamp(min=2.0 ** -100)) / 448.0
    q = x / scale.gather(1, block)
    u = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / u) * u).clamp(-448.0, 448.0), scale


def _rows64(x, rows, weights, case):
    """What each row holds, taken row by row from the slot that owns it."""
    T, k = rows.shape
    flat = rows.reshape(-1).long()
    slot = torch.full((T * k + 1,), -1, device="cuda")
    slot[flat] = torch.arange(T * k, device="cuda")          # rows of -1 write to the spare last place
    slot = slot[:-1]
    have = (slot >= 0).double()[:, None]
    token = slot.clamp(min=0) // k
    w = have if weights is None else weights.double().reshape(-1)[slot.clamp(min=0)][:, None] * have
    out = {}
    if case["bf16"]:
        out["out"] = x[token] * w
    if case["e4m3"]:
        codes, scale = _codes64(x)
        out["codes"], out["scale"] = codes[token] * have, scale[token] * w
    return out


def _sums64(y, rows, weights):
    """sum_j w[t, j] y[rows[t, j]], slot by slot."""
    total = 0.0
    for j in range(rows.shape[1]):
        r = rows[:, j].long()
        w = (r >= 0).double() if weights is None else weights[:, j].double() * (r >= 0)
        total = total + y[r.clamp(min=0)].double() * w[:, None]
    return total


def _dots64(g, y, rows):
    return torch.stack([(g * y[r.long().clamp(min=0)].double()).sum(dim=1) * (r >= 0) for r in rows.unbind(1)], dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        x = s["logits"].double()
        score = x.float() if s["bias_"] is None else (x + s["bias_"].double()).float()   # the choice is of float32 scores
        ids = _topk64(score, s["k"])
        mask = torch.zeros_like(x).scatter(1, ids, 1.0)
        if s["gate"] == "softmax":
            over = x.masked_fill(mask == 0, -math.inf) if s["renorm"] else x
            p = torch.softmax(over, dim=1)
        else:
            p = torch.sigmoid(x) * mask
            if s["renorm"]:
                p = p / p.sum(dim=1, keepdim=True)
        out = dict(ids=ids.to(torch.int32), weights=FACTOR * p.gather(1, ids))
        if s["train"]:
            g = torch.zeros_like(x).scatter(1, ids, FACTOR * s["grad"].double())
            if s["gate"] == "softmax":
                out["grad_logits"] = p * (g - (p * g).sum(dim=1, keepdim=True))
            elif s["renorm"]:
                out["grad_logits"] = p * (1 - torch.sigmoid(x)) * (g - (p * g).sum(dim=1, keepdim=True))
            else:
                out["grad_logits"] = g * p * (1 - p)
        return out
    if op == "fp4":
        w, x = s["w"], s["x"].double()
        y = torch.zeros((len(x), w.rows), dtype=torch.float64, device="cuda")
        value = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
        group = torch.arange(w.cols, device="cuda") // (32 if w.fmt == MXFP4 else 16)
        r0 = 0
        for e, r1 in enumerate(s.get("ends", [len(x)])):
            if r1 > r0:
                code = torch.empty((w.rows, w.cols), dtype=torch.long, device="cuda")
                code[:, 0::2], code[:, 1::2] = (w.data[e] & 15).long(), (w.data[e] >> 4).long()
                if w.fmt == MXFP4:
                    scale = torch.pow(2.0, w.scale[e].double() - 127)
                else:
                    scale = (w.scale[e].view(FP8).double() * w.tensor_scale[e].double()).float().to(torch.bfloat16).double()
                v = value[code & 7] * (1 - 2 * (code >> 3)) * scale[:, group]
                y[r0:r1] = x[r0:r1] @ v.to(torch.bfloat16).double().T
            r0 = r1
        return y
    if op == "dispatch":
        offsets, rows, slots = plain_sort(s["ids"], s["E"])
        out = dict(_rows64(s["x"].double(), rows, s["weights"], case), offsets=offsets, rows=rows, slots=slots)
        if s["train"]:
            out["grad_x"] = _sums64(s["grad"], rows, s["weights"])
            if s["weighted"]:
                out["grad_weights"] = _dots64(s["x"].double(), s["grad"], rows)
        return out
    out = dict(y=_sums64(s["y"], s["rows"], s["weights"]))
    if s["train"]:
        g = s["grad"].double()
        out.update(_rows64(g, s["rows"], s["weights"], case))
        out["grad_weights"] = _dots64(g, s["y"], s["rows"])
    return out


def _topk64(score, k):
    """The k best of each row, one after the other; argmax of equal values is not defined, so the lowest index is taken."""
    at = torch.arange(score.shape[1], device="cuda")
    left, got = score.clone(), []
    for _ in range(k):
        best = left == left.amax(dim=1, keepdim=True)
        e = torch.where(best, at, torch.full_like(at, score.shape[1])).amin(dim=1, keepdim=True)
        got.append(e)
        left = left.scatter(1, e, -math.inf)
    return torch.cat(got, dim=1)
