"""The memory behind AdamwTable: a parameter or copy that was given other memory is refused before
anything is launched, and the memory of what is not looked at is held.  On the CPU, with tensors
that call themselves CUDA ones."""

import pytest
import torch

from block_scaled_gemm_fp8_gb300 import bsq
from tests.test_binding_devices import library, operand  # noqa: F401

NAMES = ["params", "grads", "ms", "vs", "m_scales", "v_scales", "copies"]


def tensors(count, bits=8):
    one = {"grads": torch.bfloat16, "copies": torch.bfloat16, **(dict(ms=torch.uint8, vs=torch.uint8) if bits == 8 else {})}
    names = [n for n in NAMES if bits == 8 or not n.endswith("_scales")]
    return {n: [operand(0, 2 if n.endswith("_scales") else 200, dtype=one.get(n, torch.float32)) for _ in range(count)] for n in names}


def step(table, at=1):
    bsq.adamw(table, at, 1e-3)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("name", ["params", "copies"])
@pytest.mark.parametrize("i", [0, 2])
def test_other_memory_is_refused(library, bits, name, i):  # noqa: F811
    t = tensors(3, bits)
    table = bsq.adamw_table(**t)
    step(table)
    old = t[name][i].data
    t[name][i].data = torch.zeros_like(old)
    with pytest.raises(ValueError, match=rf"{name}\[{i}\]"):
        step(table, 2)
    assert library.calls == ["bsq_adamw"]
    t[name][i].data = old
    step(table, 2)
    assert library.calls == ["bsq_adamw"] * 2
    t[name][i].untyped_storage().resize_(0)
    with pytest.raises(ValueError, match=rf"{name}\[{i}\]"):
        step(table, 3)
    assert library.calls == ["bsq_adamw"] * 2


@pytest.mark.parametrize("bits", [8, 32])
def test_memory_is_held(library, bits):  # noqa: F811
    """The caller's lists may be emptied, its gradients and states may be given other memory."""
    t = tensors(2, bits)
    table = bsq.adamw_table(**t)
    fields = {"grads": "grad", "ms": "m", "vs": "v", "m_scales": "m_scale", "v_scales": "v_scale"}
    for name, field in fields.items():
        if name not in t:
            continue
        for i, x in enumerate(t[name]):
            x.data = torch.zeros_like(x.data)
            held = [h for h in table.held if h.data_ptr() == getattr(table.items[i], field)]
            assert len(held) == 1 and held[0].nbytes() > 0, (name, i)
    for seq in t.values():
        seq.clear()
    step(table)
    assert library.calls == ["bsq_adamw"]
    assert [p.data_ptr() for p in table.keep["params"]] == [e.param for e in table.items]


def test_empty_tensors_and_tables(library):  # noqa: F811
    bsq.adamw(bsq.adamw_table([], [], [], []), 1, 1e-3)
    empty = [operand(0, 0) for _ in range(4)]
    step(bsq.adamw_table(*([t] for t in empty)))
    assert library.calls == ["bsq_adamw"]


def test_without_torchs_comparison(library, monkeypatch):  # noqa: F811
    monkeypatch.setattr(bsq, "_at_addresses", lambda tensors, addresses, which: all(tensors[i].data_ptr() == addresses[i] for i in which))
    t = tensors(2)
    table = bsq.adamw_table(**t)
    step(table)
    t["params"][1].data = torch.zeros(200)
    with pytest.raises(ValueError, match=r"params\[1\]"):
        step(table, 2)
