"""The whole-warp roles of the FP8 product kernel never branch on a wait's outcome, or on the CTA's
abort flag, lane by lane: a lane that left alone would leave the others at a warp-wide
instruction.  Outcomes are remembered (`ok = ok && wait...`), and loops are left by a vote of the
warp.  Read from the source: no run makes lanes disagree at will."""

import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_gemm_fp8_gb300", "csrc",
                      "bsq_fp8.cu")


def roles():
    """Source of the kernel's whole-warp roles by name (the producer is one lane)."""
    text = re.sub(r"//(?! =====).*", "", open(SOURCE).read())
    marks = ["// ===== MMA issuer", "// ===== scales", "// ===== promotion", "if (lane == 0) bulk_wait_all0();"]
    at = [text.index(m) for m in marks]
    assert at == sorted(at)
    return {m: text[a:b] for m, a, b in zip(marks, at, at[1:])}


def statements(text):
    return [" ".join(s.split()) for s in re.split(r"[;{}]", text)]


def test_waits_are_remembered():
    for name, text in roles().items():
        waits = [s for s in statements(text) if re.search(r"\bwait8(_promote)?\(", s)]
        assert waits, name
        for s in waits:
            assert re.match(r"ok = (ok && )?wait8", s), (name, s)


def test_loops_are_left_by_a_vote():
    for name, text in roles().items():
        parts = statements(text)
        assert any("all_lanes(" in s for s in parts), name
        for s in parts:
            assert "goto" not in s and not re.search(r"\b(return|continue)\b", s), (name, s)
            if re.search(r"\bbreak\b", s) or "*abort_flag" in s:
                assert re.search(r"all_lanes\((ok|!\*abort_flag|ok && !\*abort_flag)\)", s), (name, s)
            assert not re.search(r"\b(if|for|while)\b.*\bok\b", re.sub(r"all_lanes\([^()]*\)", "", s)) or "elected && ok" in s, (name, s)


def test_copies_land_after_every_role_has_left():
    """The producer may have ended when another role's wait runs out: its copies are waited for behind
    the barrier that all roles reach."""
    text = open(SOURCE).read()
    teardown = text[text.index("-- teardown"):]
    assert "drain_pending" in teardown[teardown.index("__syncthreads()"):teardown.index("tmem_dealloc(")]
