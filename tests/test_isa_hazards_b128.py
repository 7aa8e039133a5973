"""LDS reads written as inline assembly in the block-128 GEMM, checked in the gfx950 assembly the build produces (no GPU
needed).

The compiler takes the result of such a read for ready at once.  The kernels wait for every read before they
use it; this test checks that the compiler put nothing between a read and its wait that touches the result's
registers (a copy, a spill, a reuse), and that no read is in flight at a label or branch, where the scan could not follow it.
LDS operations return in order, so s_waitcnt lgkmcnt(n) completes all but the last n of them.
"""
import os
import re
import subprocess
import tempfile

import pytest


def _registers(token):
    """Vector registers an operand names: v7, a3, v[4:7]."""
    m = re.fullmatch(r"([va])(\d+)", token) or re.fullmatch(r"([va])\[(\d+):(\d+)\]", token)
    if not m:
        return set()
    return {(m.group(1), r) for r in range(int(m.group(2)), int(m.group(m.lastindex)) + 1)}


def find_hazards(lines):
    """[(line number, text)] of violations in one function's assembly."""
    pending, bad, inline = [], [], False  # destinations of LDS operations in flight, oldest first; none for the compiler's own
    for n, line in enumerate(lines):
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
            continue
        text = line.split(";")[0].strip()
        if not text or text.startswith(".") and not text.startswith(".LBB"):
            continue
        if text.startswith(".LBB") or text.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            if any(pending):
                bad.append((n, "read in flight at " + text))
            pending = []
            continue
        op, _, rest = text.partition(" ")
        wait = re.search(r"lgkmcnt\((\d+)\)", text) if op == "s_waitcnt" else None
        if wait:
            keep = int(wait.group(1))
            pending = pending[len(pending) - keep:] if keep else []
            continue
        operands = [t.strip() for t in re.split(r",(?![^\[]*\])", rest)]
        touched = set().union(*(_registers(t.split()[0]) for t in operands if t)) if rest else set()
        hit = touched & set().union(*pending) if pending else set()
        if hit:
            bad.append((n, text))
        if op.startswith("ds_"):
            pending.append(_registers(operands[0].split()[0]) if inline and "read" in op else set())
    return bad


def functions(text, name):
    """{symbol: lines} of every function whose symbol contains `name`."""
    found, cur = {}, None
    for line in text.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            cur = m.group(1) if name in m.group(1) else None
        if cur:
            if line.startswith(".Lfunc_end"):
                cur = None
            else:
                found.setdefault(cur, []).append(line)
    return found


def test_scan_finds_planted_hazards():
    good = [";;#ASMSTART", "ds_read_b128 v[0:3], v9 offset:0", "ds_read_b32 v4, v9", ";;#ASMEND", "s_waitcnt lgkmcnt(1)", "v_mov_b32_e32 v8, v2",
            "s_waitcnt lgkmcnt(0)", "v_add_f32_e32 v8, v4, v4", "s_cbranch_scc0 .LBB0_1"]
    assert find_hazards(good) == []
    assert find_hazards(good[:5] + ["v_mov_b32_e32 v8, v4"] + good[6:])      # reads a result in flight
    assert find_hazards(good[:5] + ["v_mov_b32_e32 v4, v8"] + good[6:])      # overwrites one
    assert find_hazards(good[:4] + ["v_mov_b64_e32 v[6:7], v[2:3]"] + good[4:])
    assert find_hazards(good[:4] + good[-1:])                               # crosses a branch
    assert find_hazards(good[1:3] + good[-1:]) == []                        # the compiler's own read, which it tracks


def test_no_result_is_touched_before_its_wait():
    from block_scaled_precision_act_amd import build
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        cmd = [build.HIPCC] + build.COMMON + build.DEVICE + ["--cuda-device-only", "-S", os.path.join(build.CSRC, "gemm_b128.hip"),
                                                             "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        text = open(out).read()
    kernels = functions(text, "tile_kernel")
    assert kernels
    for name, lines in kernels.items():
        assert sum("ds_read_b128" in x for x in lines) > 8, name
        assert find_hazards(lines) == [], name
