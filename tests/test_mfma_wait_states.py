"""The delta rule's matrix instructions and the first use of their results, read from the compiler's assembly (no
GPU needed).  The hardware does not interlock a matrix instruction's result against other instructions: the
compiler has to leave wait states between them on every path, and where a branch stands in between it has been
seen to count them along one path only.  Here every path from every matrix instruction is followed for as many
instructions as its result takes."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from selective_state_space_03_amd import build as b

# wait states before another instruction may touch the result
WAIT = {"v_mfma_f32_16x16x32_bf16": 7, "v_mfma_f32_16x16x4_f32": 10}


def _assembly(src):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "k.s")
        cmd = [hipcc, *b.COMMON, *b.DEVICE_FLAGS, "--cuda-device-only", "-S", os.path.join(b.CSRC, src), "-o", out]
        res = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert res.returncode == 0, res.stderr[-3000:]
        return open(out).read()


def _regs(text):
    out = set()
    for m in re.finditer(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        else:
            out.add((m.group(4), int(m.group(5))))
    return out


def _functions(text):
    name, body = None, None
    for line in text.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name, body = m.group(1), []
        elif body is not None:
            if line.startswith(".Lfunc_end"):
                yield name, body
                body = None
                continue
            code = line.split(";")[0].strip()
            m = re.match(r"^(\.LBB\w+):", line)
            if m:
                body.append(m.group(1) + ":")
            elif code and not code.startswith("."):
                body.append(code)


def violations(text):
    """(matrix instructions seen, uses of a result ahead of its wait states)"""
    seen_mfma, bad = 0, []
    for name, body in _functions(text):
        label = {c[:-1]: i for i, c in enumerate(body) if c.endswith(":")}
        for i, code in enumerate(body):
            if not code.startswith("v_mfma"):
                continue
            seen_mfma += 1
            need = WAIT[code.split()[0]]
            dst = _regs(code.split(None, 1)[1].split(",")[0])
            stack, best = [(i + 1, 0)], {}
            while stack:
                j, waited = stack.pop()
                if j >= len(body) or waited >= need or best.get(j, need) <= waited:
                    continue
                best[j] = waited
                c = body[j]
                if c.endswith(":"):
                    stack.append((j + 1, waited))
                    continue
                op, _, rest = c.partition(" ")
                step = 1
                if op == "s_endpgm":
                    continue
                if op == "s_branch":
                    stack.append((label[rest.strip()], waited + 1))
                    continue
                if op.startswith("s_cbranch"):
                    stack.append((label[rest.strip()], waited + 1))
                elif op == "s_nop":
                    step = int(rest, 0) + 1
                elif op.startswith("v_mfma"):
                    ops = rest.split(",")
                    if _regs(ops[1] + "," + ops[2]) & dst:
                        bad.append((name, code, c, waited))
                        continue
                    if _regs(ops[0]) == dst:  # the accumulator handed on is interlocked
                        continue
                elif _regs(rest) & dst:
                    bad.append((name, code, c, waited))
                    continue
                stack.append((j + 1, waited + step))
    return seen_mfma, bad


@pytest.mark.parametrize("src", ["delta_prep.hip", "delta_pass.hip", "delta_grads.hip"])
def test_results_are_waited_for_on_every_path(src):
    n, bad = violations(_assembly(src))
    assert n > 100
    assert not bad, bad[:5]


def test_the_reader_sees_a_short_path():
    """A result read right behind a branch over other work, as it was once generated."""
    text = """
_Zk:
	v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[4:7], a[0:3]
	s_cbranch_vccz .LBB0_2
	v_mov_b32 v20, v21
	v_mov_b32 v22, v21
	v_mov_b32 v23, v21
	v_mov_b32 v24, v21
	v_mov_b32 v25, v21
	v_mov_b32 v26, v21
	v_mov_b32 v27, v21
.LBB0_2:
	v_accvgpr_read_b32 v1, a3
	s_endpgm
.Lfunc_end0:
"""
    assert len(violations(text)[1]) == 1
    assert not violations(text.replace("s_cbranch_vccz", "s_nop 6\n\ts_cbranch_vccz"))[1]
