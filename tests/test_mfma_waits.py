"""The large bf16 tile's matrix instructions are inline assembly, to which the compiler adds no waits.  Its
assembly (built here, no GPU needed) is read: whatever touches their results apart from another matrix
instruction comes after the written wait on every path, and no vector instruction writes their operands right
before them."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from block_scaled_fp4_02_amd import build

WAIT = 8       # wait states after a 16x16x32 MFMA before its result is read, and of the written wait
OPERAND = 2    # between a vector instruction that writes a register and an MFMA that reads it


def _registers(operand):
    out = set()
    for kind, one, kinds, lo, hi in re.findall(r"\b([av])(\d+)\b|\b([av])\[(\d+):(\d+)\]", operand):
        out |= {(kind, int(one))} if kind else {(kinds, i) for i in range(int(lo), int(hi) + 1)}
    return out


class Kernel:
    """Instructions of one kernel: (name, operands, registers, written inline), and their successors."""

    def __init__(self):
        self.code, self.labels = [], {}

    def add(self, text, inline):
        name, _, rest = text.partition(" ")
        operands = [o.strip() for o in re.split(r",\s*(?![^\[]*\])", rest)]
        self.code.append((name, operands, [_registers(o) for o in operands], inline))

    def after(self, i):
        name, operands, _, _ = self.code[i]
        if name == "s_endpgm":
            return []
        jump = [self.labels[operands[0]]] if name.startswith(("s_branch", "s_cbranch")) and operands[0] in self.labels else []
        return jump if name == "s_branch" else jump + [i + 1] * (i + 1 < len(self.code))

    def states(self, i):
        name, operands, _, _ = self.code[i]
        return int(operands[0], 0) + 1 if name == "s_nop" else 1

    def touched_before_wait(self, i):
        """The first instructions after MFMA i, on any path without the wait, that touch its result and are no MFMA."""
        result, seen, todo = self.code[i][2][0], set(), self.after(i)
        while todo:
            j = todo.pop()
            if j in seen or self.states(j) >= WAIT:
                continue
            seen.add(j)
            name, operands, regs, _ = self.code[j]
            if not name.startswith("v_mfma") and any(result & r for r in regs):
                yield name, operands
                continue
            todo += self.after(j)

    def writes_just_before(self, i):
        """Vector instructions that write a register that inline MFMA i reads, fewer than OPERAND states before it."""
        reads = set().union(*self.code[i][2][1:])
        for j in range(max(0, i - 8), i):
            name, operands, regs, _ = self.code[j]
            if name.startswith("v_") and not name.startswith("v_mfma") and regs[0] & reads:
                if sum(self.states(k) for k in range(j + 1, i)) < OPERAND:
                    yield name, operands


def _kernels(listing):
    kernels, kernel, inline = {}, None, False
    for line in listing.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
        line = line.split(";")[0].rstrip()
        label = re.match(r"([\w.$]+):$", line.strip())
        if label and not label[1].startswith("."):
            kernel = kernels.setdefault(label[1], Kernel())
        elif label and kernel:
            kernel.labels[label[1]] = len(kernel.code)
        elif kernel and line.strip() and not line.strip().startswith("."):
            kernel.add(line.strip(), inline)
    return kernels


@pytest.fixture(scope="module")
def inline_mfmas(tmp_path_factory):
    """(name, Kernel, numbers of its inline MFMAs) of every kernel that has some."""
    out = tmp_path_factory.mktemp("listing") / "bf16_gemm.s"
    flags = [f for f in build.COMPILE_FLAGS if f != "-fPIC"] + build.EXTRA_FLAGS.get("bf16_gemm.hip", [])
    subprocess.run([build.HIPCC, *build.ARCH_FLAGS, *flags, "--cuda-device-only", "-S", os.path.join(build.CSRC, "bf16_gemm.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    found = []
    for name, kernel in _kernels(out.read_text()).items():
        at = [i for i, c in enumerate(kernel.code) if c[0].startswith("v_mfma") and c[3]]
        if at:
            found.append((name, kernel, at))
    return found


def test_the_large_tiles_are_found(inline_mfmas):
    """Two plain products, the gated one, its backward pass, and four weight gradients, each with 8, 4 and 2
    column tiles in use, 8 MFMAs of each in either half of the loop."""
    assert len(inline_mfmas) == 8
    assert all(len(at) == 2 * 8 * (8 + 4 + 2) for _, _, at in inline_mfmas)


def test_results_are_read_after_the_wait(inline_mfmas):
    for name, kernel, at in inline_mfmas:
        for i in at:
            assert not list(kernel.touched_before_wait(i)), (name, kernel.code[i][:2])


def test_operands_are_not_written_just_before(inline_mfmas):
    for name, kernel, at in inline_mfmas:
        for i in at:
            assert not list(kernel.writes_just_before(i)), (name, kernel.code[i][:2])
