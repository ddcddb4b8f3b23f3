"""The matrix instructions that the product kernels write as inline assembly, in the compiled listing.

The compiler does not know that such an instruction's sums must not be touched until it has ended, by
anything but the next matrix instruction that adds to all of them. Every path through each kernel is
followed, and no other instruction may name a register of a sum less than WAIT cycles after the
instruction that wrote it: no copy to other registers, no store before the waits at the loop's end."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from partitioned_chip_accumulation_amd import build

WAIT = 19  # cycles after the longest matrix instruction (16 passes)
REGISTER = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def registers(text):
    """The vector registers of an operand, as ('v', number)."""
    out = []
    for kind, low, high, one in REGISTER.findall(text):
        out += [(kind, r) for r in (range(int(low), int(high) + 1) if low else (int(one),))]
    return out


def kernels(listing):
    """{name: [(label or None, mnemonic, operands, whether in inline assembly)]}"""
    out, name, inline = {}, None, False
    for line in listing.splitlines():
        start = re.match(r"(_Z\w+):", line)
        if start:
            name = start.group(1)
            out[name] = []
        if name is None:
            continue
        if ";#ASMSTART" in line or ";#ASMEND" in line:
            inline = "START" in line
            continue
        code = line.split(";")[0].strip()
        label = re.match(r"(\.LBB\w+):", code)
        if label:
            out[name].append((label.group(1), "", "", False))
        elif line.startswith("\t") and code and not code.startswith("."):
            mnemonic, _, operands = code.partition(" ")
            out[name].append((None, mnemonic.split("\t")[0],
                              operands or code.partition("\t")[2], inline))
        if line.startswith(".Lfunc_end"):
            name = None
    return {n: code for n, code in out.items() if any(m == "s_endpgm" for _, m, _, _ in code)}


def blocks(code):
    """[(instructions, the blocks that follow)]"""
    starts = {0}
    for i, (label, mnemonic, _, _) in enumerate(code):
        if label:
            starts.add(i)
        if mnemonic.startswith(("s_cbranch", "s_branch", "s_endpgm")) and i + 1 < len(code):
            starts.add(i + 1)
    order = sorted(starts)
    number = {s: b for b, s in enumerate(order)}
    labels = {code[s][0]: b for s, b in number.items() if code[s][0]}
    out = []
    for b, s in enumerate(order):
        part = code[s:order[b + 1] if b + 1 < len(order) else len(code)]
        _, mnemonic, operands, _ = part[-1]
        after = []
        if mnemonic.startswith(("s_cbranch", "s_branch")):
            after.append(labels[operands.strip()])
        if not mnemonic.startswith(("s_branch", "s_endpgm")) and b + 1 < len(order):
            after.append(b + 1)
        out.append((part, after))
    return out


def compiled(part):
    """(mnemonic, registers, cycles, (sum, is its own addend) of a matrix instruction, inline)"""
    out = []
    for _, mnemonic, operands, inline in part:
        if not mnemonic:
            continue
        cycles = int(operands, 0) + 1 if mnemonic == "s_nop" else 1
        product = None
        named = frozenset(registers(operands))
        if mnemonic.startswith("v_mfma"):
            d, a, b, c = [frozenset(registers(o)) for o in
                          re.findall(r"[va]\[\d+:\d+\]|[va]\d+|-?\d+", operands)[:4]]
            product = d, d == c, a | b
        out.append((mnemonic, named, cycles, product, inline, operands))
    return out


def touched_too_early(code):
    """What names a register less than WAIT cycles after an inline matrix instruction wrote it, and
    how many such instructions there are."""
    graph = [(compiled(part), after) for part, after in blocks(code)]
    count = sum(bool(i[3] and i[4]) for part, _ in graph for i in part)
    if not count:
        return [], 0
    found = set()
    known = [None] * len(graph)  # at a block's start: register -> cycles since it was written
    known[0] = {}
    work = [0]
    while work:
        b = work.pop()
        age = dict(known[b])
        part, after = graph[b]
        for mnemonic, named, cycles, product, inline, operands in part:
            if age:
                early = [r for r in named if r in age]
                if product and early:
                    d, same, factors = product
                    early = [r for r in early if r in factors or not (same and r in d)]
                if early:
                    found.add(f"{mnemonic} {operands}")
                age = {r: c + cycles for r, c in age.items() if c + cycles < WAIT}
            if product and inline:
                for r in product[0]:
                    age[r] = 0
        for n in after:
            merged = dict(known[n]) if known[n] is not None else {}
            for r, c in age.items():
                merged[r] = min(c, merged.get(r, WAIT))
            if merged != known[n]:
                known[n] = merged
                if n not in work:
                    work.append(n)
    return sorted(found), count


@pytest.fixture(scope="module", params=["experts_matmul.hip", "experts_dw.hip", "experts_int8.hip"])
def listing(request, tmp_path_factory):
    hipcc = build.hipcc() if os.path.exists(build.hipcc()) else shutil.which("hipcc")
    if not hipcc:
        pytest.skip("ROCm compiler not available")
    out = tmp_path_factory.mktemp("listing") / "device.s"
    subprocess.run([hipcc, *build.HIPCC_FLAGS, "--cuda-device-only", "-S", "-I", build.INCLUDE,
                    "-I", build.CSRC, os.path.join(build.CSRC, request.param), "-o", str(out)],
                   check=True, capture_output=True)
    return out.read_text()


def test_sums_are_left_alone_until_they_are_done(listing):
    results = {name: touched_too_early(code) for name, code in kernels(listing).items()}
    assert any(count for _, count in results.values())
    assert not {name: found[:5] for name, (found, _) in results.items() if found}


def test_a_copy_of_a_sum_is_found(listing):
    """The same listing with a register copy behind one of its matrix instructions."""
    broken, made = re.subn(r"(\tv_mfma\S+ v\[(\d+):\d+\].*\n\t;;#ASMEND\n)",
                           r"\1\tv_mov_b32_e32 v0, v\2\n", listing, count=1)
    assert made == 1
    results = [touched_too_early(code) for code in kernels(broken).values()]
    assert sum(bool(found) for found, _ in results) == 1


SNIPPET = """_Zone:
\t;;#ASMSTART
\ts_nop 1
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]
\t;;#ASMEND
%s
\ts_endpgm
.Lfunc_end0:
"""


@pytest.mark.parametrize("text,early", [
    ("\tv_mov_b32_e32 v20, v3", True),
    ("\tv_mov_b32_e32 v2, v20", True),
    ("\tds_write_b64 v30, v[2:3]", True),
    ("\tv_mov_b32_e32 v20, v4", False),
    ("\ts_nop 15\n\ts_nop 1\n\tv_mov_b32_e32 v20, v3", True),
    ("\ts_nop 15\n\ts_nop 2\n\tv_mov_b32_e32 v20, v3", False),
    ("\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", False),
    ("\tv_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], v[0:3]", True),
    ("\tv_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], v[4:7]", True),
    ("\ts_cbranch_scc1 .LBB0_2\n\ts_nop 15\n\ts_nop 15\n.LBB0_2:\n\tv_mov_b32_e32 v20, v3", True),
    ("\ts_branch .LBB0_2\n.LBB0_1:\n\tv_mov_b32_e32 v20, v3\n.LBB0_2:\n\ts_nop 15\n\ts_nop 3",
     False),
])
def test_the_check_itself(text, early):
    found, count = touched_too_early(kernels(SNIPPET % text)["_Zone"])
    assert count == 1 and bool(found) == early
