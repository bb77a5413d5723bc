"""A check of built machine code for the one hazard that inline assembly
leaves open: the compiler keeps no wait states around it.

A vector memory instruction has to stand five wait states behind a vector
instruction that writes a scalar register it reads (v_readlane of a spilled
scalar, v_readfirstlane), and one behind the write of m0.  violations() goes
back from every buffer load into LDS over all paths that lead to it.
"""
from __future__ import annotations

import os
import re
import subprocess
import tempfile

SCALAR_WAITS, M0_WAITS = 5, 1

_INSN = re.compile(r"^\s+([a-z]\w*)\s*(.*?)\s*(?://.*)?$")
_LABEL = re.compile(r"^[0-9a-f]+ <(.+)>:\s*$")
_FUNCTION = re.compile(r"(?m)^(?=[0-9a-f]+ <(?!L\d+>))")
_REGS = re.compile(r"^(?:s(\d+)|s\[(\d+):(\d+)\])$")
# vector instructions with a scalar as their second result
_CARRIES = re.compile(r"^v_(add|sub|subrev|addc|subb|subbrev)_co_|^v_div_scale_|^v_mad_[iu]64_")


def _scalars(operand):
    """Numbers of the scalar registers in an operand; -1: m0."""
    operand = operand.strip()
    if operand == "m0":
        return {-1}
    m = _REGS.match(operand)
    if not m:
        return set()
    if m.group(1):
        return {int(m.group(1))}
    return set(range(int(m.group(2)), int(m.group(3)) + 1))


def _parse(text):
    """[(mnemonic, operands)] and {label: index of the instruction behind it}."""
    code, labels = [], {}
    for line in text.splitlines():
        m = _LABEL.match(line)
        if m:
            labels[m.group(1)] = len(code)
            continue
        m = _INSN.match(line)
        if m:
            code.append((m.group(1), [o for o in m.group(2).split(", ") if o]))
    return code, labels


def _written(mnemonic, operands):
    """Scalars that a vector instruction writes."""
    if not mnemonic.startswith("v_") or not operands:
        return set()
    out = _scalars(operands[0])
    if _CARRIES.match(mnemonic) and len(operands) > 1:
        out |= _scalars(operands[1])
    return out


def violations(text):
    """Loads of a listing (llvm-objdump -d --symbolize-operands, one function
    or several) that stand too close behind a write of a scalar they read."""
    bad, loads = [], 0
    for part in _FUNCTION.split(text):
        code, labels = _parse(part)
        into = {}
        for i, (name, ops) in enumerate(code):
            if name.startswith(("s_branch", "s_cbranch")) and ops:
                target = ops[0].split()[0]
                if target not in labels:
                    raise ValueError(f"no label {target}")
                into.setdefault(labels[target], []).append(i)
            elif name.startswith(("s_setpc", "s_swappc", "s_call")):
                raise ValueError(f"{name}: a jump that is not followed")
        for i, (name, ops) in enumerate(code):
            if not (name.startswith("buffer_load") and ops[-1].split()[-1] == "lds"):
                continue
            loads += 1
            reads = set().union(*(_scalars(o.split()[0]) for o in ops[1:])) | {-1}
            seen, todo = set(), [(i, 0)]
            while todo:
                at, waits = todo.pop()
                if waits >= SCALAR_WAITS or (at, waits) in seen:
                    continue
                seen.add((at, waits))
                before = list(into.get(at, ()))
                if at > 0 and not code[at - 1][0].startswith(("s_branch", "s_endpgm")):
                    before.append(at - 1)
                for b in before:
                    bname, bops = code[b]
                    m0 = bname.startswith("s_") and bops and _scalars(bops[0]) == {-1}
                    if (_written(bname, bops) & reads) or (m0 and waits < M0_WAITS):
                        bad.append(f"{name} {', '.join(ops)}: {waits} wait states behind "
                                   f"{bname} {', '.join(bops)}")
                    todo.append((b, waits + 1 + (int(bops[0], 0) if bname == "s_nop" else 0)))
    return bad, loads


def listing(obj, llvm="/opt/rocm/llvm/bin", arch="gfx950"):
    """The machine code for `arch` in a HIP object file."""
    with tempfile.TemporaryDirectory() as d:
        here = os.path.join(d, "o")
        os.symlink(os.path.abspath(obj), here)
        objdump = os.path.join(llvm, "llvm-objdump")
        subprocess.run([objdump, "--offloading", here], check=True, cwd=d, capture_output=True)
        codes = [f for f in os.listdir(d) if arch in f]
        if len(codes) != 1:
            raise RuntimeError(f"{obj}: {len(codes)} code objects for {arch}")
        return subprocess.run([objdump, "-d", "--symbolize-operands", os.path.join(d, codes[0])],
                              check=True, capture_output=True, text=True).stdout


def check_object(obj, **kw):
    """Raises where the device code of a HIP object file breaks the rule."""
    bad, loads = violations(listing(obj, **kw))
    if bad or not loads:
        raise RuntimeError(f"{obj}: {loads} loads into LDS, {len(bad)} too close behind the "
                           "write of a scalar that they read:\n" + "\n".join(bad[:20]))
    return loads
