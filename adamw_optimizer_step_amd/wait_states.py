"""Wait states in this package's own gfx950 code, out of its disassembly.

The compiler keeps the distances that gfx950 wants between dependent instructions
for what it emits itself; it cannot see into inline assembly. ``build`` checks the
machine code of every source that has a matrix instruction or a copy into LDS in
inline assembly, over every path of control:

- a vector register written by a vector instruction is read by a matrix instruction
  (either operand, the accumulator, a scale) 2 wait states later at the earliest;
- the result of a scaled matrix instruction is read or written, but as the whole
  accumulator of the next one, 12 wait states later at the earliest (8 passes;
  8 where both operands are of 4 bits: 4 passes);
- a scalar register written by a vector instruction is the address of a memory
  access 5 wait states later at the earliest;
- a copy into LDS comes 1 wait state after m0 was written at the earliest.

An instruction is one wait state, ``s_nop n`` n + 1.
"""
from __future__ import annotations

import os
import re
import subprocess
import tempfile
from typing import Dict, Iterator, List, NamedTuple, Optional, Set, Tuple

OBJDUMP = os.environ.get("MA_OBJDUMP", "/opt/rocm/llvm/bin/llvm-objdump")

VALU_TO_MFMA, VALU_SGPR_TO_VMEM, M0_TO_LDS_COPY = 2, 5, 1
MFMA_SCALE = "v_mfma_scale_f32_16x16x128_f8f6f4"


class Instr(NamedTuple):
    address: int
    op: str
    args: Tuple[str, ...]     # operands, then modifiers such as cbsz:4
    target: Optional[int]     # of a branch


_LINE = re.compile(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):[^<]*(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?\s*$")
_SYMBOL = re.compile(r"^([0-9a-f]+) <(\S+)>:")
_REGS = re.compile(r"\b([vsa])(?:(\d+)\b|\[(\d+):(\d+)\])")


def parse(text: str) -> Dict[str, List[Instr]]:
    """{kernel: its instructions} of ``llvm-objdump -d``'s output."""
    symbols = {m.group(2): int(m.group(1), 16) for m in map(_SYMBOL.match, text.splitlines()) if m}
    out: Dict[str, List[Instr]] = {}
    cur = None
    for line in text.splitlines():
        m = _SYMBOL.match(line)
        if m:
            cur = out.setdefault(m.group(2), [])
            continue
        m = _LINE.match(line)
        if not m or cur is None:
            continue
        op, args, at, sym, off = m.groups()
        target = symbols[sym] + int(off or "0", 16) if sym and op.startswith(("s_branch", "s_cbranch")) else None
        cur.append(Instr(int(at, 16), op, tuple(a.strip() for a in re.split(r",\s*(?![^\[]*\])|\s+(?=\w+:)", args) if a.strip()), target))
    return out


def regs(arg: str) -> Set[str]:
    """The registers that an operand names: v0, s4, ..; vcc, exec and m0 by their names."""
    out = set()
    for kind, one, lo, hi in _REGS.findall(arg):
        out |= {f"{kind}{i}" for i in ([int(one)] if one else range(int(lo), int(hi) + 1))}
    for name in ("vcc", "exec", "m0"):
        if re.search(rf"\b{name}", arg):
            out.add(name)
    return out


def _mfma(i: Instr) -> bool:
    return i.op.startswith(("v_mfma", "v_smfmac"))


def _valu(i: Instr) -> bool:
    return i.op.startswith("v_") and not _mfma(i)


def _memory(i: Instr) -> bool:
    return i.op.startswith(("global_", "flat_", "buffer_", "scratch_"))


def _written(i: Instr) -> Set[str]:
    """What an instruction writes: the first operand, of carries and v_*_swap the second too."""
    if not i.args or i.op.startswith(("global_store", "flat_store", "buffer_store", "ds_write", "s_cmp", "s_cbranch", "s_branch", "s_nop", "s_waitcnt")):
        return set()
    out = regs(i.args[0])
    if "_swap_" in i.op or re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_mad_[ui]64|v_div_scale", i.op):
        out |= regs(i.args[1])
    return out


def _passes(i: Instr) -> int:
    return 4 if "cbsz:4" in i.args and "blgp:4" in i.args else 8


def _ahead(code: List[Instr], index: Dict[int, int], start: int, states: int) -> Iterator[Tuple[int, Instr]]:
    """Every instruction that can issue fewer than `states` wait states after code[start], with its distance."""
    todo, seen = [(start + 1, 0)], {}
    first = code[start]
    if first.target is not None:
        todo.append((index[first.target], 0))
    while todo:
        k, d = todo.pop()
        if k >= len(code) or d >= states or seen.get(k, states) <= d:
            continue
        seen[k] = d
        i = code[k]
        yield d, i
        if i.op.startswith("s_endpgm"):
            continue
        after = d + (int(i.args[0], 0) + 1 if i.op == "s_nop" else 1)
        if i.target is not None:
            todo.append((index[i.target], after))
        if i.op != "s_branch":
            todo.append((k + 1, after))


def violations(text: str) -> List[str]:
    """The places in ``llvm-objdump -d``'s output that keep a distance too short, as messages."""
    bad = []
    for kernel, code in parse(text).items():
        index = {i.address: k for k, i in enumerate(code)}
        for k, i in enumerate(code):
            def report(rule: str, at: Instr, d: int) -> None:
                bad.append(f"{kernel}: {rule}: {i.op} {', '.join(i.args)} at {i.address:x}, {d} wait states before {at.op} {', '.join(at.args)} at {at.address:x}")
            if _valu(i):
                w = _written(i)
                vector, scalar = {r for r in w if r[0] == "v" and r != "vcc"}, {r for r in w if r[0] == "s" or r == "vcc"}
                for d, j in _ahead(code, index, k, VALU_TO_MFMA) if vector else ():
                    if _mfma(j) and any(vector & regs(a) for a in j.args[1:]):
                        report("vector result into a matrix instruction", j, d)
                for d, j in _ahead(code, index, k, VALU_SGPR_TO_VMEM) if scalar else ():
                    if _memory(j) and any(scalar & regs(a) for a in j.args):
                        report("vector result as a scalar address", j, d)
            elif i.op == MFMA_SCALE:
                w = regs(i.args[0])
                for d, j in _ahead(code, index, k, _passes(i) + 4):
                    if not any(w & regs(a) for a in j.args):
                        continue
                    # (as the accumulator, whole, without a distance)
                    if _mfma(j) and not any(w & regs(a) for n, a in enumerate(j.args) if n not in (0, 3)) and regs(j.args[3]) == w \
                            and (regs(j.args[0]) == w or not regs(j.args[0]) & w):
                        continue
                    report("matrix result", j, d)
            elif i.op.startswith("s_") and "m0" in _written(i):
                for d, j in _ahead(code, index, k, M0_TO_LDS_COPY):
                    if "_load_lds_" in j.op:
                        report("m0 into a copy to LDS", j, d)
    return bad


def disassemble(obj: str) -> str:
    """The gfx950 code in an object or library that hipcc wrote, as ``llvm-objdump -d`` prints it."""
    with tempfile.TemporaryDirectory() as tmp:
        copy = os.path.join(tmp, "o")
        os.symlink(os.path.abspath(obj), copy)
        subprocess.run([OBJDUMP, "--offloading", copy], cwd=tmp, check=True, capture_output=True)
        parts = [os.path.join(tmp, f) for f in sorted(os.listdir(tmp)) if "amdgcn" in f]
        return "".join(subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", p], check=True, capture_output=True, text=True).stdout for p in parts)
