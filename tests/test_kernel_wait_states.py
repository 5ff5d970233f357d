"""Wait states in the built kernels that the hardware does not supply itself.

The compiler inserts them between instructions that it emits, but neither into
inline asm nor in front of it, so they are checked in the built library:

* a scalar write of m0 needs one instruction (or s_nop) between itself and a
  load that places its data in LDS by m0;
* a scalar register written by a vector instruction (readfirstlane) needs five
  wait states before a memory instruction takes its address from it.
"""
import os
import re
import struct
import subprocess
import tempfile

import pytest

from combine_routing_preprocess_amd import build as B

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(path):
    """The gfx950 code objects bundled in the library."""
    with open(path, "rb") as f:
        blob = f.read()
    at = blob.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            off, size, l = struct.unpack_from("<QQQ", blob, p)
            name = blob[p + 24:p + 24 + l].decode()
            p += 24 + l
            if B.ARCH in name and size:
                yield blob[at + off:at + off + size]
        at = blob.find(MAGIC, at + len(MAGIC))


def _functions(code):
    """(name, [(mnemonic, operands)]) of every function of a code object."""
    with tempfile.NamedTemporaryFile(suffix=".co") as f:
        f.write(code)
        f.flush()
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f.name], check=True, stdout=subprocess.PIPE,
                              text=True).stdout
    name, body = "", []
    for line in text.splitlines():
        head = re.match(r"^[0-9a-f]+ <(.+)>:", line)
        if head:
            if body:
                yield name, body
            name, body = head.group(1), []
            continue
        ins = line.split("//")[0].strip().split(None, 1)
        if ins and line[:1].isspace():
            body.append((ins[0], ins[1] if len(ins) > 1 else ""))
    if body:
        yield name, body


def to_lds(op, args):
    return "_load_lds_" in op or (op.startswith("buffer_load") and re.search(r"\blds\b", args) is not None)


def writes_m0(op, args):
    return op.startswith("s_") and re.match(r"m0\b", args) is not None


def m0_hazards(body):
    """Loads to LDS directly behind a scalar write of m0."""
    return [i for i in range(1, len(body)) if to_lds(*body[i]) and writes_m0(*body[i - 1])]


def _sgprs(args):
    regs = set()
    for a, b, c in re.findall(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)", args):
        regs |= set(range(int(a), int(b) + 1)) if a else {int(c)}
    return regs


def scalar_base_hazards(body):
    """Memory instructions whose scalar registers a vector instruction wrote
    fewer than five wait states before."""
    found = []
    for i, (op, args) in enumerate(body):
        if not op.startswith(("global_", "buffer_", "flat_", "scratch_")):
            continue
        regs, states, j = _sgprs(args), 0, i - 1
        while regs and j >= 0 and states < 5:
            prev, pargs = body[j]
            if prev.startswith("v_") and _sgprs(pargs.split(",")[0]) & regs:
                found.append(i)
                break
            states += 1 + (int(pargs, 0) if prev == "s_nop" else 0)
            j -= 1
    return found


def test_the_checks_see_what_they_look_for():
    load = ("global_load_lds_dwordx4", "v1, s[4:5]")
    assert m0_hazards([("s_mov_b32", "m0, s2"), load]) == [1]
    assert m0_hazards([("s_add_i32", "m0, s2, 16"), ("s_nop", "0"), load]) == []
    assert m0_hazards([("s_mov_b32", "m0, s2"), ("global_load_dwordx4", "v[0:3], v1, s[4:5]")]) == []
    write = ("v_readfirstlane_b32", "s5, v0")
    assert scalar_base_hazards([write, ("s_nop", "3"), load]) == [2]
    assert scalar_base_hazards([write, ("s_nop", "4"), load]) == []
    assert scalar_base_hazards([("v_readfirstlane_b32", "s6, v0"), load]) == []


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs the ROCm disassembler")
def test_loads_to_lds_wait_for_m0_and_their_base():
    if not os.path.exists(B.LIB):
        B.build(verbose=False)
    loads, m0, base = 0, {}, {}
    for code in _code_objects(B.LIB):
        for name, body in _functions(code):
            loads += sum(to_lds(*ins) for ins in body)
            for found, where in ((m0_hazards(body), m0), (scalar_base_hazards(body), base)):
                if found:
                    where[name] = len(found)
    assert loads > 1000          # the GEMMs' transfers were seen
    assert not m0, m0
    assert not base, base
