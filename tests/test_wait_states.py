"""CPU test of the compiled kernels: the wait states that gfx9 hardware does not check by itself.

The compiler inserts them for the instructions it chooses, but does not look into inline assembly:

  - a scalar register written by a vector instruction (v_readfirstlane, v_cmp, ..) is read by a memory
    instruction no sooner than 5 wait states later: a buffer descriptor's size or a base address read too early is
    the old one, and the access may leave its array;
  - M0 is written at least 1 wait state before a load to LDS, which takes its LDS address from it.

An instruction is one wait state, s_nop n is n + 1.  The listing of each kernel in the built library is followed
backwards from every memory instruction, over branches."""
import os
import re
import struct
import subprocess

import pytest

import rotation_then_quantize_amd as rtq

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
VCC = 106      # register number of vcc
VMEM = ("buffer_", "global_", "flat_", "scratch_")
VALU_TO_VMEM, M0_TO_LDS = 5, 1


def code_objects(library):
    """The gfx950 code objects in a library's offload bundles."""
    at = library.find(MAGIC)
    while at >= 0:
        (count,) = struct.unpack_from("<Q", library, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, n = struct.unpack_from("<QQQ", library, p)
            triple = library[p + 24:p + 24 + n].decode()
            p += 24 + n
            if triple.endswith("gfx950") and size:
                yield library[at + offset:at + offset + size]
        at = library.find(MAGIC, at + len(MAGIC))


def scalars(operand):
    """Numbers of the scalar registers an operand names."""
    m = re.fullmatch(r"-?\|?s(\d+)\|?", operand)
    if m:
        return {int(m[1])}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    return {"vcc": {VCC, VCC + 1}, "vcc_lo": {VCC}, "vcc_hi": {VCC + 1}}.get(operand, set())


class Instr:
    __slots__ = ("text", "name", "waits", "valu_writes", "writes_m0", "before")

    def __init__(self, text):
        self.text = text
        self.name, _, rest = text.partition(" ")
        operands = [o.strip().split(" ")[0] for o in rest.split(",")] if rest else []
        self.waits = int(operands[0], 0) + 1 if self.name == "s_nop" else 1
        self.valu_writes = set()
        if self.name.startswith("v_") and operands:
            self.valu_writes = scalars(operands[0])
            if len(operands) > 1 and re.search(r"_co_|div_scale|mad_[ui]64", self.name):
                self.valu_writes = self.valu_writes | scalars(operands[1])
        self.writes_m0 = self.name.startswith("s_") and bool(operands) and operands[0] == "m0" and not self.name.startswith("s_cmp")
        self.before = []      # indexes of the instructions that may run right before this one

    @property
    def scalar_reads(self):
        words = re.split(r"[,\s]+", self.text)[1:]
        return set().union(*(scalars(w) for w in words)) if words else set()

    @property
    def to_lds(self):
        return self.name.startswith("buffer_load") and self.text.endswith(" lds") or "_load_lds_" in self.name


LINE = re.compile(r"^\t(\S[^/]*?)\s*// ([0-9A-F]+):(?:.*<([^>+]+)(?:\+0x([0-9a-f]+))?>)?")


def kernels(listing):
    """(name, instructions) of each function in an objdump listing, linked to what may run before each."""
    name, base, body = None, 0, []
    for line in listing.splitlines() + ["0000 <end>:"]:
        head = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if head:
            if body:
                yield name, link(body, base)
            name, base, body = head[2], int(head[1], 16), []
            continue
        m = LINE.match(line)
        if m:
            body.append((int(m[2], 16), re.sub(r"\s+", " ", m[1]), int(m[4] or "0", 16) if m[3] else None))


def link(body, base):
    code = [Instr(text) for _, text, _ in body]
    index = {address: i for i, (address, _, _) in enumerate(body)}
    for i, (_, _, target) in enumerate(body):
        branch = code[i].name.startswith(("s_branch", "s_cbranch"))
        if i + 1 < len(code) and code[i].name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            code[i + 1].before.append(i)
        if branch:
            assert target is not None, code[i].text
            code[index[base + target]].before.append(i)
    return code


def reached(code, i, limit, hit):
    """The instruction that satisfies `hit` fewer than `limit` wait states before instruction i, if any."""
    seen, todo = {}, [(b, 0) for b in code[i].before]
    while todo:
        j, between = todo.pop()
        if between >= limit or seen.get(j, limit) <= between:
            continue
        seen[j] = between
        if hit(code[j]):
            return code[j], between
        todo += [(b, between + code[j].waits) for b in code[j].before]
    return None


def hazards(listing):
    found = []
    for name, code in kernels(listing):
        for i, instr in enumerate(code):
            if not instr.name.startswith(VMEM):
                continue
            reads = instr.scalar_reads
            r = reached(code, i, VALU_TO_VMEM, lambda c: c.valu_writes & reads) if reads else None
            if r:
                found.append(f"{name}: '{r[0].text}', {r[1]} wait states before '{instr.text}'")
            r = reached(code, i, M0_TO_LDS, lambda c: c.writes_m0) if instr.to_lds else None
            if r:
                found.append(f"{name}: '{r[0].text}', {r[1]} wait states before '{instr.text}'")
    return found


def test_the_check_sees_what_it_looks_for():
    listing = """
0000000000001000 <k>:
	v_readfirstlane_b32 s6, v0                                 // 000000001000: 7E0C0500
	s_mov_b32 m0, s9                                           // 000000001004: BEFC0009
	buffer_load_dwordx4 v1, s[4:7], 0 offen lds                // 000000001008: E05D1000 80010001
	v_cmp_gt_i32_e32 vcc, 1, v2                                // 000000001010: 7D880481
	s_nop 4                                                    // 000000001014: BF800004
	global_load_dword v3, v4, vcc                              // 000000001018: DC508000 036A0004
	v_readfirstlane_b32 s8, v0                                 // 000000001020: 7E100500
	s_cbranch_scc0 2                                           // 000000001024: BF840002 <k+0x30>
	s_nop 4                                                    // 000000001028: BF800004
	s_nop 0                                                    // 00000000102C: BF800000
	buffer_load_dword v1, v2, s[8:11], 0 offen                 // 000000001030: E0501000 80020102
	s_endpgm                                                   // 000000001038: BF810000
"""
    found = hazards(listing)
    assert len(found) == 3
    assert "s6" in found[0] and "1 wait states" in found[0] and "m0" in found[1] and "s8" in found[2]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_kernels_keep_the_wait_states(tmp_path):
    with open(rtq.LIB_PATH, "rb") as f:
        library = f.read()
    found, seen = [], 0
    for n, code in enumerate(code_objects(library)):
        path = tmp_path / f"{n}.elf"
        path.write_bytes(code)
        listing = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
        seen += listing.count("s_endpgm")
        found += hazards(listing)
    assert seen > 100
    assert not found, f"{len(found)} places, among them:\n" + "\n".join(found[:8])
