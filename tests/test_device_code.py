"""CPU checks of the instructions that the library's kernels were compiled to.

The compiler puts the wait states that the hardware asks for between its own
instructions, but it does not look inside inline assembly.  Of the rules for
gfx9's manually inserted wait states two meet the copies into LDS, which are
written that way:
  - a scalar register written by the vector ALU (v_readfirstlane, a comparison, a
    carry) may be read by a memory instruction 5 wait states later;
  - M0 written by the scalar ALU may be used by a copy into LDS 1 wait state later.
An instruction is one wait state, s_nop n is n + 1.  Every way through a kernel is followed."""
import os
import re
import shutil
import struct
import subprocess
import tempfile

import pytest

import w4a4_rank_corrected_smooth_amd as S

OBJDUMP = shutil.which("llvm-objdump") or os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
M0, VCC = 124, (106, 107)
MEMORY = ("global_", "buffer_", "flat_", "scratch_")


def code_objects(path):
    """The gfx950 code objects of the library's offload bundles."""
    data, magic = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        p = at + 32
        for _ in range(struct.unpack_from("<Q", data, at + 24)[0]):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + n]:
                yield data[at + off:at + off + size]
            p += 24 + n
        at = data.find(magic, at + 24)


def scalars(operands):
    """The numbers of the scalar registers in a text of operands."""
    found = set()
    for m in re.finditer(r"\bs(\d+)\b|\bs\[(\d+):(\d+)\]|\b(vcc)\b|\b(m0)\b", operands):
        if m[1]:
            found.add(int(m[1]))
        elif m[2]:
            found |= set(range(int(m[2]), int(m[3]) + 1))
        else:
            found |= set(VCC) if m[4] else {M0}
    return found


def kernels(code):
    """(name, [(mnemonic, operands, index of the branch's target or None)]) of a code object."""
    with tempfile.NamedTemporaryFile(suffix=".o") as f:
        f.write(code)
        f.flush()
        text = subprocess.run([OBJDUMP, "-d", "-z", f.name], capture_output=True, text=True, check=True).stdout
    for name, body in re.findall(r"^[0-9a-f]+ <(.*)>:\n((?:\t.*\n)*)", text, re.M):
        lines = [re.match(r"\t(\S+) *(.*?) *// ([0-9A-F]+): [0-9A-F ]+(?:<.*?(?:\+0x([0-9a-f]+))?>)?$", l) for l in body.splitlines()]
        assert all(lines), name
        first = int(lines[0][3], 16)
        index = {int(l[3], 16) - first: i for i, l in enumerate(lines)}
        yield name, [(l[1], l[2].split(", "), index[int(l[4] or "0", 16)] if l[1].startswith(("s_branch", "s_cbranch")) else None)
                     for l in lines]


def vector_writes(name, ops):
    """Scalar registers that a vector instruction writes."""
    if name.startswith(("v_readfirstlane", "v_readlane", "v_cmp")):
        return scalars(ops[0])
    if name.startswith("v_") and ("_co_" in name or name.startswith(("v_mad_u64", "v_mad_i64", "v_div_scale"))):
        return scalars(ops[1])
    return set()


def too_early(body):
    """Memory instructions that some way through the kernel reaches too early: (index, mnemonic, operands, wait states)."""
    # at each instruction, the wait states since a register was written, by (register, how)
    need = {"vector": 5, "m0": 1}
    state = [None] * len(body)
    state[0], stack = {}, [0]

    def reach(i, new):
        old = state[i]
        if old is not None and all(old.get(r, 9) <= n for r, n in new.items()):
            return
        state[i] = dict(new) if old is None else {r: min(old.get(r, 9), new.get(r, 9)) for r in {*old, *new}}
        stack.append(i)

    while stack:
        i = stack.pop()
        name, ops, target = body[i]
        passed = int(ops[0], 0) + 1 if name == "s_nop" else 1
        after = {r: n + passed for r, n in state[i].items() if n + passed < need[r[1]]}
        if name.startswith("s_") and not name.startswith(("s_cmp", "s_bitcmp", "s_nop", "s_waitcnt", "s_branch", "s_cbranch")):
            for r in scalars(ops[0]):              # the scalar ALU's write takes the register over
                after.pop((r, "vector"), None)
                if r == M0:
                    after[M0, "m0"] = 0
        for r in vector_writes(name, ops):
            after[r, "vector"] = 0
        if target is not None:
            reach(target, after)
        if name not in ("s_branch", "s_endpgm", "s_setpc_b64") and i + 1 < len(body):
            reach(i + 1, after)
    found = []
    for i, (name, ops, _) in enumerate(body):
        if name.startswith(MEMORY) and state[i]:
            read = {(r, "vector") for r in scalars(", ".join(ops))} | ({(M0, "m0")} if "_lds_" in name else set())
            found += [(i, name, ops, state[i][r]) for r in sorted(read & set(state[i]))]
    return found


def test_the_search_finds_what_it_looks_for():
    copy = ("global_load_lds_dwordx4", ["v1", "s[2:3]"], None)
    lane, move, m0, end = ("v_readfirstlane_b32", ["s3", "v0"], None), ("s_mov_b64", ["s[2:3]", "s[4:5]"], None), \
        ("s_mov_b32", ["m0", "s6"], None), ("s_endpgm", [""], None)
    nop = lambda n: ("s_nop", [str(n)], None)
    assert too_early([lane, m0, nop(0), copy, end]) == [(3, *copy[:2], 2)]
    assert not too_early([lane, m0, nop(3), copy, end]) and not too_early([lane, m0, move, copy, end])
    assert too_early([m0, copy, end]) == [(1, *copy[:2], 0)]
    # around a loop: the write behind the copy reaches it by the branch back
    assert too_early([m0, nop(0), copy, lane, ("s_cbranch_scc1", ["1"], 2), end]) == [(2, *copy[:2], 1)]


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_copies_into_lds_wait_for_their_scalar_registers():
    copies, bad = 0, []
    for code in code_objects(S.LIB_PATH):
        for name, body in kernels(code):
            copies += sum(n.startswith("global_load_lds") for n, _, _ in body)
            bad += [(name, *b) for b in too_early(body)]
    assert copies > 1000                           # the library's kernels were read
    assert not bad, (len(bad), bad[:4])
