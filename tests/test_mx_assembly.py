"""The built MXFP4 kernels keep the wait states of the matrix instruction.

The tile kernel writes v_mfma_scale_* as inline assembly, for which the compiler inserts no waits: that no vector instruction
writes an operand right before it, and that its sums are left alone until they are there, depends on the registers
and the order that the compiler happens to choose. The disassembly of the built library is followed along every path:
  - two wait states between a vector instruction that writes an operand (a sum's old value included) and the MFMA;
  - 18 wait states between the MFMA and anything but an MFMA's own accumulation that touches its sums.
An instruction counts as one wait state, s_nop n as n + 1."""
import os
import re
import shutil
import subprocess

import pytest

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")

BEFORE, AFTER = 2, 18
OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")


def registers(text):
    found = set()
    for file, first, last, single in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        found.update((file, i) for i in (range(int(first), int(last) + 1) if first else [int(single)]))
    return found


class Instruction:
    def __init__(self, address, text):
        self.address = address
        self.op, _, rest = text.strip().partition(" ")
        self.args = [a.strip() for a in re.split(r",(?![^\[]*\])", rest)] if rest else []
        self.mfma = self.op.startswith("v_mfma")
        self.states = int(self.args[0], 0) + 1 if self.op == "s_nop" else 1
        self.touched = registers(rest)
        self.writes = set()
        if self.op.startswith("v_") and not self.mfma and self.args:
            self.writes = registers(" ".join(self.args[:2]) if "swap" in self.op else self.args[0])
        if self.mfma:
            self.sums = registers(self.args[0])
            scales = [a.split()[0] for a in self.args[4:6]]
            self.factors = registers(" ".join(self.args[1:3] + scales))
            self.operands = self.factors | registers(self.args[3].split()[0])


def functions(listing):
    """name -> (instructions in order, predecessors of each: their indexes)."""
    base, bodies, name = {}, {}, None
    for line in listing.splitlines():
        head = re.match(r"([0-9a-f]+) <(\S+)>:$", line)
        if head:
            name = head[2]
            base[name], bodies[name] = int(head[1], 16), []
            continue
        body = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):", line)
        if body and name:
            target = re.search(r"<(\S+?)(?:\+0x([0-9a-f]+))?>\s*$", line)
            bodies[name].append((Instruction(int(body[2], 16), body[1]), target))
    for name, body in bodies.items():
        at = {i.address: n for n, (i, _) in enumerate(body)}
        before = [set() for _ in body]
        for n, (i, target) in enumerate(body):
            if n + 1 < len(body) and i.op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                before[n + 1].add(n)
            if i.op.startswith(("s_branch", "s_cbranch")):
                assert target, f"a branch without its target: {i.op} {i.args}"
                before[at[base[target[1]] + int(target[2] or "0", 16)]].add(n)
        yield name, [i for i, _ in body], before


def hazards(listing):
    """(matrix instructions seen, descriptions of what comes too soon)."""
    count, bad = 0, []
    for name, code, before in functions(listing):
        for n, here in enumerate(code):
            if not (here.mfma or here.touched):
                continue
            count += here.mfma
            # backwards over every path; `left` of a place: the most wait states still to be looked through from it
            left, todo = {}, [(p, AFTER) for p in before[n]]
            while todo:
                p, states = todo.pop()
                if states <= left.get(p, 0):
                    continue
                left[p] = states
                there = code[p]
                if there.mfma:
                    # an MFMA may take up sums where another left them, in whole
                    own = here.mfma and here.sums == there.sums
                    if there.sums & (here.factors if own else here.touched):
                        bad.append(f"{name}: {there.op} {there.args} then {here.op} {here.args}")
                elif here.mfma and AFTER - states < BEFORE and there.writes & here.operands:
                    bad.append(f"{name}: {there.op} {there.args} then {here.op} {here.args}")
                todo.extend((q, states - there.states) for q in before[p])
    return count, bad


def listing_of(library, folder):
    """The library's device code, disassembled."""
    shutil.copy(library, os.path.join(folder, "lib.so"))
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=folder, check=True, capture_output=True)
    parts = sorted(f for f in os.listdir(folder) if "gfx950" in f)
    assert parts
    for part in parts:
        yield subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", "--no-show-raw-insn", part], cwd=folder, check=True, capture_output=True,
                             text=True).stdout


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump of ROCm")
def test_matrix_instructions_keep_their_wait_states(tmp_path):
    texts = [t for t in listing_of(fp4.LIB_PATH, tmp_path) if "gemm_kernelINS_4Tile" in t]
    assert len(texts) == 1
    assert len(re.findall(r"<_ZN2mx11gemm_kernelINS_4Tile\S+>:", texts[0])) == 9       # three tiles, three output types
    count, bad = hazards(texts[0])
    assert count > 500 and not bad, bad[:5]


# ---------------------------------------------------------------------------------------------- of the check itself

MFMA = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[6:9], v[62:65], a[0:3], v178, v172 op_sel_hi:[0,0,0] cbsz:4 blgp:4"


def lines(*code, name="f"):
    out = ["0000000000001000 <f>:"]
    at = {}
    for n, text in enumerate(code):
        if ":" in text.split()[0] and not text.startswith("v_"):
            label, text = text.split(": ", 1)
            at[label] = 4 * n
        out.append((n, text))
    done = [out[0]]
    for n, text in out[1:]:
        op, _, label = text.partition(" @")
        done.append(f"\t{op} // {0x1000 + 4 * n:012X}:" + (f" BF880000 <f+0x{at[label]:x}>" if label else " BF800000"))
    return "\n".join(done)


@pytest.mark.parametrize("write", ["v_mov_b32_e32 v7, 0", "v_perm_b32 v172, v1, v2, v3", "v_accvgpr_write_b32 a2, 0",
                                   "v_permlane32_swap_b32 v1, v62"])
def test_the_check_sees_an_operand_written_too_late(write):
    other = "s_add_i32 s0, s0, 1"
    assert hazards(lines(write, MFMA, "s_endpgm"))[1]
    assert hazards(lines(write, other, MFMA, "s_endpgm"))[1]
    assert not hazards(lines(write, other, other, MFMA, "s_endpgm"))[1]
    assert hazards(lines(write, "s_nop 0", MFMA, "s_endpgm"))[1]
    assert hazards(lines(write, "s_nop 1", MFMA, "s_endpgm")) == (1, [])
    assert not hazards(lines("v_mov_b32_e32 v10, v7", MFMA, "s_endpgm"))[1]            # reads it
    # around a loop: the write at its end, the MFMA at its start
    around = lines("s_nop 15", "top: " + MFMA, "s_nop 15", "s_nop 15", write, "s_cbranch_scc1 @top", "s_endpgm")
    assert hazards(around)[1]


@pytest.mark.parametrize("use", ["v_accvgpr_read_b32 v1, a3", "global_store_dwordx4 v1, a[0:3], s[2:3]", "v_accvgpr_write_b32 a0, 0",
                                 MFMA.replace("a[0:3]", "a[2:5]"), MFMA.replace("a[0:3]", "a[4:7]").replace("v[6:9]", "a[0:3]")])
def test_the_check_sees_sums_touched_too_early(use):
    assert hazards(lines(MFMA, use, "s_endpgm"))[1]
    assert hazards(lines(MFMA, "s_nop 15", "s_nop 0", use, "s_endpgm"))[1]
    assert not hazards(lines(MFMA, "s_nop 15", "s_nop 1", use, "s_endpgm"))[1]
    assert not hazards(lines(MFMA, MFMA, MFMA, "s_endpgm"))[1]


def test_the_check_follows_branches():
    code = lines("s_cbranch_scc1 @far", "v_mov_b32_e32 v6, 0", "s_branch @far", "s_nop 15", "far: " + MFMA, "s_endpgm")
    assert hazards(code)[1]
    assert not hazards(code.replace("v6, 0", "v5, 0"))[1]
