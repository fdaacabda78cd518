"""The compiled MXFP4 kernels keep the waits that matrix instructions need (no GPU: the library's own device code is
listed and walked).

The hardware does not hold back an instruction that touches the result of a matrix instruction in flight.  For the
16 x 16 instructions of four passes that these kernels use, eight wait states have to lie between the two, and two
between a vector instruction's result and the matrix instruction that reads it; a matrix instruction may take another's
whole result as its addend at once.  The compiler sees to it where it knows the instruction, and not where the
instruction is written as inline assembly.
"""
import os
import re
import shutil
import subprocess

import pytest

from weight_only_bit_group_amd import build

RESULT_WAIT, OPERAND_WAIT = 8, 2
FOUR_PASSES = ("v_mfma_scale_f32_16x16x128_f8f6f4", "v_mfma_f32_16x16x32_bf16")
_OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")) if p and os.path.exists(p)), None)
_REG = re.compile(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+))(?![\w:\[])")


def _regs(text):
    """The vector registers that an operand text names, as (file, number)."""
    out = set()
    for m in _REG.finditer(text):
        lo, hi = (int(m[2]), int(m[3])) if m[2] else (int(m[4]), int(m[4]))
        out.update((m[1], i) for i in range(lo, hi + 1))
    return out


class Instr:
    def __init__(self, text):
        self.text = text
        self.op, _, rest = text.partition(" ")
        ops = [o.strip() for o in re.split(r",(?![^\[]*\])", rest)]
        self.all = _regs(rest)
        self.mfma = self.op.startswith(("v_mfma", "v_smfma"))
        # (a compare writes scalar registers first, a store's first operand is an address: _regs of the first operand
        # only matters for vector instructions)
        self.dst = _regs(ops[0]) if self.op.startswith("v_") else set()
        if self.mfma:
            self.addend = _regs(ops[3])
            self.reads = _regs(",".join(ops[1:3] + ops[4:]))
        self.waits = int(rest.split()[0], 0) + 1 if self.op == "s_nop" else 1
        self.next = []


def parse(listing):
    """{kernel: [Instr]} of an objdump listing, the successors of each filled in."""
    kernels, at = {}, {}
    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if head:
            name, base = head[2], int(head[1], 16)
            kernels[name], at = [], {}
            continue
        m = re.match(r"^\s+(\S.*?)\s*// ([0-9A-F]+):[^<]*(?:<(.+?)(?:\+0x([0-9a-f]+))?>)?$", line)
        if not m:
            continue
        i = Instr(m[1])
        i.target = base + int(m[4] or "0", 16) if m[3] else None
        i.addr = int(m[2], 16)
        at[i.addr] = i
        kernels[name].append(i)
        kernels[name][-1].map = at
    for code in kernels.values():
        for i, nxt in zip(code, code[1:] + [None]):
            assert not i.op.startswith(("s_setpc", "s_swappc", "s_cbranch_i", "s_cbranch_g")), i.text
            if i.op == "s_endpgm":
                continue
            if i.op in ("s_branch",) or i.op.startswith("s_cbranch"):
                assert i.target in i.map, i.text
                i.next.append(i.map[i.target])
            if i.op != "s_branch" and nxt is not None:
                i.next.append(nxt)
    return kernels


def _within(start, wait):
    """The instructions that come, on some path, before `wait` wait states after `start` have passed."""
    seen, todo = {}, [(n, 0) for n in start.next]
    while todo:
        i, passed = todo.pop()
        if passed >= wait or seen.get(id(i), wait) <= passed:
            continue
        seen[id(i)] = passed
        yield i, passed
        todo += [(n, passed + i.waits) for n in i.next]


def faults(code):
    """(instruction, the one that comes too early after it, wait states between them)."""
    out = []
    for i in code:
        if i.mfma:
            for j, passed in _within(i, RESULT_WAIT):
                if not i.dst & j.all:
                    continue
                if j.mfma and j.addend == i.dst and j.dst == i.dst and not j.reads & i.dst:
                    continue
                out.append((i.text, j.text, passed))
        elif i.dst:
            for j, passed in _within(i, OPERAND_WAIT):
                if j.mfma and i.dst & (j.reads | j.addend):
                    out.append((i.text, j.text, passed))
    return out


def _listing(lines):
    """An objdump listing of one kernel with an instruction every 8 bytes; "-> n" gives a branch's target line."""
    text = ["0000000000001000 <k>:"]
    for n, line in enumerate(lines):
        line, _, to = line.partition(" -> ")
        text.append(f"\t{line} // {0x1000 + 8 * n:012X}: 00000000" + (f" <k+0x{8 * int(to):x}>" if to else ""))
    return "\n".join(text)


A4 = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[0:3], v[4:7], a[0:3], v8, v9 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
A16 = "v_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], v[4:7], a[4:7]"


@pytest.mark.parametrize("lines,count", [
    ([A4, "s_nop 7", "v_accvgpr_read_b32 v0, a3", "s_endpgm"], 0),
    ([A4, "s_nop 6", "v_accvgpr_read_b32 v0, a3", "s_endpgm"], 1),
    ([A4, "s_nop 6", "v_mov_b32_e32 v1, v2", "v_accvgpr_read_b32 v0, a3", "s_endpgm"], 0),
    ([A4, "s_nop 1", "v_accvgpr_read_b32 v0, a4", "s_endpgm"], 0),            # another accumulator
    ([A4, "s_nop 1", A4, "s_nop 7", "ds_write_b32 v0, a1", "s_endpgm"], 0),   # the addend of the next one
    ([A4, A16, "ds_write_b32 v0, a1", "s_endpgm"], 1),
    ([A4, "s_nop 3", "global_store_dwordx4 v[0:1], a[2:5], off", "s_endpgm"], 1),
    ([A4, "s_cbranch_scc1 2 -> 4", "s_nop 7", "s_nop 0", "v_accvgpr_mov_b32 a9, a2", "s_endpgm"], 1),   # by the branch alone
    (["v_accvgpr_mov_b32 a9, a0", "s_nop 3", A4, "s_cbranch_scc1 -3 -> 0", "s_endpgm"], 1),             # on the back edge
    (["s_nop 0", "v_accvgpr_mov_b32 a9, a0", "s_nop 3", A4, "s_nop 7", "s_cbranch_scc1 -3 -> 0", "s_endpgm"], 0),
    (["v_mov_b32_e32 v5, v9", "s_nop 0", A4, "s_endpgm"], 1),
    (["v_mov_b32_e32 v8, v9", "s_nop 1", A4, "s_endpgm"], 0),
    (["v_accvgpr_write_b32 a2, 0", "s_nop 0", A4, "s_endpgm"], 1),
    (["v_mov_b32_e32 v10, v9", A4, "s_endpgm"], 0),
])
def test_the_walk_finds_what_comes_too_early(lines, count):
    assert len(faults(parse(_listing(lines))["k"])) == count


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The MXFP4 kernels of the built library."""
    if not os.path.exists(build.LIB_PATH):
        pytest.skip("libaq.so not built")
    if _OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    here = tmp_path_factory.mktemp("code")
    shutil.copy(build.LIB_PATH, here / "lib.so")
    subprocess.run([_OBJDUMP, "--offloading", "lib.so"], cwd=here, check=True, capture_output=True)
    found = {}
    for part in sorted(here.glob("lib.so.*gfx950")):
        symbols = subprocess.run([_OBJDUMP, "-t", part], check=True, capture_output=True, text=True).stdout
        if "mxfp4_" not in symbols:
            continue
        listing = subprocess.run([_OBJDUMP, "-d", part], check=True, capture_output=True, text=True).stdout
        found.update((k, v) for k, v in parse(listing).items() if "mxfp4_" in k)
    return found


def test_compiled_kernels_wait_for_matrix_results(kernels):
    with_mfma = {name: code for name, code in kernels.items() if any(i.mfma for i in code)}
    assert sum("mxfp4_split_kernel" in n for n in with_mfma) >= 8 and sum("mxfp4_tile_kernel" in n for n in with_mfma) >= 8
    assert {i.op for code in with_mfma.values() for i in code if i.mfma} <= set(FOUR_PASSES)
    found = {name: faults(code) for name, code in with_mfma.items()}
    bad = {name: f for name, f in found.items() if f}
    assert not bad, f"{len(bad)} of {len(found)} kernels, the first: {next(iter(bad.items()))}"
