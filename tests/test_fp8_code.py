"""The compiled FP8 products keep the waits that matrix instructions need (no GPU: the library's own device code is
listed and walked, see test_mxfp4_code).

The FP8 instruction of 16 x 16 x 128 has eight passes and needs twelve wait states between it and a reader of its result,
the bf16 one of 16 x 16 x 32 four and eight; two lie between a vector instruction's result and the matrix instruction
that reads it.  A matrix instruction may take another's whole result as its addend at once, and one of the same kind
may write the same registers behind it.  The compiler sees to the waits but has lost them where a branch came between
an instruction and its result's reader.
"""
import os
import shutil
import subprocess

import pytest

from tests.test_mxfp4_code import _OBJDUMP, _listing, _within, parse
from weight_only_bit_group_amd import build

RESULT_WAIT = {"v_mfma_f32_16x16x128_f8f6f4": 12, "v_mfma_f32_16x16x32_bf16": 8}
OPERAND_WAIT = 2


def faults(code):
    """(instruction, the one that comes too early after it, wait states between them)."""
    out = []
    for i in code:
        if i.mfma:
            for j, passed in _within(i, RESULT_WAIT[i.op]):
                if not i.dst & j.all:
                    continue
                if j.mfma and j.op == i.op and not j.reads & i.dst and (j.addend == i.dst or not j.addend & i.dst):
                    continue
                out.append((i.text, j.text, passed))
        elif i.dst:
            for j, passed in _within(i, OPERAND_WAIT):
                if j.mfma and i.dst & (j.reads | j.addend):
                    out.append((i.text, j.text, passed))
    return out


F8 = "v_mfma_f32_16x16x128_f8f6f4 v[0:3], v[8:15], v[16:23], 0"
F16 = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[4:7]"


@pytest.mark.parametrize("lines,count", [
    ([F8, "s_nop 11", "v_fmac_f32_e32 v40, v3, v41", "s_endpgm"], 0),
    ([F8, "s_nop 10", "v_fmac_f32_e32 v40, v3, v41", "s_endpgm"], 1),
    ([F8, F8, "s_nop 11", "v_fmac_f32_e32 v40, v3, v41", "s_endpgm"], 0),
    ([F16, "v_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], v[0:3]", "s_nop 7", "v_mov_b32_e32 v40, v4", "s_endpgm"], 0),
    ([F16, "v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], 0", "s_nop 7", "s_endpgm"], 1),
    ([F16, "s_cbranch_scc1 2 -> 3", "s_nop 7", "v_mov_b32_e32 v40, v4", "v_mov_b32_e32 v40, v1", "s_endpgm"], 1),
    (["v_mov_b32_e32 v8, v41", "s_nop 0", F8, "s_endpgm"], 1),
])
def test_the_walk_finds_what_comes_too_early(lines, count):
    assert len(faults(parse(_listing(lines))["k"])) == count


def test_compiled_kernels_wait_for_matrix_results(tmp_path):
    if not os.path.exists(build.LIB_PATH):
        pytest.skip("libaq.so not built")
    if _OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    shutil.copy(build.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([_OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    kernels = {}
    for part in sorted(tmp_path.glob("lib.so.*gfx950")):
        symbols = subprocess.run([_OBJDUMP, "-t", part], check=True, capture_output=True, text=True).stdout
        if "fp8_tile_kernel" in symbols:
            listing = subprocess.run([_OBJDUMP, "-d", part], check=True, capture_output=True, text=True).stdout
            kernels.update((k, v) for k, v in parse(listing).items() if "fp8_" in k and any(i.mfma for i in v))
    assert sum("fp8_split_kernel" in n for n in kernels) >= 16 and sum("fp8_tile_kernel" in n for n in kernels) >= 8
    assert {i.op for code in kernels.values() for i in code if i.mfma} == set(RESULT_WAIT)
    found = {name: faults(code) for name, code in kernels.items()}
    bad = {name: f for name, f in found.items() if f}
    assert not bad, f"{len(bad)} of {len(found)} kernels, the first: {next(iter(bad.items()))}"
