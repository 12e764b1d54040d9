"""What the compiler made of latent attention's kernels, read from this build's own objects.

Where registers are full, the compiler (AMD clang 22 of ROCm 7.2) has placed copies that
free registers between a branch's join and the instruction that brings the lanes back,
so that lanes which had not taken the branch lost their values.  The kernels are written to
give it no occasion: among their matrix instructions no branch is one that lanes take by
themselves.  Two things are held here: from a kernel's first matrix instruction to its last
no instruction writes the lane mask, and nowhere in these objects does a vector instruction
stand between a join and its restore of the mask."""
import os
import re
import shutil
import subprocess

import pytest

from gated_delta_rule_55_amd import build

OBJDUMP = shutil.which("llvm-objdump") or os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin",
                                                       "llvm-objdump")
# kernels with matrix instructions: (dn, dr, dv) or (dc, dr) each way, two types; units of 64 in bf16 alone
OBJECTS = {"kda_latent_attend": 12, "kda_latent_prefill": 16, "kda_latent_cache": 0}
# (readlane and its like work on one lane whatever the mask)
VECTOR = re.compile(r"(v_(?!readlane|writelane|readfirstlane)|ds_|buffer_|global_|flat_|scratch_)")
WRITES_MASK = re.compile(r"(s_\w+_saveexec_b64|s_\w+ exec(_lo|_hi)?,|v_cmpx)")


def kernels(text):
    """Functions of a disassembly: name -> its lines, labels ('<L12>:') among them."""
    out, lines = {}, None
    for line in text.splitlines():
        line = line.split("//")[0].strip()
        m = re.match(r"(?:[0-9a-f]+ )?<([^>]+)>:$", line)
        if m and not re.fullmatch(r"L\d+", m.group(1)):
            lines = out.setdefault(m.group(1), [])
        elif line and lines is not None:
            lines.append(f"<{m.group(1)}>:" if m else line)
    return out


def masks_among_products(lines):
    """Writes of the lane mask between the first matrix instruction and the last."""
    at = [i for i, x in enumerate(lines) if x.startswith("v_mfma")]
    return [x for x in lines[at[0]:at[-1]] if WRITES_MASK.match(x)] if at else []


def copies_before_restores(lines):
    """Vector instructions between a label and an `s_or_b64 exec` that follows without a branch."""
    found, block = [], None
    for x in lines:
        if x.startswith("<"):
            block = []
        elif block is not None:
            if x.startswith("s_or_b64 exec, exec,"):
                found += block
                block = None
            elif x.startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc")) or WRITES_MASK.match(x):
                block = None
            elif VECTOR.match(x):
                block.append(x)
    return found


@pytest.mark.parametrize("name", OBJECTS)
def test_lanes_stay_together(name, tmp_path):
    obj = os.path.join(build.PKG, "_build", name + ".o")
    if not (os.path.exists(obj) and os.path.exists(OBJDUMP)):
        pytest.skip("needs the library's objects (build first) and llvm-objdump")
    copy = shutil.copy(obj, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", copy], cwd=tmp_path, check=True, capture_output=True)
    code = [os.path.join(tmp_path, f) for f in os.listdir(tmp_path) if build.ARCH in f]
    assert len(code) == 1
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", code[0]], check=True,
                          capture_output=True, text=True).stdout
    found = kernels(text)
    assert sum(any(x.startswith("v_mfma") for x in lines) for lines in found.values()) == OBJECTS[name]
    for kernel, lines in found.items():
        assert not masks_among_products(lines), kernel
        assert not copies_before_restores(lines), kernel


PLANTED = """
0000000000001000 <kernel>:
    v_cmp_gt_i32_e32 vcc, 5, v0           // 000000001000: 7D880085
    s_and_saveexec_b64 s[2:3], vcc
    s_cbranch_execz L0
    v_mov_b32_e32 v1, 0
<L0>:
    {join}
    s_or_b64 exec, exec, s[2:3]
    v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]
    {among}
    v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]
    v_cmpx_gt_i32_e32 5, v0
    s_endpgm
"""


@pytest.mark.parametrize("join,among,copies,masks", [
    ("s_nop 0", "s_nop 0", 0, 0), ("v_writelane_b32 v9, s4, 0", "s_mov_b64 s[4:5], exec", 0, 0),
    ("v_mov_b32_e32 v2, v1", "s_nop 0", 1, 0), ("v_accvgpr_write_b32 a3, v1", "s_nop 0", 1, 0),
    ("scratch_load_dword v2, off, s0", "s_nop 0", 1, 0), ("s_nop 0", "s_and_saveexec_b64 s[4:5], vcc", 0, 1),
    ("s_nop 0", "s_mov_b64 exec, s[4:5]", 0, 1), ("s_nop 0", "s_xor_b64 exec, exec, s[4:5]", 0, 1),
])
def test_planted_code_is_found(join, among, copies, masks):
    (lines,) = kernels(PLANTED.format(join=join, among=among)).values()
    assert len(copies_before_restores(lines)) == copies and len(masks_among_products(lines)) == masks
