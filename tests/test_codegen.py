"""What the compiler made of the library's LDS stores (its disassembly; no GPU).

This compiler merges two 4- or 8-byte LDS stores at constant offsets into one instruction. Where an accumulator register
(AGPR) is the value of some of them and a VGPR that of others, it gives up one pairing after it has already divided an
offset by the element's size, and divides it again in the next: of the 16 stores of four 16 x 16 tiles with rows of 68
floats it made ds_write2_b32 .. offset0:51 offset1:220 where the source has elements 204 and 220. Such a kernel shows the
stores that were left single, with an AGPR as their value; 16-byte stores are not merged and may have them."""
import os
import re
import shutil
import subprocess

import pytest

TOOLS = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MERGED = re.compile(r"\bds_write(2|2st64)?_b(8|16|32|64)\S*\s+(.*)")


def agpr_stores(lines):
    """(function, instruction) of the LDS stores of up to 8 bytes whose value is an AGPR."""
    found, name = [], ""
    for line in lines:
        if line.startswith("_Z") or re.match(r"[0-9a-f]+ <", line):
            name = line.strip()
        m = MERGED.search(line)
        if m and any(re.match(r"a(\d|\[)", op.strip()) for op in m.group(3).split("//")[0].split(",")[1:]):
            found.append((name, line.strip()))
    return found


def test_the_mark_is_seen():
    bad = ["_Zkernel:", "\tds_write_b32 v52, a6 offset:608", "\tds_write2_b32 v52, v0, v1 offset0:51 offset1:220",
           "\tds_write_b128 v29, a[4:7] offset:17408", "\tds_write_b64 v1, a[2:3]", "0000 <next>:",
           "\tds_write2_b32 v7, v3, a1 offset1:68   // 00000007B730: D9B60000"]
    assert [b[1].split()[0] for b in agpr_stores(bad)] == ["ds_write_b32", "ds_write_b64", "ds_write2_b32"]
    assert agpr_stores(bad)[0][0] == "_Zkernel:" and agpr_stores(bad)[2][0] == "0000 <next>:"


def test_no_small_lds_store_has_an_agpr(tmp_path):
    from linear_recurrent_sequence_amd import build, retention
    retention.load()
    tool = os.path.join(TOOLS, "llvm-objdump")
    if not os.path.exists(tool):
        pytest.skip("llvm-objdump is not installed")
    lib = shutil.copy(build.LIB_PATH, tmp_path)
    subprocess.run([tool, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    objects = [f for f in os.listdir(tmp_path) if f.endswith(build.ARCH)]
    assert objects
    stores = 0
    for f in objects:
        text = subprocess.run([tool, "-d", "--no-show-raw-insn", f], cwd=tmp_path, check=True, capture_output=True,
                              text=True).stdout
        lines = text.splitlines()
        stores += sum(MERGED.search(x) is not None for x in lines)
        assert agpr_stores(lines) == [], f
    assert stores > 1000  # the disassembly was one
