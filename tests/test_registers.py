"""What the compiler made of the full-attention layers' kernels (CPU only, from the built library's own code).

In an earlier form of the attention kernel the compiler, short of registers, put some aside and brought them back at the end of a
branch in front of the instruction that makes the other lanes active again: those kept old values, and rows came out wrong.  So
no kernel of these files may put vector registers aside at all, and no register may be brought back at such a place."""
import os
import re
import struct
import subprocess

import pytest

from tests.test_abi import kda  # noqa: F401  (fixture)

LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
KERNELS = re.compile(r"paged_attention_kernel|attention_chunk_kernel|join_pieces_kernel|append_kv_kernel|read_kv_kernel|qk_norm_rope")
WIDENS = re.compile(r"s_(?:or|mov|andn2|xor|orn2)_b64 exec|s_or_saveexec_b64|s_cselect_b64 exec")
BACK = re.compile(r"v_accvgpr_read|scratch_load")


def code_objects(path):
    """The gfx950 code objects of a HIP library."""
    data, magic, at = open(path, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        entry = at + len(magic) + 8
        for _ in range(struct.unpack_from("<Q", data, at + len(magic))[0]):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            if b"gfx950" in data[entry + 24:entry + 24 + length] and size:
                yield data[at + offset:at + offset + size]
            entry += 24 + length
        at += len(magic)


def functions(listing):
    """(name, lines) of a disassembly with labels."""
    for part in re.split(r"\n(?=[0-9a-f]+ <_Z)", listing):
        if m := re.match(r"[0-9a-f]+ <(_Z\w+)>:\n", part):
            yield m[1], part[m.end():].splitlines()


def brought_back_too_early(lines):
    """Registers brought back between the end of a branch that some lanes did not take and the instruction that makes
    those lanes active."""
    ends = {m[1] for line in lines if (m := re.search(r"s_cbranch_execz (L\d+)", line))}
    found, narrow = [], False
    for line in lines:
        if m := re.match(r"[0-9a-f]+ <(L\d+)>:", line):
            narrow = m[1] in ends
        elif narrow and (WIDENS.search(line) or re.search(r"s_(?:c?branch|endpgm)", line)):
            narrow = False
        elif narrow and BACK.search(line):
            found.append(line.strip())
    return found


def test_the_scan_itself():
    head = ["\ts_and_saveexec_b64 s[0:1], vcc  // 0", "\ts_cbranch_execz L1  // 4", "\tv_add_f32_e32 v0, v0, v1  // 8", "", "0000000000000010 <L1>:"]
    back, wide = "\tv_accvgpr_read_b32 v3, a7  // 10", "\ts_or_b64 exec, exec, s[0:1]  // 18"
    assert brought_back_too_early(head + [back, wide]) == [back.strip()]
    assert brought_back_too_early(head + ["\tscratch_load_dword v3, off, off offset:8  // 10", wide])
    assert brought_back_too_early(head + [wide, back]) == []
    assert brought_back_too_early([x.replace("execz", "scc0") for x in head] + [back, wide]) == []


@pytest.fixture(scope="module")
def library(kda):  # noqa: F811
    if not os.path.exists(os.path.join(LLVM, "llvm-objdump")):
        pytest.skip("no llvm-objdump")
    return [x for x in code_objects(kda.LIB_PATH)]


def test_nothing_is_put_aside(library, tmp_path):
    seen = 0
    for i, code in enumerate(library):
        path = tmp_path / f"{i}.elf"
        path.write_bytes(code)
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", path], capture_output=True, text=True, check=True).stdout
        for kernel in re.split(r"\n  - ", notes):
            name = re.search(r"\.name: +(_Z\w+)\n", kernel)
            if name and KERNELS.search(name[1]):
                seen += 1
                for of in ("vgpr_spill_count", "private_segment_fixed_size"):
                    assert re.search(rf"\.{of}: +(\d+)", kernel)[1] == "0", (name[1], of)
    assert seen >= 90


def test_nothing_is_brought_back_too_early(library, tmp_path):
    seen = 0
    for i, code in enumerate(library):
        path = tmp_path / f"{i}.elf"
        path.write_bytes(code)
        listing = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--symbolize-operands", "--no-show-raw-insn", path],
                                 capture_output=True, text=True, check=True).stdout
        for name, lines in functions(listing):
            if KERNELS.search(name):
                seen += 1
                assert not brought_back_too_early(lines), name
    assert seen >= 90
