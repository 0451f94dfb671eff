"""The machine code built here, read on the CPU: loads that go straight to LDS
take their place there from m0 and their buffer from scalar registers, and
the hardware does not wait for either where they were written just before
(one wait state after a scalar write of m0, five after a vector instruction's
write of a scalar register).  Code inside an asm block has to see to that
itself.  No kernel is launched here."""
import os
import re
import shutil
import struct
import subprocess

import pytest

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump") or "")
                if os.path.exists(p)), None)


def device_code(path):
    """The gfx950 code objects in a library (uncompressed bundles)."""
    data = open(path, "rb").read()
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(magic))
        pos = at + len(magic) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, pos)
            name = data[pos + 24:pos + 24 + length]
            pos += 24 + length
            if b"gfx950" in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(magic, at + 1)


def scalars(text):
    """Numbers of the scalar registers that an operand list names."""
    out = set()
    for low, high, one in re.findall(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        out |= set(range(int(low), int(high) + 1)) if low else {int(one)}
    return out


def faults(lines):
    """(loads to LDS, those that come too early, as texts)"""
    loads, bad, before = 0, [], []
    for line in lines:
        op, _, args = line.partition(" ")
        if op.startswith("buffer_load") and re.search(r"\blds\b", args):
            loads += 1
            reads, states = scalars(args), 0
            for x in reversed(before):
                o, _, a = x.partition(" ")
                to = a.split(",")[0]
                if o.startswith("s_") and to == "m0" and states < 1:
                    bad.append(f"{x}; {line}")
                if o.startswith("v_") and scalars(to) & reads and states < 5:
                    bad.append(f"{x}; ({states} states) {line}")
                states += int(a, 0) + 1 if o == "s_nop" else 1
                if states >= 5:
                    break
        before = before[-8:] + [line]
    return loads, bad


def test_faults_are_seen():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    assert faults(["s_mov_b32 m0, s8", load]) == (1, ["s_mov_b32 m0, s8; " + load])
    assert faults(["s_add_u32 m0, m0, 0x400", load])[1]
    assert not faults(["s_mov_b32 m0, s8", "s_nop 0", load])[1]
    assert faults(["v_readlane_b32 s6, v9, 3", "s_mov_b32 m0, s8", "s_nop 2", load])[1]
    assert not faults(["v_readlane_b32 s6, v9, 3", "s_mov_b32 m0, s8", "s_nop 3", load])[1]
    assert not faults(["v_readlane_b32 s8, v9, 3", "s_mov_b32 m0, s8", "s_nop 0", load])[1]


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_loads_to_lds_wait_for_what_they_read(tmp_path):
    import lossless_bf16_kv_split_amd as sz
    loads, bad = 0, []
    for i, code in enumerate(device_code(sz.lib_path)):
        path = tmp_path / f"{i}.o"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(path)],
                              check=True, capture_output=True, text=True).stdout
        lines = [line.split("//")[0].strip() for line in text.splitlines()]
        n, b = faults([x for x in lines if x and not x.endswith(":")])
        loads, bad = loads + n, bad + b
    assert loads > 0
    assert not bad, (len(bad), bad[:3])
