"""Wait states of the loads into LDS, in the compiled kernels.

The compiler adds the wait states that the hardware asks for everywhere but inside inline assembly, where the loads
into LDS are written.  Such a load needs one between the scalar write of M0 and itself, and five between
a vector instruction's write of a scalar register that it reads and itself (an instruction counts
as one, s_nop n as n + 1)."""

import os
import re
import shutil
import struct
import subprocess

import pytest

import fp4_grouped_gemm_amd as fgg

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"

pytestmark = [pytest.mark.skipif(not os.path.exists(fgg.library_path()),
                                 reason="libfgg.so not built (run __graft_entry__.build())"),
              pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")]

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
SCALAR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b")


def code_objects(path):
    """The gfx950 code objects of a library's offload bundles (24 bytes of magic, a count, then offset, size and
    name of each)."""
    data = open(path, "rb").read()
    at, out = data.find(MAGIC), []
    while at >= 0:
        (count,), p = struct.unpack_from("<Q", data, at + len(MAGIC)), at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if size and b"gfx950" in data[p + 24:p + 24 + length]:
                out.append(data[at + offset:at + offset + size])
            p += 24 + length
        at = data.find(MAGIC, at + 1)
    return out


def scalars(text):
    for first, last, one in SCALAR.findall(text):
        yield from range(int(first), int(last) + 1) if first else (int(one),)


def short_waits(listing):
    """(loads into LDS, those that come too soon): in the order of the listing, function by function."""
    loads, bad, where = 0, [], ""
    now, m0, written = 0, -9, {}
    for line in listing:
        if line.endswith(">:"):
            where, now, m0, written = line.split("<")[1][:-2], 0, -9, {}
            continue
        line = line.split("//")[0].strip()
        op, _, operands = line.partition(" ")
        if not op.startswith(("s_", "v_", "buffer_load", "global_load_lds")):
            now += 1
            continue
        if op.startswith("global_load_lds") or op.startswith("buffer_load") and operands.endswith(" lds"):
            loads += 1
            between = now - m0 - 1
            if between < 1:
                bad.append((where, line, "M0", between))
            for s in scalars(operands):
                between = now - written.get(s, -9) - 1
                if between < 5:
                    bad.append((where, line, f"s{s}", between))
        dest = operands.split(",")[0]
        if op.startswith("v_") and dest[:1] == "s":
            written.update((s, now) for s in scalars(dest))
        elif op.startswith("s_"):
            if dest == "m0":
                m0 = now
            for s in scalars(dest):
                written.pop(s, None)
        now += int(operands, 0) + 1 if op == "s_nop" else 1
    return loads, bad


def test_the_reader_finds_short_waits():
    text = ["0 <k>:", "v_readfirstlane_b32 s4, v0", "s_mov_b32 m0, s9", "global_load_lds_dword v1, s[4:5]",
            "s_mov_b32 m0, s9", "s_nop 2", "buffer_load_dwordx4 v1, s[4:7], 0 offen lds", "s_mov_b32 s4, 0",
            "s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dword v1, s[4:5]"]
    loads, bad = short_waits(text)
    assert loads == 3 and [b[2:] for b in bad] == [("M0", 0), ("s4", 1)]


def test_loads_into_lds_wait(tmp_path):
    objects = code_objects(fgg.library_path())
    assert objects
    loads, bad = 0, []
    for i, o in enumerate(objects):
        f = tmp_path / f"{i}.co"
        f.write_bytes(o)
        r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], capture_output=True, text=True, check=True)
        n, b = short_waits(r.stdout.splitlines())
        loads, bad = loads + n, bad + b
    assert loads > 1000
    assert not bad, f"{len(bad)} of {loads} loads, e.g. {bad[0]}"
