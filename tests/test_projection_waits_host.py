"""The waits that the hand-written loads of the 8-bit products need, read from the machine code of
the build (no GPU).

A load straight into LDS takes its place there from m0, and its address from a pair of scalar registers.  This
chip does not hold the load back until they are written: one wait state has to pass after the
write of m0, five after a vector instruction (v_readfirstlane, v_readlane) wrote one of the pair.  The compiler keeps to
that for instructions of its own and does not look into assembly."""
import os
import re
import shutil
import struct
import subprocess

import pytest

import genomic_lm_amd as G

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")) if p and os.path.exists(p)),
               None)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(G.LIB_PATH):
        from genomic_lm_amd import build
        build.build()
    yield


def code_objects(data):
    """The gfx950 images in the library's bundles."""
    at = data.find(MAGIC)
    while at >= 0:
        n, = struct.unpack_from("<Q", data, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, p)


def numbers(text):
    """Scalar registers named by an operand list: s7, s[8:9]."""
    out = {int(m) for m in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out


def missing_waits(lines):
    """(loads into LDS, those issued too early).  lines: one kernel's instructions in order."""
    loads, early = 0, []
    for i, text in enumerate(lines):
        if not re.match(r"global_load_lds|buffer_load_\w+ .*\blds\b", text):
            continue
        loads += 1
        pair = numbers(text.split(",", 1)[1])
        states, m0 = 0, False                          # wait states between that line and the load
        for back in reversed(lines[max(0, i - 6):i]):
            op, _, rest = back.partition(" ")
            dest = rest.split(",")[0]
            if op.startswith("s_") and dest == "m0":
                m0 = True
                if states < 1:
                    early.append((back, text, states))
            if op.startswith("v_") and states < 5 and numbers(dest) & pair:
                early.append((back, text, states))
            states += 1 + (int(rest, 0) if op == "s_nop" else 0)
        if not m0:
            early.append(("no write of m0", text, states))
    return loads, early


def test_the_reading_itself():
    good = ["v_readfirstlane_b32 s8, v1", "s_mov_b32 m0, s2", "s_nop 3", "global_load_lds_dwordx4 v34, s[8:9]"]
    assert missing_waits(good) == (1, [])
    assert len(missing_waits(good[:2] + good[3:])[1]) == 2          # m0, and the pair
    assert len(missing_waits(good[:2] + ["s_nop 2"] + good[3:])[1]) == 1
    assert missing_waits(["v_readfirstlane_b32 s10, v1"] + good[1:2] + ["s_nop 0"] + good[3:]) == (1, [])
    assert len(missing_waits(good[3:])[1]) == 1


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_loads_into_lds_wait_for_their_registers(tmp_path):
    kernels = {}
    with open(G.LIB_PATH, "rb") as f:
        data = f.read()
    for k, image in enumerate(code_objects(data)):
        if b"linear_" not in image:
            continue
        path = tmp_path / f"{k}.co"
        path.write_bytes(image)
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(path)], capture_output=True,
                             text=True, check=True).stdout
        name = None
        for line in out.splitlines():
            m = re.match(r"^[0-9a-f]* ?<(\S+)>:$", line)
            if m:
                name = m.group(1)
                kernels[name] = []
            elif name and line.strip():
                kernels[name].append(re.sub(r"\s+", " ", line.split("//")[0]).strip())
    total, early = 0, []
    for name, lines in kernels.items():
        n, bad = missing_waits(lines)
        total += n
        early += [(name, *b) for b in bad]
        if "linear_turns" in name or "_dma_kernel" in name:
            assert n > 0, name
    assert total > 500, total
    assert not early, (len(early), early[:3])
